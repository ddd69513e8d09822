"""GPU tests of the operators between the products of a training step: 8-bit
activation copies, layer norm and its gradients, RMSNorm's gradients, and the
squared-ReLU gate with its gradient, each against a plain 64-bit form.

Tolerances.  u = 2^-24 is fp32's half step, and storing a result in its type
costs a relative eps(T) / 2.  Codes, scales, restored values and everything of
the gate are products of a few fp32 values in a stated order, so they are
compared bit for bit.  A sum of n terms in fp32 is off by at most (depth of the
additions) * u * (sum of magnitudes): a row's sums have at most 128 additions
per thread and 10 tree levels (DEPTH covers them with the terms' own few
roundings), a column's sums at most one addition per row, and beyond 600 rows
they are split into partial sums whose chains are shorter than that."""
import threading

import pytest

import bitlinear_absmean_ternary_b200 as bl
from bitlinear_absmean_ternary_b200 import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEPTH = 160
EPS = 1e-5
GROUP = 64
FLT_MAX = (2.0 - 2.0 ** -23) * 2.0 ** 127
torch = pytest.importorskip("torch")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bl.lib()
    return torch.device("cuda:0")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tensor(dev, M, K, dtype, seed, scale=1.0, shift=0.0, loud=True):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    x = torch.randn(M, K, generator=gen, dtype=torch.float64) * scale
    if loud and K >= 64:
        x[:, (7 * seed + 5) % K] *= 20.0
    return (x + shift).to(DTYPES[dtype]).to(dev)


def vector(dev, K, dtype, seed, lo=0.5, hi=1.5):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(1000 + seed)
    return (torch.rand(K, generator=gen, dtype=torch.float64) * (hi - lo) + lo).to(DTYPES[dtype]).to(dev)


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0.0, (what, float((got - want).abs().max()), float(over.max()))


# ------------------------------------------------------------ 8-bit copies


def codes64(x):
    """Codes and scales by the definition, with its fp32 steps."""
    M, K = x.shape
    v = x.float().cpu().view(M, K // GROUP, GROUP)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2)
    live = (amax >= 2.0 ** -120) & ~bad
    safe = torch.where(live, amax, torch.ones_like(amax))
    inv = torch.full_like(safe, 127.0) / safe
    q = torch.where(live.unsqueeze(2), v * inv.unsqueeze(2), torch.zeros_like(v))
    largest = torch.tensor(FLT_MAX / 127.0, dtype=torch.float64).float()
    largest = largest if float(largest) * 127.0 <= FLT_MAX else torch.nextafter(largest, torch.tensor(0.0))
    scale = torch.where(live, (safe / torch.full_like(safe, 127.0)).minimum(largest), torch.zeros_like(safe))
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return q.round().to(torch.int8).view(M, K), scale


def values64(x8, x_scale):
    M, K = x8.shape
    return (x8.double().view(M, K // GROUP, GROUP) * x_scale.double().unsqueeze(2)).view(M, K)


COPY_SHAPES = [(1, 64), (1, 2560), (4, 256), (3, 192), (77, 640), (333, 704), (5, 21504), (2, 40000 // 64 * 64),
               (1000, 64), (513, 2560)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", COPY_SHAPES)
def test_checkpoint_codes_scales_and_restored_values(dev, M, K, dtype):
    x = tensor(dev, M, K, dtype, M + K)
    q, scale = bl.bitnet_act_checkpoint(x)
    q_ref, s_ref = codes64(x)
    assert torch.equal(scale.cpu(), s_ref)
    assert torch.equal(q.cpu(), q_ref)
    for out in (torch.float32, torch.bfloat16):
        back = bl.bitnet_act_restore(q, scale, out)
        want = (q_ref.float().view(M, -1, GROUP) * s_ref.unsqueeze(2)).view(M, K).to(out)
        assert torch.equal(back.cpu(), want)
    # within half a code of x, up to the roundings of 127 / amax, of the product and of the scale
    err = (values64(q, scale) - x.double()).abs().view(M, -1, GROUP)
    assert bool((err <= scale.double().unsqueeze(2) * (0.5 + 127 * 4 * U)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_checkpoint_of_one_group_per_row_is_the_per_token_quantisation(dev, dtype):
    x = tensor(dev, 600, 64, dtype, 3)
    q, scale = bl.bitnet_act_checkpoint(x)
    xq, a, _ = bl.bitnet_quant_act(x)
    assert torch.equal(q, xq) and torch.equal(scale.view(-1), a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_checkpoint_edge_groups(dev, dtype):
    x = tensor(dev, 8, 256, dtype, 11)
    x[0] = 0.0
    x[1, :64] = 0.0
    x[1, 64] = -0.0
    x[2, 70] = float("inf")
    x[3, 130] = float("nan")
    x[4, 255] = -float("inf")
    x[5] = 2.0 ** -121                    # below the smallest stored magnitude
    x[6] = 2.0 ** -120                    # the smallest
    x[7, :64] = torch.finfo(DTYPES[dtype]).max
    x[7, 1] = -torch.finfo(DTYPES[dtype]).max
    q, scale = bl.bitnet_act_checkpoint(x)
    q_ref, s_ref = codes64(x)
    assert torch.equal(q.cpu(), q_ref)
    assert torch.equal(torch.nan_to_num(scale.cpu(), nan=-1.0), torch.nan_to_num(s_ref, nan=-1.0))
    back = bl.bitnet_act_restore(q, scale, torch.float32).cpu()
    for m, k in ((2, 64), (3, 128), (4, 192)):
        assert torch.isnan(back[m, k:k + 64]).all()
        keep = torch.ones(256, dtype=torch.bool)
        keep[k:k + 64] = False
        assert torch.isfinite(back[m, keep]).all()
    assert (back[0] == 0).all() and (back[5] == 0).all() and (back[6] == 2.0 ** -120).all()
    assert torch.isfinite(back[7]).all() and back[7, 0] == -back[7, 1] and back[7, 0] > 0


# ---------------------------------------------------------------- layer norm


def ln_stats64(x):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, var


def check_layernorm(x, gain, bias, y, mean, rstd, eps=EPS):
    K = x.shape[1]
    m64, v64 = ln_stats64(x)
    r64 = (v64 + eps).rsqrt()
    d_mean = DEPTH * U * x.double().abs().mean(1) + U * m64.abs()
    d_var = DEPTH * U * v64 + d_mean.square()
    rel_r = 0.5 * d_var / (v64 + eps) + 4 * U
    close(mean, m64, d_mean + 1e-38, "mean")
    # second order in rel_r: a row whose variance vanishes in its own rounding has rel_r up to 1
    close(rstd, r64, r64 * rel_r * 2 + 1e-38, "rstd")
    n = (x.double() - m64[:, None]) * r64[:, None]
    dn = 4 * U * n.abs() + (d_mean * r64)[:, None] + n.abs() * 2 * rel_r[:, None]
    g = gain.double() if gain is not None else torch.ones(K, dtype=torch.float64, device=x.device)
    b = bias.double() if bias is not None else torch.zeros(K, dtype=torch.float64, device=x.device)
    want = n * g + b
    tol = dn * g.abs() + 2 * U * ((n * g).abs() + b.abs()) + half_step(x.dtype) * (want.abs() + dn * g.abs()) * 1.001
    close(y, want, tol + 1e-38, "y")


LN_SHAPES = [(1, 64), (4, 256), (3, 320), (2, 640), (77, 640), (5, 2560), (300, 2560), (1100, 1088), (9, 5376),
             (650, 5376), (7, 6912), (2, 21504), (310, 21504), (1, 32768), (160, 32768), (5000, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", LN_SHAPES)
def test_layernorm(dev, M, K, dtype):
    x = tensor(dev, M, K, dtype, M + K, shift=0.5)
    gain, bias = vector(dev, K, dtype, 1), vector(dev, K, dtype, 2, -0.3, 0.3)
    y, mean, rstd = bl.bitnet_layernorm(x, gain, bias, EPS)
    check_layernorm(x, gain, bias, y, mean, rstd)
    y2, mean2, rstd2, x8, x_scale = bl.bitnet_layernorm(x, gain, bias, EPS, checkpoint=True)
    q, scale = bl.bitnet_act_checkpoint(x)
    assert torch.equal(x8, q) and torch.equal(x_scale, scale)
    check_layernorm(x, gain, bias, y2, mean2, rstd2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(6, 256), (40, 2560), (600, 5376)])
def test_layernorm_without_gain_or_bias(dev, M, K, dtype):
    x = tensor(dev, M, K, dtype, 5, scale=3.0)
    gain, bias = vector(dev, K, dtype, 1), vector(dev, K, dtype, 2, -0.3, 0.3)
    for g, b in ((None, None), (gain, None), (None, bias)):
        check_layernorm(x, g, b, *bl.bitnet_layernorm(x, g, b, EPS))


def test_layernorm_rows_far_from_zero_and_constant_rows(dev):
    # a mean 1000 times the spread: the variance comes from the centred values
    x = tensor(dev, 33, 2560, "f32", 8, scale=1.0, shift=1000.0, loud=False)
    check_layernorm(x, None, None, *bl.bitnet_layernorm(x))
    # an outlier in the first place
    x = tensor(dev, 33, 2560, "f32", 9, loud=False)
    x[:, 0] = 1.0e6
    check_layernorm(x, None, None, *bl.bitnet_layernorm(x))
    # equal values: no variance, y is the bias (K = 256 sums of 2.0 are exact)
    x = torch.full((3, 256), 2.0, device=dev)
    bias = vector(dev, 256, "f32", 3)
    y, mean, rstd = bl.bitnet_layernorm(x, None, bias, EPS)
    assert torch.equal(mean, torch.full((3,), 2.0, device=dev))
    assert torch.equal(y, bias.expand(3, 256))
    close(rstd, torch.full((3,), EPS, device=dev).double().rsqrt(), 4 * U * EPS ** -0.5, "rstd")


def test_layernorm_nonfinite_rows_stay_in_their_rows(dev):
    x = tensor(dev, 40, 640, "bf16", 4)
    x[3, 100] = float("nan")
    x[17, 0] = float("inf")
    y, mean, rstd = bl.bitnet_layernorm(x)
    clean = [m for m in range(40) if m not in (3, 17)]
    assert torch.isfinite(y[clean]).all() and torch.isfinite(rstd[clean]).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[17]).all()
    check_layernorm(x[clean], None, None, y[clean], mean[clean], rstd[clean])


# ------------------------------------------------------------ norm gradients


def column_depth(M):
    return min(M, 600) + 24


def check_norm_backward(dy, x64, centre, r, gain, dx, dgain, dbias, rel_r):
    """x64: the values that the kernel read; centre, r: of each row, r known up to rel_r."""
    K = dy.shape[1]
    d = dy.double()
    g = gain.double() if gain is not None else torch.ones(K, dtype=torch.float64, device=dy.device)
    c, r = centre[:, None], r[:, None]
    rel = rel_r[:, None]
    n = (x64 - c) * r
    # x itself may be a product (code * scale), x - mean one rounding, times r another
    dn = U * (4 * n.abs() + 2 * (x64.abs() + c.abs()) * r) + rel * n.abs()
    t = d * g
    layer = dbias is not False
    m1 = t.mean(1, keepdim=True) if layer else torch.zeros_like(r)
    d_m1 = DEPTH * U * t.abs().mean(1, keepdim=True) if layer else torch.zeros_like(r)
    m2 = (t * n).mean(1, keepdim=True)
    d_m2 = DEPTH * U * (t * n).abs().mean(1, keepdim=True) + (t.abs() * dn).mean(1, keepdim=True)
    want = r * (t - m1 - n * m2)
    parts = t.abs() + m1.abs() + (n * m2).abs()
    tol = r * (8 * U * parts + d_m1 + n.abs() * d_m2 + dn * m2.abs() + rel * parts)
    tol = tol * 1.01 + half_step(dy.dtype) * (want.abs() + tol) * 1.001 + 1e-38
    close(dx, want, tol, "dx")
    if dgain is not None:
        close(dgain, (d * n).sum(0), (column_depth(dy.shape[0]) * U * (d * n).abs() + d.abs() * dn).sum(0) * 1.01 + 1e-38,
              "dgain")
    if dbias is not None and layer:
        close(dbias, d.sum(0), (column_depth(dy.shape[0]) * U * d.abs()).sum(0) + 1e-38, "dbias")


def rms64(x64, eps=EPS):
    r = (x64.square().mean(1) + eps).rsqrt()
    return r, torch.full_like(r, 0.5 * DEPTH * U + 4 * U)


BWD_SHAPES = [(1, 64), (1, 2560), (4, 256), (3, 320), (2, 640), (333, 640), (16, 5376), (65, 2560), (1200, 2560),
              (4500, 192), (640, 6912), (7, 6912), (2, 21504), (310, 21504), (3, 32768), (170, 32768), (200, 8256),
              (150, 16448)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", BWD_SHAPES)
def test_layernorm_backward(dev, M, K, dtype):
    x = tensor(dev, M, K, dtype, M + K, shift=0.5)
    dy = tensor(dev, M, K, dtype, M + K + 1, scale=0.01, loud=False)
    gain = vector(dev, K, dtype, 1)
    _, mean, rstd, x8, x_scale = bl.bitnet_layernorm(x, gain, None, EPS, checkpoint=True)
    none = torch.zeros(M, dtype=torch.float64, device=dev)
    dx, dgain, dbias = bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain)
    check_norm_backward(dy, x.double(), mean.double(), rstd.double(), gain, dx, dgain, dbias, none)
    dx, dgain, dbias = bl.bitnet_layernorm_backward(dy, mean, rstd, x8=x8, x_scale=x_scale, gain=gain)
    check_norm_backward(dy, values64(x8, x_scale), mean.double(), rstd.double(), gain, dx, dgain, dbias, none)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", BWD_SHAPES)
def test_rmsnorm_backward(dev, M, K, dtype):
    x = tensor(dev, M, K, dtype, M + K)
    dy = tensor(dev, M, K, dtype, M + K + 1, scale=0.01, loud=False)
    gain = vector(dev, K, dtype, 1)
    zero = torch.zeros(M, dtype=torch.float64, device=dev)
    r, rel = rms64(x.double())
    dx, dgain = bl.bitnet_rmsnorm_backward(dy, x=x, gain=gain, rms_eps=EPS)
    check_norm_backward(dy, x.double(), zero, r, gain, dx, dgain, False, rel)
    x8, x_scale = bl.bitnet_act_checkpoint(x)
    r, rel = rms64(values64(x8, x_scale))
    dx, dgain = bl.bitnet_rmsnorm_backward(dy, x8=x8, x_scale=x_scale, gain=gain, rms_eps=EPS)
    check_norm_backward(dy, values64(x8, x_scale), zero, r, gain, dx, dgain, False, rel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 37])
def test_norms_at_every_width(dev, M, dtype):
    """Every K the norms take, with the column sums of one CTA and with those of several."""
    zero = torch.zeros(M, dtype=torch.float64, device=dev)
    big_x, big_dy = tensor(dev, M, 32768, dtype, 5, shift=0.3), tensor(dev, M, 32768, dtype, 6, scale=0.01, loud=False)
    big_g, big_b = vector(dev, 32768, dtype, 1), vector(dev, 32768, dtype, 2, -0.3, 0.3)
    for K in range(64, 32768 + 64, 64):
        x, dy, gain, bias = big_x[:, :K].contiguous(), big_dy[:, :K].contiguous(), big_g[:K], big_b[:K]
        y, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, bias, EPS, checkpoint=True)
        check_layernorm(x, gain, bias, y, mean, rstd)
        check_layernorm(x, gain, bias, *bl.bitnet_layernorm(x, gain, bias, EPS))
        for a, b in zip((x8, xs), bl.bitnet_act_checkpoint(x)):
            assert torch.equal(a, b), K
        for form in ({"x": x}, {"x8": x8, "x_scale": xs}):
            read = x.double() if "x" in form else values64(x8, xs)
            got = bl.bitnet_layernorm_backward(dy, mean, rstd, gain=gain, **form)
            check_norm_backward(dy, read, mean.double(), rstd.double(), gain, *got, zero)
            r, rel = rms64(read)
            check_norm_backward(dy, read, zero, r, gain, *bl.bitnet_rmsnorm_backward(dy, gain=gain, **form), False, rel)
    assert bl.bitnet_get_device_status() == bl.BITNET_OK


@pytest.mark.parametrize("M,K", [(5, 256), (300, 2560), (30, 21504)])
def test_norm_backward_outputs_that_are_not_wanted(dev, M, K):
    x = tensor(dev, M, K, "bf16", 3)
    dy = tensor(dev, M, K, "bf16", 4, loud=False)
    gain = vector(dev, K, "bf16", 1)
    _, mean, rstd = bl.bitnet_layernorm(x, gain)
    full = bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain)
    for want_g in (True, False):
        for want_b in (True, False):
            got = bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain, want_dgain=want_g, want_dbias=want_b)
            assert torch.equal(got[0], full[0])
            assert (got[1] is not None) == want_g and (got[2] is not None) == want_b
            assert not want_g or torch.equal(got[1], full[1])
            assert not want_b or torch.equal(got[2], full[2])
    r_full = bl.bitnet_rmsnorm_backward(dy, x=x, gain=gain)
    dx, dgain = bl.bitnet_rmsnorm_backward(dy, x=x, gain=gain, want_dgain=False)
    assert dgain is None and torch.equal(dx, r_full[0])
    # no gain is a gain of ones
    ones = torch.ones(K, dtype=torch.bfloat16, device=dev)
    for a, b in zip(bl.bitnet_layernorm_backward(dy, mean, rstd, x=x),
                    bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=ones)):
        assert torch.equal(a, b)
    for a, b in zip(bl.bitnet_rmsnorm_backward(dy, x=x), bl.bitnet_rmsnorm_backward(dy, x=x, gain=ones)):
        assert torch.equal(a, b)


def test_rmsnorm_backward_of_zero_rows(dev):
    x = torch.zeros(5, 256, device=dev)
    x[1] = 1.0
    dy = tensor(dev, 5, 256, "f32", 2, loud=False)
    r, rel = rms64(x.double())
    dx, dgain = bl.bitnet_rmsnorm_backward(dy, x=x)
    check_norm_backward(dy, x.double(), torch.zeros(5, dtype=torch.float64, device=dev), r, None, dx, dgain, False, rel)
    x8, x_scale = bl.bitnet_act_checkpoint(x)
    assert torch.equal(bl.bitnet_rmsnorm_backward(dy, x8=x8, x_scale=x_scale)[0], dx)


def test_norm_gradients_against_differences(dev):
    """The kernels' gradients along random directions against central
    differences of the norms in 64 bits.  With step h the difference is off by
    the third derivative's h^2 / 6 and by 2^-52 |loss| / h: below 1e-8 of the
    terms at h = 1e-4.  The kernels' own part is an fp32 dot product's:
    (DEPTH + 16) u times the magnitudes' sum, for each of the three factors of
    a term."""
    M, K, h = 6, 320, 1e-4
    x = tensor(dev, M, K, "f32", 21, shift=0.3, loud=False)
    dy = tensor(dev, M, K, "f32", 22, loud=False)
    gain, bias = vector(dev, K, "f32", 1), vector(dev, K, "f32", 2)
    _, mean, rstd = bl.bitnet_layernorm(x, gain, bias, EPS)
    ln = dict(zip(("x", "gain", "bias"), bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain)))
    rms = dict(zip(("x", "gain"), bl.bitnet_rmsnorm_backward(dy, x=x, gain=gain, rms_eps=EPS)))

    def loss(kind, x, gain, bias):
        c = x - x.mean(1, keepdim=True) if kind == "ln" else x
        y = c * (c.square().mean(1, keepdim=True) + EPS).rsqrt() * gain
        return float(((y + bias) * dy.double()).sum())

    for kind, grads in (("ln", ln), ("rms", rms)):
        for name, grad in grads.items():
            for seed in range(3):
                at = {"x": x.double(), "gain": gain.double(), "bias": bias.double()}
                v = torch.randn(at[name].shape, dtype=torch.float64,
                                generator=torch.Generator().manual_seed(seed)).to(dev)
                up, down = dict(at), dict(at)
                up[name], down[name] = at[name] + h * v, at[name] - h * v
                want = (loss(kind, **up) - loss(kind, **down)) / (2 * h)
                got = float((grad.double() * v).sum())
                size = float((grad.double() * v).abs().sum()) + float(dy.double().abs().sum()) * 0.1
                assert abs(got - want) <= size * (3 * (DEPTH + 16) * U + 1e-6), (kind, name, got, want)


# ---------------------------------------------------------------------- gate


def gate_ref(u, g):
    u, g = u.float().cpu(), g.float().cpu()
    r = torch.where(g > 0, g, torch.zeros_like(g))
    return (r * r) * u


def gate_backward_ref(dh, u, g):
    d = dh.float().cpu()
    r = torch.where(g > 0, g, torch.zeros_like(g))
    return d * (r * r), (d * u) * (2.0 * r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,F", [(1, 64), (4, 256), (77, 6912), (333, 704), (2, 21504), (1030, 640)])
def test_gate_and_its_gradient(dev, M, F, dtype):
    dt = DTYPES[dtype]
    u, g = tensor(dev, M, F, dtype, 1), tensor(dev, M, F, dtype, 2)
    g[0, :3] = torch.tensor([0.0, -0.0, -1.0], dtype=dt, device=dev)
    dh = tensor(dev, M, F, dtype, 3, scale=0.01, loud=False)
    h = bl.bitnet_relu2_gate(u, g)
    assert torch.equal(h.cpu(), gate_ref(u, g).to(dt))
    h2, u8, us, g8, gs = bl.bitnet_relu2_gate(u, g, checkpoint=True)
    assert torch.equal(h2, h)
    for t, q, s in ((u, u8, us), (g, g8, gs)):
        q_ref, s_ref = bl.bitnet_act_checkpoint(t)
        assert torch.equal(q, q_ref) and torch.equal(s, s_ref)
    du, dg = bl.bitnet_relu2_gate_backward(dh, u=u, g=g)
    du_ref, dg_ref = gate_backward_ref(dh, u.float().cpu(), g.float().cpu())
    assert torch.equal(du.cpu(), du_ref.to(dt)) and torch.equal(dg.cpu(), dg_ref.to(dt))
    du, dg = bl.bitnet_relu2_gate_backward(dh, u8=u8, u_scale=us, g8=g8, g_scale=gs)
    du_ref, dg_ref = gate_backward_ref(dh, bl.bitnet_act_restore(u8, us, torch.float32).cpu(),
                                       bl.bitnet_act_restore(g8, gs, torch.float32).cpu())
    assert torch.equal(du.cpu(), du_ref.to(dt)) and torch.equal(dg.cpu(), dg_ref.to(dt))


def test_gate_matches_the_gated_product(dev):
    """The same h as the product that has the gate in its epilogue, from its fp32 u and g."""
    M, F, K = 33, 128, 256
    x = tensor(dev, M, K, "bf16", 5)
    Wu, Wg = (torch.from_numpy(synth.weights(F, K, 0.02, s, 1)).to(dev) for s in (1, 2))
    (Pu, gu), (Pg, gg) = bl.bitnet_pack_weights(Wu), bl.bitnet_pack_weights(Wg)
    xq, a, rs = bl.bitnet_quant_act(x, want_rowsum=True)
    u = bl.bitnet_linear_gemm(Pu, gu, xq, a, rs, out_dtype=torch.float32)
    g = bl.bitnet_linear_gemm(Pg, gg, xq, a, rs, out_dtype=torch.float32)
    h = bl.bitnet_linear_upgate_gemm(Pu, gu, Pg, gg, xq, a, rs)
    assert torch.equal(bl.bitnet_relu2_gate(u, g).to(torch.bfloat16), h)


def test_gate_gradient_against_differences(dev):
    """du and dg along random directions against central differences in 64
    bits.  h is cubic: with step 1e-4 the difference is off by v^3 h^2 =
    1e-8 v^3 (and by sign changes of g within a step, of second order too), the
    kernel by 3u of each term."""
    M, F, h = 5, 192, 1e-4
    u, g, dh = (tensor(dev, M, F, "f32", s, loud=False) for s in (1, 2, 3))
    du, dg = (t.double() for t in bl.bitnet_relu2_gate_backward(dh, u=u, g=g))
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        vu, vg = (torch.randn(M, F, dtype=torch.float64, generator=gen).to(dev) for _ in range(2))

        def loss(sign):
            return float((((g.double() + sign * h * vg).relu().square()) * (u.double() + sign * h * vu)
                          * dh.double()).sum())

        want = (loss(1) - loss(-1)) / (2 * h)
        got = float((du * vu + dg * vg).sum())
        size = float((du * vu).abs().sum() + (dg * vg).abs().sum())
        assert abs(got - want) <= size * (4 * U + 1e-6)


def test_gate_nonfinite_values(dev):
    u, g, dh = (tensor(dev, 4, 128, "f32", s) for s in (1, 2, 3))
    g[0, 0] = float("nan")      # not above zero: the gate is closed
    g[1, 5] = float("inf")
    u[2, 64] = float("nan")
    g[2, 64] = 1.0
    h, u8, us, g8, gs = bl.bitnet_relu2_gate(u, g, checkpoint=True)
    assert torch.equal(torch.nan_to_num(h.cpu(), nan=7.0), torch.nan_to_num(gate_ref(u, g), nan=7.0))
    assert torch.isnan(gs[0, 0]) and torch.isnan(gs[1, 0]) and torch.isnan(us[2, 1])
    assert int(torch.isnan(gs).sum()) == 2 and int(torch.isnan(us).sum()) == 1


# ------------------------------------------------------- all of them together


@pytest.mark.parametrize("M,D,F", [(5, 256, 640), (130, 640, 1728), (300, 2560, 6912)])
def test_ffn_training_step(dev, M, D, F):
    """Forward and backward of an FFN block, y = x + down(subnorm(gate(up(n), gate(n)))),
    n = layernorm(x), with every activation that the backward pass reads held in
    8 bits.  Each stage is checked on the inputs that the GPU's stage before it
    made, so each keeps its own tolerance."""
    x = tensor(dev, M, D, "bf16", 1, shift=0.2)
    gain_in, bias_in, gain_sub = vector(dev, D, "bf16", 1), vector(dev, D, "bf16", 2, -0.1, 0.1), vector(dev, F, "bf16", 3)
    (Pu, gu), (Pg, gg), (Pd, gd) = (bl.bitnet_pack_weights(torch.from_numpy(synth.weights(n, k, 0.02, s, 1)).to(dev))
                                    for n, k, s in ((F, D, 1), (F, D, 2), (D, F, 3)))
    # forward
    n, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain_in, bias_in, EPS, checkpoint=True)
    nq, na, nrs = bl.bitnet_quant_act(n, want_rowsum=True)
    u = bl.bitnet_linear_gemm(Pu, gu, nq, na, nrs)
    g = bl.bitnet_linear_gemm(Pg, gg, nq, na, nrs)
    h, u8, us, g8, gs = bl.bitnet_relu2_gate(u, g, checkpoint=True)
    h8, hs = bl.bitnet_act_checkpoint(h)
    hq, ha, hrs = bl.bitnet_quant_act(h, gain_sub, EPS, want_rowsum=True)
    bl.bitnet_linear_gemm(Pd, gd, hq, ha, hrs)
    # backward
    dY = tensor(dev, M, D, "bf16", 9, scale=0.01, loud=False)
    dWd = bl.bitnet_ste_backward_weight(dY, hq, ha)
    dhn = bl.bitnet_ste_backward_input(Pd, gd, dY, out_dtype=torch.bfloat16)
    dh, dgain_sub = bl.bitnet_rmsnorm_backward(dhn, x8=h8, x_scale=hs, gain=gain_sub, rms_eps=EPS)
    du, dg = bl.bitnet_relu2_gate_backward(dh, u8=u8, u_scale=us, g8=g8, g_scale=gs)
    dWu, dWg = bl.bitnet_ste_backward_weight(du, nq, na), bl.bitnet_ste_backward_weight(dg, nq, na)
    dn = (bl.bitnet_ste_backward_input(Pu, gu, du) + bl.bitnet_ste_backward_input(Pg, gg, dg)).to(torch.bfloat16)
    dx, dgain_in, dbias_in = bl.bitnet_layernorm_backward(dn, mean, rstd, x8=x8, x_scale=xs, gain=gain_in)
    torch.cuda.synchronize()
    assert bl.bitnet_get_device_status() == bl.BITNET_OK

    check_layernorm(x, gain_in, bias_in, n, mean, rstd)
    for t, q, s in ((x, x8, xs), (u, u8, us), (g, g8, gs), (h, h8, hs)):
        q_ref, s_ref = codes64(t)
        assert torch.equal(q.cpu(), q_ref) and torch.equal(s.cpu(), s_ref)
    assert torch.equal(h.cpu(), gate_ref(u, g).to(torch.bfloat16))
    r, rel = rms64(values64(h8, hs))
    zero = torch.zeros(M, dtype=torch.float64, device=dev)
    check_norm_backward(dhn, values64(h8, hs), zero, r, gain_sub, dh, dgain_sub, False, rel)
    f32 = [bl.bitnet_act_restore(q, s, torch.float32).cpu() for q, s in ((u8, us), (g8, gs))]
    du_ref, dg_ref = gate_backward_ref(dh, *f32)
    assert torch.equal(du.cpu(), du_ref.to(torch.bfloat16)) and torch.equal(dg.cpu(), dg_ref.to(torch.bfloat16))
    check_norm_backward(dn, values64(x8, xs), mean.double(), rstd.double(), gain_in, dx, dgain_in, dbias_in, zero)
    for t in (dWd, dWu, dWg):
        assert torch.isfinite(t).all() and bool(t.any())


# -------------------------------------------------------- how they are called


def all_calls(x, dy, gain, bias):
    """Every operator once; a flat list of outputs."""
    y, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, bias, EPS, checkpoint=True)
    out = [y, mean, rstd, x8, xs]
    out += bl.bitnet_layernorm_backward(dy, mean, rstd, x8=x8, x_scale=xs, gain=gain)
    out += bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain)
    out += bl.bitnet_rmsnorm_backward(dy, x=x, gain=gain)
    out += bl.bitnet_rmsnorm_backward(dy, x8=x8, x_scale=xs, gain=gain)
    q, s = bl.bitnet_act_checkpoint(y)
    out += [q, s, bl.bitnet_act_restore(q, s, x.dtype)]
    h, u8, us, g8, gs = bl.bitnet_relu2_gate(x, y, checkpoint=True)
    out += [h, u8, us, g8, gs]
    out += bl.bitnet_relu2_gate_backward(dy, u8=u8, u_scale=us, g8=g8, g_scale=gs)
    out += bl.bitnet_relu2_gate_backward(dy, u=x, g=y)
    return out


def call_inputs(dev, M, K, dtype, seed):
    return (tensor(dev, M, K, dtype, seed), tensor(dev, M, K, dtype, seed + 1, scale=0.01),
            vector(dev, K, dtype, 1), vector(dev, K, dtype, 2))


@pytest.mark.parametrize("M,K,dtype", [(3, 256, "f32"), (700, 2560, "bf16"), (300, 21504, "bf16")])
def test_same_bits_again_on_another_stream_and_from_a_graph(dev, M, K, dtype):
    args = call_inputs(dev, M, K, dtype, 31)
    first = [t.clone() for t in all_calls(*args)]
    for a, b in zip(first, all_calls(*args)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        other = all_calls(*args)
    torch.cuda.current_stream(dev).wait_stream(side)
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_calls(*args)
    for t in captured:
        t.view(torch.uint8).fill_(0x55)
    graph.replay()
    for a, b in zip(first, captured):
        assert torch.equal(a, b)
    # new inputs in the same places
    fresh = call_inputs(dev, M, K, dtype, 77)
    for a, b in zip(args, fresh):
        a.copy_(b)
    graph.replay()
    for a, b in zip(all_calls(*fresh), captured):
        assert torch.equal(a, b)


def test_two_host_threads(dev):
    args = [call_inputs(dev, 200, 2560, "bf16", s) for s in (1, 2)]
    want = [[t.clone() for t in all_calls(*a)] for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream(dev)):
            for _ in range(20):
                got = all_calls(*args[i])
                torch.cuda.current_stream().synchronize()
                wrong.extend(k for k, (a, b) in enumerate(zip(want[i], got)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


@pytest.mark.parametrize("M,K,dtype", [(3, 64, "f32"), (5, 320, "bf16"), (130, 2560, "bf16"), (9, 21504, "f32")])
def test_nothing_is_written_outside_the_outputs(dev, M, K, dtype):
    """Outputs inside larger buffers: the bytes around them stay as they were."""
    dt = DTYPES[dtype]
    x, dy, gain, bias = call_inputs(dev, M, K, dtype, 5)
    arenas = []

    def room(shape, t):
        n = 1
        for s in shape:
            n *= s
        size = n * torch.empty(0, dtype=t).element_size()
        arena = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=dev)
        arenas.append((arena, size))
        return arena[256:256 + size].view(t).view(shape)

    G = (M, K // GROUP)
    f32, i8 = torch.float32, torch.int8
    _, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, bias, EPS, True, room((M, K), dt), room((M,), f32),
                                                room((M,), f32), room((M, K), i8), room(G, f32))
    ws = room((bl.bitnet_norm_backward_workspace_bytes(M, K),), torch.uint8)
    bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain, dx=room((M, K), dt), dgain=room((K,), f32),
                                 dbias=room((K,), f32), workspace=ws)
    bl.bitnet_rmsnorm_backward(dy, x8=x8, x_scale=xs, gain=gain, dx=room((M, K), dt), dgain=room((K,), f32),
                               workspace=ws)
    bl.bitnet_act_checkpoint(x, room((M, K), i8), room(G, f32))
    bl.bitnet_act_restore(x8, xs, dt, room((M, K), dt))
    bl.bitnet_relu2_gate(x, dy, True, room((M, K), dt), room((M, K), i8), room(G, f32), room((M, K), i8), room(G, f32))
    bl.bitnet_relu2_gate_backward(dy, x, x, du=room((M, K), dt), dg=room((M, K), dt))
    torch.cuda.synchronize()
    for arena, size in arenas:
        assert bool((arena[:256] == 0xA5).all()) and bool((arena[256 + size:] == 0xA5).all())


def test_more_values_than_32_bits_count(dev):
    """2^31 + 64 * 704 values in rows of 704: the last rows against the same rows alone."""
    K = 704
    M = (1 << 31) // K + 64
    if torch.cuda.get_device_properties(dev).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x.random_(-100, 100)
    tail = x[-5:].contiguous()
    y, mean, rstd, x8, xs = bl.bitnet_layernorm(x, checkpoint=True)
    ty, tmean, trstd, tx8, txs = bl.bitnet_layernorm(tail, checkpoint=True)
    for a, b in ((y, ty), (mean, tmean), (rstd, trstd), (x8, tx8), (xs, txs)):
        assert torch.equal(a[-5:], b)
    dx, _, _ = bl.bitnet_layernorm_backward(y, mean, rstd, x8=x8, x_scale=xs)
    assert torch.equal(dx[-5:], bl.bitnet_layernorm_backward(ty, tmean, trstd, x8=tx8, x_scale=txs)[0])
    du, dg = bl.bitnet_relu2_gate_backward(y, u=x, g=dx)
    for a, b in zip((du, dg), bl.bitnet_relu2_gate_backward(ty, u=tail, g=dx[-5:].contiguous())):
        assert torch.equal(a[-5:], b)
    bl.bitnet_act_restore(x8, xs, x=du)
    assert torch.equal(du[-5:], bl.bitnet_act_restore(tx8, txs))


def test_binding_refuses(dev):
    x = tensor(dev, 4, 256, "bf16", 1)
    dy = tensor(dev, 4, 256, "bf16", 2)
    gain = vector(dev, 256, "bf16", 1)
    _, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, checkpoint=True)
    bad = [
        lambda: bl.bitnet_act_checkpoint(x.half()),
        lambda: bl.bitnet_act_checkpoint(x.int()),
        lambda: bl.bitnet_act_checkpoint(x.view(-1)),
        lambda: bl.bitnet_act_checkpoint(x.t()),
        lambda: bl.bitnet_act_checkpoint(x[:, :128]),
        lambda: bl.bitnet_act_checkpoint(x, x8=x8[:3]),
        lambda: bl.bitnet_act_checkpoint(x, x_scale=xs.double()),
        lambda: bl.bitnet_act_restore(x8, xs[:, :3]),
        lambda: bl.bitnet_act_restore(x8.view(torch.uint8), xs),
        lambda: bl.bitnet_act_restore(x8, xs, torch.float16),
        lambda: bl.bitnet_act_restore(x8, None),
        lambda: bl.bitnet_layernorm(x, gain.float()),
        lambda: bl.bitnet_layernorm(x, gain[:64]),
        lambda: bl.bitnet_layernorm(x, None, gain.cpu()),
        lambda: bl.bitnet_layernorm(x, x8=x8),
        lambda: bl.bitnet_layernorm_backward(dy, mean, rstd),
        lambda: bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, x8=x8, x_scale=xs),
        lambda: bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, x_scale=xs),
        lambda: bl.bitnet_layernorm_backward(dy, mean, rstd, x8=x8),
        lambda: bl.bitnet_layernorm_backward(dy, mean, None, x=x),
        lambda: bl.bitnet_layernorm_backward(dy, mean[:2], rstd, x=x),
        lambda: bl.bitnet_layernorm_backward(dy.float(), mean, rstd, x=x),
        lambda: bl.bitnet_layernorm_backward(dy[:2], mean, rstd, x=x),
        lambda: bl.bitnet_rmsnorm_backward(dy, x=x, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: bl.bitnet_rmsnorm_backward(dy, x=x, dgain=gain),
        lambda: bl.bitnet_relu2_gate(x, dy[:2]),
        lambda: bl.bitnet_relu2_gate(x, dy.float()),
        lambda: bl.bitnet_relu2_gate(x, dy, g8=x8),
        lambda: bl.bitnet_relu2_gate_backward(dy),
        lambda: bl.bitnet_relu2_gate_backward(dy, u=x),
        lambda: bl.bitnet_relu2_gate_backward(dy, u=x, g=x, u8=x8, u_scale=xs),
        lambda: bl.bitnet_relu2_gate_backward(dy, u8=x8, u_scale=xs, g8=x8),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    refused = [
        lambda: bl.bitnet_act_checkpoint(x[:0]),
        lambda: bl.bitnet_act_checkpoint(torch.zeros(4, 96, device=dev)),
        lambda: bl.bitnet_layernorm(torch.zeros(2, 32768 + 64, device=dev)),
        lambda: bl.bitnet_layernorm(x, eps=0.0),
        lambda: bl.bitnet_layernorm(x, eps=float("nan")),
        lambda: bl.bitnet_rmsnorm_backward(dy, x=x, rms_eps=-1.0),
        lambda: bl.bitnet_layernorm_backward(dy, mean, rstd, x=x,
                                             workspace=torch.empty(64, dtype=torch.uint8, device=dev)),
        lambda: bl.bitnet_relu2_gate(torch.zeros(1, 100, device=dev), torch.zeros(1, 100, device=dev)),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(bl.BitnetError):
            call()
            pytest.fail(f"call {i} was accepted")
