"""GPU tests of the norms' accuracy: rows far from zero, outliers, infinities,
and the rounding of 1 / sqrt, against 64-bit forms.

Tolerances count fp32's half steps u = 2^-24.  The additions between a value and
its row's result number at most DEPTH: 16 in a thread (two halves of at most 16
columns), 6 in the tree of a warp, 2 + 5 between warps, with a term's own few
roundings."""
import pytest

import bitlinear_absmean_ternary_b200 as bl
from test_gpu_train_ops import EPS, U, close, dev, half_step, tensor, values64, vector  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DEPTH = 40


def check_layernorm_f32(x, gain, bias, y, mean, rstd, eps=EPS, first=0.0):
    """Of fp32 rows.  A warp's pivot is off its mean by at most e = DEPTH u max |x|, and differences from it are
    rounded relative to themselves, so that the variance is off by a few DEPTH u (var + e^2), whatever the mean.
    The warps' are joined about the first warp's mean, which is at most `first` off the others' beside the spread."""
    x = x.double()
    m = x.mean(1)
    v = (x - m[:, None]).square().mean(1)
    r = (v + eps).rsqrt()
    spread = (v + (DEPTH * U * x.abs().amax(1)).square()).sqrt()
    d_mean = U * m.abs() + 8 * U * first + DEPTH * U * spread
    d_var = 2 * DEPTH * U * (spread.square() + first * spread)
    rel = 0.5 * d_var / (v + eps) + 3 * U
    close(mean, m, d_mean + 1e-38, "mean")
    close(rstd, r, r * rel * 1.001, "rstd")
    n = (x - m[:, None]) * r[:, None]
    dn = 3 * U * n.abs() + (d_mean * r)[:, None] + n.abs() * rel[:, None]
    g, b = gain.double(), bias.double()
    close(y, n * g + b, dn * 1.001 * g.abs() + 2 * U * ((n * g).abs() + b.abs()), "y")


SHAPES = [(37, 64), (37, 256), (37, 640), (9, 1600), (333, 2560), (37, 5376), (21, 21504), (5, 32768)]


@pytest.mark.parametrize("offset", [0.0, 1e3, -1e4, 1e5])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_of_rows_far_from_zero(dev, M, K, offset):
    x = tensor(dev, M, K, "f32", K, shift=offset, loud=False)
    gain, bias = vector(dev, K, "f32", 1), vector(dev, K, "f32", 2, -0.3, 0.3)
    check_layernorm_f32(x, gain, bias, *bl.bitnet_layernorm(x, gain, bias, EPS))
    check_layernorm_f32(x, gain, bias, *bl.bitnet_layernorm(x, gain, bias, EPS, checkpoint=True)[:3])


@pytest.mark.parametrize("first", [1, 8, 100])
@pytest.mark.parametrize("M,K", SHAPES[1:])
def test_layernorm_of_rows_whose_first_columns_are_loud(dev, M, K, first):
    x = tensor(dev, M, K, "f32", K, loud=False)
    x[:, :first] += 1000.0
    gain, bias = vector(dev, K, "f32", 1), vector(dev, K, "f32", 2, -0.3, 0.3)
    # a warp has 128 columns or more, or all
    check_layernorm_f32(x, gain, bias, *bl.bitnet_layernorm(x, gain, bias, EPS), first=first * 1000.0 / min(K, 128))


@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_of_bf16_rows_far_from_zero(dev, M, K):
    """A mean 50 times the spread.  A warp's pivot is the mean of eight neighbours, sums about it are as exact as the
    spread about it is small, and the warps' means are rounded to u of the mean before they are compared."""
    x = tensor(dev, M, K, "bf16", K, scale=2.0, shift=100.0, loud=False)
    gain, bias = vector(dev, K, "bf16", 1), vector(dev, K, "bf16", 2, -0.3, 0.3)
    y, mean, rstd = bl.bitnet_layernorm(x, gain, bias, EPS)
    x = x.double()
    m = x.mean(1)
    v = (x - m[:, None]).square().mean(1)
    r = (v + EPS).rsqrt()
    s = (v + (x.view(M, K // 8, 8).mean(2) - m[:, None]).square().amax(1)).sqrt()
    d_mean = 4 * U * m.abs() + DEPTH * U * s
    rel = 0.5 * (2 * DEPTH * U * s.square() + 8 * U * s * m.abs()) / (v + EPS) + 3 * U
    close(mean, m, d_mean, "mean")
    close(rstd, r, r * rel * 1.001, "rstd")
    n = (x - m[:, None]) * r[:, None]
    dn = 3 * U * n.abs() + (d_mean * r)[:, None] + n.abs() * rel[:, None]
    g, b = gain.double(), bias.double()
    want, tol = n * g + b, dn * 1.001 * g.abs() + 2 * U * ((n * g).abs() + b.abs())
    close(y, want, tol + half_step(torch.bfloat16) * (want.abs() + tol), "y")


@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_mean_of_rows_with_infinities(dev, M, K):
    """The mean of a row is its sum / K, so an Inf stays one; rstd and y of the row are NaN."""
    for dtype in ("bf16", "f32"):
        for at in sorted({0, K // 3, K - 1}):
            x = tensor(dev, M, K, dtype, K, loud=False)
            x[0, at] = float("inf")
            x[1, at] = -float("inf")
            x[2, at] = float("nan")
            x[3, 0], x[3, K - 1] = float("inf"), -float("inf")
            y, mean, rstd = bl.bitnet_layernorm(x, None, None, EPS)
            assert mean[:2].tolist() == [float("inf"), -float("inf")] and torch.isnan(mean[2:4]).all()
            assert torch.isnan(rstd[:4]).all() and torch.isnan(y[:4]).all()
            assert torch.isfinite(mean[4:]).all() and torch.isfinite(rstd[4:]).all() and torch.isfinite(y[4:]).all()


def check_backward(dy, x64, mean, rstd, gain, dx, dgain, dbias):
    """x - mean is one rounding and its product with rstd another, whatever the mean.  dx of bf16 rows takes mean rstd
    apart: n m2 to a few u |mean| rstd |m2|, far below dx's own half step."""
    M = dy.shape[0]
    d, g = dy.double(), gain.double()
    c, r = mean.double()[:, None], rstd.double()[:, None]
    n = (x64 - c) * r
    dn = 2.01 * U * n.abs()
    t = d * g
    m1, m2 = t.mean(1, keepdim=True), (t * n).mean(1, keepdim=True)
    d_m1 = DEPTH * U * t.abs().mean(1, keepdim=True)
    d_m2 = DEPTH * U * (t * n).abs().mean(1, keepdim=True) + (t.abs() * dn).mean(1, keepdim=True)
    parts = t.abs() + m1.abs() + (n * m2).abs()
    want, tol = r * (t - m1 - n * m2), r * (8 * U * parts + d_m1 + n.abs() * d_m2 + dn * m2.abs())
    if dy.dtype == torch.bfloat16:
        tol = tol + r * 4 * U * (x64.abs() + c.abs()) * r * m2.abs()
        tol = tol + half_step(dy.dtype) * (want.abs() + tol)
    close(dx, want, 1.01 * tol + 1e-38, "dx")
    close(dgain, (d * n).sum(0), 1.01 * ((M + 8) * U * (d * n).abs() + d.abs() * dn).sum(0) + 1e-38, "dgain")
    close(dbias, d.sum(0), (M + 8) * U * d.abs().sum(0) + 1e-38, "dbias")


@pytest.mark.parametrize("offset", [0.0, 1e3, -1e4, 1e5])
@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_backward_of_rows_far_from_zero(dev, M, K, offset):
    x = tensor(dev, M, K, "f32", K, shift=offset, loud=False)
    # a gradient along n, so that its share of dx counts
    dy = 0.1 * tensor(dev, M, K, "f32", K + 1, loud=False) + (x - offset)
    gain = vector(dev, K, "f32", 1)
    _, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, None, EPS, checkpoint=True)
    check_backward(dy, x.double(), mean, rstd, gain, *bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain))
    check_backward(dy, values64(x8, xs), mean, rstd, gain,
                       *bl.bitnet_layernorm_backward(dy, mean, rstd, x8=x8, x_scale=xs, gain=gain))


@pytest.mark.parametrize("M,K", SHAPES)
def test_layernorm_backward_of_nearly_constant_bf16_rows(dev, M, K):
    """Rows of 1000 with one value a step above: a mean of thousands of spreads; and rows of 1000 alone, where n is 0."""
    x = torch.full((M, K), 1000.0, dtype=torch.bfloat16, device=dev)
    x[::2, K // 2] = 1008.0
    dy = tensor(dev, M, K, "bf16", K, scale=0.1, loud=False)
    gain = vector(dev, K, "bf16", 1)
    _, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, None, EPS, checkpoint=True)
    check_backward(dy, x.double(), mean, rstd, gain, *bl.bitnet_layernorm_backward(dy, mean, rstd, x=x, gain=gain))
    check_backward(dy, values64(x8, xs), mean, rstd, gain,
                   *bl.bitnet_layernorm_backward(dy, mean, rstd, x8=x8, x_scale=xs, gain=gain))


def short_values(dev, n, seed):
    """Values of eight mantissa bits, whose squares add up without a rounding."""
    gen = torch.Generator().manual_seed(seed)
    v = torch.rand(n, generator=gen, dtype=torch.float64) * 4 + 0.01
    return v.to(torch.bfloat16).float().to(dev)


def check_r(r, square, eps):
    """r against 1 / sqrt(RN(square + eps)): half a step, and a second-order rest below a thousandth of one."""
    want = (square + torch.full_like(square, eps)).double().rsqrt()
    step = 2.0 ** (torch.floor(torch.log2(want)) - 23)
    over = (r.double() - want).abs() / step
    assert float(over.max()) <= 0.501, float(over.max())


@pytest.mark.parametrize("K", [64, 256, 2048, 8192, 32768])
def test_rmsnorm_backward_rounds_r_once(dev, K):
    """Rows of equal magnitude and a gradient that adds up to nothing along them: dx is r.  K is a power of two, so
    that the mean square has no rounding."""
    M = 2048 if K < 20000 else 512
    v = short_values(dev, M, K)
    x = v[:, None].repeat(1, K)
    dy = torch.ones(M, K, device=dev)
    dy[:, 1::2] = -1.0
    dx, _ = bl.bitnet_rmsnorm_backward(dy, x=x, rms_eps=EPS)
    check_r(dx[:, 0], v * v, EPS)
    assert torch.equal(dx, dx[:, :1] * dy)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 256, 2048, 8192, 32768])
def test_layernorm_rounds_rstd_once(dev, K, dtype):
    """Rows of v, -v, v, -v, ...: mean 0, variance v^2, both without a rounding as K is a power of two."""
    M = 2048 if K < 20000 else 512
    v = short_values(dev, M, K)
    x = v[:, None].repeat(1, K)
    x[:, 1::2] *= -1.0
    _, mean, rstd = bl.bitnet_layernorm(x.to(torch.bfloat16 if dtype == "bf16" else torch.float32), eps=EPS)
    assert not mean.any()
    check_r(rstd, v * v, EPS)


def test_norms_of_tiny_and_huge_variance(dev):
    """eps alone, of any size, and variances that fp32 does not hold: rstd is 1 / sqrt(eps), or 0."""
    for eps in (1e-38, 1e-30, 1e-12, 1.0, 1e30):
        x = torch.zeros(3, 128, device=dev)
        x[1] = 1e25
        x[1, ::2] = -1e25
        y, _, rstd = bl.bitnet_layernorm(x, eps=eps)
        want = torch.tensor(eps, dtype=torch.float32).double() ** -0.5
        assert abs(float(rstd[0]) - float(want)) <= float(want) * 1.01 * U
        assert float(rstd[1]) == 0.0 and not y.any()
        dx, _ = bl.bitnet_rmsnorm_backward(torch.ones_like(x), x=x, rms_eps=eps)
        assert abs(float(dx[0, 0]) - float(want)) <= float(want) * 1.01 * U
        assert not dx[1].any()
