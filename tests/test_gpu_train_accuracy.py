"""GPU tests of the norms' accuracy: rows far from zero, outliers and
infinities, against 64-bit forms.

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
