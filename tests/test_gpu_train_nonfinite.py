"""GPU tests of Inf and NaN in the gradients of the operators between the products: what holds one shows it, and
nothing else does."""
import pytest

import bitlinear_absmean_ternary_b200 as bl
from test_gpu_train_ops import DTYPES, EPS, dev, gate_backward_ref, tensor, vector  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def same(a, b):
    a, b = a.cpu(), b.cpu()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,F", [(3, 128), (333, 704)])
def test_gate_gradient_from_copies_of_bad_groups(dev, M, F, dtype):
    """A group with an Inf or a NaN restores to NaN, so its gradients are NaN, not those of closed gates."""
    dt = DTYPES[dtype]
    u, g, dh = (tensor(dev, M, F, dtype, s) for s in (1, 2, 3))
    g[0, 5] = float("inf")
    g[1, 64] = float("nan")
    g[2, F - 1] = -float("inf")
    u[0, 64] = float("nan")
    h, u8, us, g8, gs = bl.bitnet_relu2_gate(u, g, checkpoint=True)
    du, dg = bl.bitnet_relu2_gate_backward(dh, u8=u8, u_scale=us, g8=g8, g_scale=gs)
    bad_u, bad_g = (torch.isnan(s).repeat_interleave(64, 1) for s in (us, gs))
    assert int(bad_g.sum()) == 3 * 64 and int(bad_u.sum()) == 64
    assert torch.equal(torch.isnan(du), bad_g) and torch.equal(torch.isnan(dg), bad_g | bad_u)
    zero_u, zero_g = (torch.where(b, torch.zeros((), device=dev), bl.bitnet_act_restore(q, s, torch.float32))
                      for b, q, s in ((bad_u, u8, us), (bad_g, g8, gs)))
    du_ref, dg_ref = (t.to(dt) for t in gate_backward_ref(dh, zero_u.cpu(), zero_g.cpu()))
    assert torch.equal(du.cpu()[~bad_g.cpu()], du_ref[~bad_g.cpu()])
    fine = ~(bad_g | bad_u).cpu()
    assert torch.equal(dg.cpu()[fine], dg_ref[fine])
    # from u and g themselves a NaN closes the gate, and an Inf stays one
    du, dg = bl.bitnet_relu2_gate_backward(dh, u=u, g=g)
    du_ref, dg_ref = gate_backward_ref(dh, u.float().cpu(), g.float().cpu())
    assert same(du, du_ref.to(dt)) and same(dg, dg_ref.to(dt))


NORM_SHAPES = [(37, 256), (37, 2560), (9, 6912), (11, 21504)]


def norm_gradients(kind, form, x, dy, gain):
    """(dx, dgain, dbias or None) from x or from its copy."""
    _, mean, rstd, x8, xs = bl.bitnet_layernorm(x, gain, None, EPS, checkpoint=True)
    kept = {"x": x} if form == "x" else {"x8": x8, "x_scale": xs}
    if kind == "layer":
        return bl.bitnet_layernorm_backward(dy, mean, rstd, gain=gain, **kept)
    return bl.bitnet_rmsnorm_backward(dy, gain=gain, rms_eps=EPS, **kept) + (None,)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["x", "copy"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm_gradients_keep_a_bad_value_in_its_row_and_columns(dev, M, K, kind, form, dtype):
    x, dy = tensor(dev, M, K, dtype, 1, shift=0.3), tensor(dev, M, K, dtype, 2, scale=0.1, loud=False)
    gain = vector(dev, K, dtype, 1)
    base = [None if t is None else t.clone() for t in norm_gradients(kind, form, x, dy, gain)]
    assert all(t is None or bool(torch.isfinite(t).all()) for t in base)
    row, col = 5, K // 2 + 3
    rows = torch.arange(M, device=dev) != row
    cols = torch.arange(K, device=dev) != col

    bad = dy.clone()
    bad[row, col] = float("inf")
    dx, dgain, dbias = norm_gradients(kind, form, x, bad, gain)
    assert torch.equal(dx[rows], base[0][rows]) and not torch.isfinite(dx[row]).any()
    for got, want in ((dgain, base[1]), (dbias, base[2])):
        assert want is None or (torch.equal(got[cols], want[cols]) and not torch.isfinite(got[col]))

    for value in (float("nan"), -float("inf")):
        bad = x.clone()
        bad[row, col] = value
        dx, dgain, dbias = norm_gradients(kind, form, bad, dy, gain)
        assert torch.equal(dx[rows], base[0][rows]) and torch.isnan(dx[row]).all()
        assert dbias is None or torch.equal(dbias, base[2])
        # n of the row is NaN, but of an infinite sum of squares n = x * 0
        alone = kind == "rms" and form == "x" and value == -float("inf")
        assert torch.isnan(dgain[col]) and bool(torch.isfinite(dgain[cols]).all() if alone else torch.isnan(dgain).all())
