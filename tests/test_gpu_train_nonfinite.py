"""GPU tests of Inf and NaN in the gradients of the operators between the products: what holds one shows it, and
nothing else does."""
import pytest

import bitlinear_absmean_ternary_b200 as bl
from test_gpu_train_ops import DTYPES, dev, gate_backward_ref, tensor  # noqa: F401 (dev is a fixture)

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
