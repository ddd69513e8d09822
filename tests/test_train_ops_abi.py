"""Refusals of the operators between the products of a training step: every
call below fails validation on the host, so nothing is launched and no address
is dereferenced.  Also the binding's refusal of host tensors."""
import math

import pytest

import bitlinear_absmean_ternary_b200 as bl
from bitlinear_absmean_ternary_b200 import build as blbuild

FAKE = 0x10000   # 16-byte aligned, never dereferenced: validation fails first
MIS = FAKE + 4
ARG, SHAPE = bl.BITNET_ERR_INVALID_ARG, bl.BITNET_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    return bl.lib()


def test_declared_and_bound(L):
    names = {"bitnet_act_checkpoint", "bitnet_act_restore", "bitnet_layernorm", "bitnet_layernorm_backward",
             "bitnet_rmsnorm_backward", "bitnet_norm_backward_workspace_bytes", "bitnet_relu2_gate",
             "bitnet_relu2_gate_backward"}
    assert names <= set(bl.declared_functions())
    for n in names:
        assert hasattr(L, n) and callable(getattr(bl, n))


def test_copies_refuse(L):
    for fn in ("checkpoint", "restore"):
        def call(x=FAKE, dt=bl.BITNET_F32, M=4, K=64, x8=FAKE, s=FAKE):
            if fn == "checkpoint":
                return L.bitnet_act_checkpoint(x, dt, M, K, x8, s, None)
            return L.bitnet_act_restore(x8, s, M, K, x, dt, None)

        for kw in ({"x": None}, {"x8": None}, {"s": None}, {"x": MIS}, {"x8": MIS}, {"s": FAKE + 2},
                   {"dt": bl.BITNET_I32}, {"dt": 7}):
            assert call(**kw) == ARG, kw
        for kw in ({"K": 0}, {"K": 96}, {"K": -64}, {"M": 0}, {"M": 1 << 31}, {"M": 1 << 30, "K": 1 << 12}):
            assert call(**kw) == SHAPE, kw


def test_layernorm_refuses(L):
    def call(x=FAKE, dt=bl.BITNET_BF16, M=4, K=64, g=FAKE, b=FAKE, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE, x8=FAKE,
             s=FAKE):
        return L.bitnet_layernorm(x, dt, M, K, g, b, eps, y, mean, rstd, x8, s, None)

    for kw in ({"x": None}, {"y": None}, {"x": MIS}, {"y": MIS}, {"g": MIS}, {"b": MIS}, {"x8": MIS},
               {"mean": FAKE + 2}, {"rstd": FAKE + 1}, {"s": FAKE + 2}, {"x8": None}, {"s": None},
               {"dt": bl.BITNET_I32}, {"eps": 0.0}, {"eps": -1.0}, {"eps": math.nan}, {"eps": math.inf}):
        assert call(**kw) == ARG, kw
    for kw in ({"K": 32}, {"K": 32768 + 64}, {"M": 0}, {"M": -1}, {"M": 1 << 31}):
        assert call(**kw) == SHAPE, kw


def test_norm_backward_refuses(L):
    assert bl.bitnet_norm_backward_workspace_bytes(0, 64) == 0
    assert bl.bitnet_norm_backward_workspace_bytes(4, 100) == 0
    assert bl.bitnet_norm_backward_workspace_bytes(4, 32768 + 64) == 0
    for M, K in ((1, 64), (4, 256), (4096, 2560), (2048, 21504), (1 << 30, 64)):
        assert 0 < bl.bitnet_norm_backward_workspace_bytes(M, K) < (1 << 30) + 5 * M

    def common(call):
        for kw in ({"dy": None}, {"dx": None}, {"dy": MIS}, {"dx": MIS}, {"x": MIS}, {"g": MIS}, {"dg": MIS},
                   {"x": None}, {"x8": FAKE}, {"x8": FAKE, "s": FAKE}, {"s": FAKE}, {"x": None, "x8": FAKE},
                   {"x": None, "x8": MIS, "s": FAKE}, {"x": None, "x8": FAKE, "s": FAKE + 2},
                   {"dt": bl.BITNET_I32}, {"ws": None}, {"ws": MIS}, {"wsb": 0}, {"wsb": 64}):
            assert call(**kw) == ARG, kw
        for kw in ({"K": 32}, {"K": 32768 + 64}, {"M": 0}, {"M": 1 << 31}):
            assert call(**kw) == SHAPE, kw

    def ln(dy=FAKE, dt=bl.BITNET_BF16, M=4, K=64, x=FAKE, x8=None, s=None, mean=FAKE, rstd=FAKE, g=FAKE, dx=FAKE,
           dg=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30):
        return L.bitnet_layernorm_backward(dy, dt, M, K, x, x8, s, mean, rstd, g, dx, dg, db, ws, wsb, None)

    def rms(dy=FAKE, dt=bl.BITNET_BF16, M=4, K=64, x=FAKE, x8=None, s=None, g=FAKE, eps=1e-5, dx=FAKE, dg=FAKE,
            ws=FAKE, wsb=1 << 30):
        return L.bitnet_rmsnorm_backward(dy, dt, M, K, x, x8, s, g, eps, dx, dg, ws, wsb, None)

    common(ln)
    common(rms)
    for kw in ({"mean": None}, {"rstd": None}, {"mean": FAKE + 2}, {"db": MIS}, {"dg": None, "ws": None}):
        assert ln(**kw) == ARG, kw
    for kw in ({"eps": 0.0}, {"eps": math.nan}):
        assert rms(**kw) == ARG, kw


def test_gate_refuses(L):
    def fwd(u=FAKE, g=FAKE, dt=bl.BITNET_F32, M=4, F=64, h=FAKE, u8=FAKE, us=FAKE, g8=FAKE, gs=FAKE):
        return L.bitnet_relu2_gate(u, g, dt, M, F, h, u8, us, g8, gs, None)

    for kw in ({"u": None}, {"g": None}, {"h": None}, {"u": MIS}, {"g": MIS}, {"h": MIS}, {"u8": MIS}, {"g8": MIS},
               {"us": FAKE + 2}, {"gs": FAKE + 2}, {"u8": None}, {"us": None}, {"g8": None}, {"gs": None},
               {"dt": bl.BITNET_I32}):
        assert fwd(**kw) == ARG, kw
    for kw in ({"F": 65}, {"M": 0}, {"M": 1 << 30, "F": 1 << 12}):
        assert fwd(**kw) == SHAPE, kw

    def bwd(dh=FAKE, dt=bl.BITNET_F32, M=4, F=64, u=FAKE, g=FAKE, u8=None, us=None, g8=None, gs=None, du=FAKE, dg=FAKE):
        return L.bitnet_relu2_gate_backward(dh, dt, M, F, u, g, u8, us, g8, gs, du, dg, None)

    copies = {"u": None, "g": None, "u8": FAKE, "us": FAKE, "g8": FAKE, "gs": FAKE}
    for kw in ({"dh": None}, {"du": None}, {"dg": None}, {"u": None}, {"g": None}, {"u": None, "g": None},
               {"u8": FAKE}, {"gs": FAKE}, {"u8": FAKE, "us": FAKE, "g8": FAKE, "gs": FAKE},
               {"dh": MIS}, {"du": MIS}, {"dg": MIS}, {"u": MIS}, {"dt": 5},
               {**copies, "u": FAKE}, {**copies, "g": FAKE}, {**copies, "us": None}, {**copies, "gs": None},
               {**copies, "u8": MIS}, {**copies, "gs": FAKE + 2}):
        assert bwd(**kw) == ARG, kw
    for kw in ({"F": 0}, {"M": 0}, {**copies, "F": 96}):
        assert bwd(**kw) == SHAPE, kw


def test_binding_refuses_host_tensors(L):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    v = torch.zeros(2)
    x8, s = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 1)
    for call in (lambda: bl.bitnet_act_checkpoint(x), lambda: bl.bitnet_act_restore(x8, s),
                 lambda: bl.bitnet_layernorm(x), lambda: bl.bitnet_layernorm_backward(x, v, v, x=x),
                 lambda: bl.bitnet_rmsnorm_backward(x, x=x), lambda: bl.bitnet_relu2_gate(x, x),
                 lambda: bl.bitnet_relu2_gate_backward(x, u=x, g=x)):
        with pytest.raises(ValueError):
            call()
