"""GPU tests of the operators between the products at sizes where their kernels take several 16-byte pieces per
thread, add up long columns, or count past 32 bits.

The 8-bit copies take four pieces per thread, the gate with copies two, where that leaves every SM eight CTAs of 256
threads: from 9.7 and 4.9 million bf16 values on 148 SMs, half as many of fp32.  1403 rows of 6976 are above both
and no whole number of CTAs in either type."""
import pytest

import bitlinear_absmean_ternary_b200 as bl
from test_gpu_train_ops import DTYPES, GROUP, codes64, dev, gate_backward_ref, gate_ref, tensor  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

M, K = 1403, 6976


def restored(q, scale, dtype):
    return (q.float().view(q.shape[0], -1, GROUP) * scale.unsqueeze(2)).view(q.shape).to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_copies_bit_for_bit(dev, dtype):
    x = tensor(dev, M, K, dtype, 7)
    x[3, 70], x[1400, 6900] = float("inf"), float("nan")
    q, scale = bl.bitnet_act_checkpoint(x)
    q_ref, s_ref = codes64(x)
    assert torch.equal(q.cpu(), q_ref)
    assert torch.equal(torch.nan_to_num(scale.cpu(), nan=-1.0), torch.nan_to_num(s_ref, nan=-1.0))
    for out in (torch.float32, torch.bfloat16):
        back, want = bl.bitnet_act_restore(q, scale, out).cpu(), restored(q_ref, s_ref, out)
        assert torch.equal(torch.nan_to_num(back, nan=7.0), torch.nan_to_num(want, nan=7.0))
        assert int(torch.isnan(back).sum()) == 2 * GROUP


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_gate_bit_for_bit(dev, dtype):
    dt = DTYPES[dtype]
    u, g, dh = tensor(dev, M, K, dtype, 1), tensor(dev, M, K, dtype, 2), tensor(dev, M, K, dtype, 3, scale=0.01)
    want = gate_ref(u, g).to(dt)
    assert torch.equal(bl.bitnet_relu2_gate(u, g).cpu(), want)
    h, u8, us, g8, gs = bl.bitnet_relu2_gate(u, g, checkpoint=True)
    assert torch.equal(h.cpu(), want)
    f32 = []
    for t, q, s in ((u, u8, us), (g, g8, gs)):
        q_ref, s_ref = codes64(t)
        assert torch.equal(q.cpu(), q_ref) and torch.equal(s.cpu(), s_ref)
        f32.append(restored(q_ref, s_ref, torch.float32))
    for kept, values in (({"u": u, "g": g}, (u.float().cpu(), g.float().cpu())),
                         ({"u8": u8, "u_scale": us, "g8": g8, "g_scale": gs}, f32)):
        for got, ref in zip(bl.bitnet_relu2_gate_backward(dh, **kept), gate_backward_ref(dh, *values)):
            assert torch.equal(got.cpu(), ref.to(dt))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_calls_write_nothing_outside_their_outputs(dev, dtype):
    dt = DTYPES[dtype]
    x, dy = tensor(dev, M, K, dtype, 5), tensor(dev, M, K, dtype, 6)
    arenas = []

    def room(shape, t):
        size = torch.Size(shape).numel() * torch.empty(0, dtype=t).element_size()
        arena = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device=dev)
        arenas.append((arena, size))
        return arena[4096:4096 + size].view(t).view(shape)

    def copy():
        return room((M, K), torch.int8), room((M, K // GROUP), torch.float32)

    x8, xs = bl.bitnet_act_checkpoint(x, *copy())
    bl.bitnet_act_restore(x8, xs, dt, room((M, K), dt))
    bl.bitnet_relu2_gate(x, dy, h=room((M, K), dt))
    bl.bitnet_relu2_gate(x, dy, True, room((M, K), dt), *copy(), *copy())
    bl.bitnet_relu2_gate_backward(dy, x, x, du=room((M, K), dt), dg=room((M, K), dt))
    bl.bitnet_relu2_gate_backward(dy, u8=x8, u_scale=xs, g8=x8, g_scale=xs, du=room((M, K), dt), dg=room((M, K), dt))
    for arena, size in arenas:
        assert bool((arena[:4096] == 0xA5).all()) and bool((arena[4096 + size:] == 0xA5).all())


def column_sums(dy, n):
    """Sums over rows of dy * n and of dy for whole numbers, without a rounding."""
    dgain, dbias = (torch.zeros(dy.shape[1], dtype=torch.int64, device=dy.device) for _ in range(2))
    for i in range(0, dy.shape[0], 1 << 15):
        d = dy[i:i + (1 << 15)].to(torch.int32)
        dgain += (d * n[i:i + (1 << 15)].to(torch.int32)).sum(0)
        dbias += d.sum(0)
    return dgain, dbias


@pytest.mark.parametrize("M,K", [((1 << 21) + 65, 1024), (20011, 32768)])
def test_long_column_sums_of_whole_numbers(dev, M, K):
    """Whole numbers whose sums stay below 2^24 have no rounding in any order, so the gradients of gain and bias are
    exact however long the chains: layer norm with mean 0 and rstd 1, RMSNorm of rows of -1 and 1."""
    if torch.cuda.get_device_properties(dev).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    gen = torch.Generator(device=dev)
    gen.manual_seed(K)
    x8 = torch.randint(-3, 4, (M, K), dtype=torch.int8, device=dev, generator=gen)
    dy = torch.randint(-2, 3, (M, K), dtype=torch.int8, device=dev, generator=gen)
    want_g, want_b = column_sums(dy, x8)
    assert int(want_g.abs().max()) < 1 << 22  # and so do the sums on the way
    dy = dy.to(torch.bfloat16)
    mean, rstd = torch.zeros(M, device=dev), torch.ones(M, device=dev)
    ones = torch.ones(M, K // GROUP, device=dev)
    for kept in ({"x": x8.to(torch.bfloat16)}, {"x8": x8, "x_scale": ones}):
        _, dgain, dbias = bl.bitnet_layernorm_backward(dy, mean, rstd, **kept)
        assert torch.equal(dgain.long(), want_g) and torch.equal(dbias.long(), want_b)
    del kept
    x8 = (x8 & 1) * 2 - 1
    want_g, _ = column_sums(dy, x8)
    for kept in ({"x": x8.to(torch.bfloat16)}, {"x8": x8, "x_scale": ones}):
        _, dgain = bl.bitnet_rmsnorm_backward(dy, rms_eps=1e-12, **kept)
        assert torch.equal(dgain.long(), want_g)


def test_copies_gate_and_rmsnorm_past_32_bits(dev):
    """2^31 + 64 * 704 values in rows of 704: the last rows against the same rows alone."""
    K = 704
    M = (1 << 31) // K + 64
    if torch.cuda.get_device_properties(dev).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x.random_(-100, 100)
    u = x.flip(0)

    def tail(t):
        return t[-5:].contiguous()

    x8, xs = bl.bitnet_act_checkpoint(x)
    for a, b in zip((x8, xs), bl.bitnet_act_checkpoint(tail(x))):
        assert torch.equal(a[-5:], b)
    assert torch.equal(bl.bitnet_relu2_gate(u, x)[-5:], bl.bitnet_relu2_gate(tail(u), tail(x)))
    for a, b in zip(bl.bitnet_relu2_gate(u, x, checkpoint=True),
                    bl.bitnet_relu2_gate(tail(u), tail(x), checkpoint=True)):
        assert torch.equal(a[-5:], b)
    dx, _ = bl.bitnet_rmsnorm_backward(u, x=x)
    assert torch.equal(dx[-5:], bl.bitnet_rmsnorm_backward(tail(u), x=tail(x))[0])
    dx, _ = bl.bitnet_rmsnorm_backward(u, x8=x8, x_scale=xs, dx=dx)
    assert torch.equal(dx[-5:], bl.bitnet_rmsnorm_backward(tail(u), x8=tail(x8), x_scale=tail(xs))[0])
