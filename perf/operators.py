"""Cases of the operators between the products of a BitLinear training step.

Around the ternary products and their straight-through gradients a training
step needs the norm in front of a BitLinear with its backward pass, the
squared-ReLU gate of the FFN with its backward pass, and the activations that
the backward pass reads, kept in 8 bits (int8 codes, one fp32 scale for each
64 columns of a row).  Each case is one of

  layernorm_fwd     y = (x - mean) * rstd * gain + bias, with mean and rstd
  layernorm_bwd     dx, dgain, dbias from dy and x, or from x's 8-bit copy
  layernorm_step    the forward pass that also writes the 8-bit copy, then the
                    backward pass that reads it
  rmsnorm_bwd       dx, dgain of x * r * gain, r = 1 / sqrt(mean(x^2) + eps),
                    from x or from its 8-bit copy
  checkpoint        x into its 8-bit copy and back
  gate_step         h = relu(g)^2 * u, then du and dg from dh, with u and g
                    kept as they are or in 8 bits in between
  gate_bwd          du and dg from dh and the 8-bit copies of u and g

`M` is tokens, `K` columns, `dtype` the type of every activation, gradient of
an activation, gain and bias; `ckpt` says that the backward pass reads 8-bit
copies.  The gradients of gain and bias are fp32.
"""
import math

import torch

own = False

EPS = 1e-5
GROUP = 64            # columns that share a scale
TINY = 2.0 ** -120    # a group whose largest magnitude is below this is stored as zeros

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_OPS = ("layernorm_fwd", "layernorm_bwd", "layernorm_step", "rmsnorm_bwd", "checkpoint", "gate_step", "gate_bwd")


def listed():
    return [
        # the smallest layer of the benchmark set: four tokens, where a call's latency is all there is
        {"name": "layernorm_fwd_m4_k256_f32", "op": "layernorm_fwd", "M": 4, "K": 256, "dtype": "f32", "ckpt": False},
        # the attention and FFN input norm of the 2.5B block over one training sequence
        {"name": "layernorm_fwd_m4096_k2560", "op": "layernorm_fwd", "M": 4096, "K": 2560, "dtype": "bf16", "ckpt": False},
        # its backward pass with the input still in memory
        {"name": "layernorm_bwd_m4096_k2560", "op": "layernorm_bwd", "M": 4096, "K": 2560, "dtype": "bf16", "ckpt": False},
        # a ragged micro-batch in fp32, as a numerics check or a small model trains it
        {"name": "layernorm_bwd_m333_k640_f32", "op": "layernorm_bwd", "M": 333, "K": 640, "dtype": "f32", "ckpt": False},
        # the 27B block's input norm, forward and backward, with only 8 bits of x kept in between
        {"name": "layernorm_step_m2048_k5376_ckpt", "op": "layernorm_step", "M": 2048, "K": 5376, "dtype": "bf16", "ckpt": True},
        # the same width for a handful of tokens: few rows, so few CTAs' worth of work
        {"name": "rmsnorm_bwd_m16_k5376", "op": "rmsnorm_bwd", "M": 16, "K": 5376, "dtype": "bf16", "ckpt": False},
        # the norm before the 2.5B down projection, from the 8-bit copy
        {"name": "rmsnorm_bwd_m4096_k6912_ckpt", "op": "rmsnorm_bwd", "M": 4096, "K": 6912, "dtype": "bf16", "ckpt": True},
        # the norm before the 27B down projection: the longest rows
        {"name": "rmsnorm_bwd_m2048_k21504", "op": "rmsnorm_bwd", "M": 2048, "K": 21504, "dtype": "bf16", "ckpt": False},
        # one token's copy: the latency of two short kernels
        {"name": "checkpoint_m1_k2560", "op": "checkpoint", "M": 1, "K": 2560, "dtype": "bf16", "ckpt": True},
        # the widest activation of the 27B block, saved and restored
        {"name": "checkpoint_m2048_k21504", "op": "checkpoint", "M": 2048, "K": 21504, "dtype": "bf16", "ckpt": True},
        # the 2.5B FFN's gate over one sequence, u and g kept in 8 bits
        {"name": "gate_step_m4096_k6912_ckpt", "op": "gate_step", "M": 4096, "K": 6912, "dtype": "bf16", "ckpt": True},
        # an odd token count in fp32, u and g kept as they are
        {"name": "gate_step_m77_k6912_f32", "op": "gate_step", "M": 77, "K": 6912, "dtype": "f32", "ckpt": False},
    ]


def draw(rng):
    op = rng.choice(_OPS)
    dtype = "bf16" if rng.random() < 0.7 else "f32"
    ckpt = {"layernorm_fwd": False, "layernorm_step": True, "checkpoint": True, "gate_bwd": True}.get(op, rng.random() < 0.5)
    most = 2048 * 21504 * 2 // (_SIZE[dtype] * (2 if op.endswith("step") or op.startswith("gate") else 1))  # values of one tensor
    K = 64 * int(round(math.exp(rng.uniform(0.0, math.log(21504 / 64)))))
    M = int(round(math.exp(rng.uniform(0.0, math.log(min(16384, most // K))))))
    return {"op": op, "M": max(1, M), "K": K, "dtype": dtype, "ckpt": ckpt}


# ------------------------------------------------------------------ inputs


def _activations(gen, M, K, dtype, shift=0.0):
    """Normal values with 1% of the channels 20 times as large, as a trained
    model's residual stream has them."""
    loud = torch.ones(K, device="cuda")
    at = torch.randint(0, K, (max(1, round(0.01 * K)),), device="cuda", generator=gen)
    loud[at] = 20.0
    x = torch.randn(M, K, device="cuda", generator=gen)
    return (x * loud + shift).to(_DT[dtype])


def _gradient(gen, M, K, dtype):
    return (torch.randn(M, K, device="cuda", generator=gen) * 0.01).to(_DT[dtype])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, K, dt, op = case["M"], case["K"], case["dtype"], case["op"]
    s = dict(case)
    if op.startswith("gate"):
        s["u"], s["g"] = _activations(gen, M, K, dt), _activations(gen, M, K, dt)
        s["dh"] = _gradient(gen, M, K, dt)
    else:
        s["x"] = _activations(gen, M, K, dt, shift=0.25 if op.startswith("layernorm") else 0.0)
    if op.startswith(("layernorm", "rmsnorm")):
        s["gain"] = (torch.rand(K, device="cuda", generator=gen) + 0.5).to(_DT[dt])
        s["bias"] = (torch.randn(K, device="cuda", generator=gen) * 0.1).to(_DT[dt])
        s["dy"] = _gradient(gen, M, K, dt)
    return s


def prepare(case, seed):
    """What the program holds before the call: the inputs and, for a backward
    pass alone, the statistics and the 8-bit copies that the forward left."""
    s = _inputs(case, seed)
    op = s["op"]
    if op == "layernorm_bwd":
        s["mean"], s["rstd"] = _stats(s["x"].float())
    if op in ("layernorm_bwd", "rmsnorm_bwd") and s["ckpt"]:
        s["x8"], s["x_scale"] = _codes(s.pop("x"))
    if op == "gate_bwd":
        s["u8"], s["u_scale"] = _codes(s.pop("u"))
        s["g8"], s["g_scale"] = _codes(s.pop("g"))
    return s


# -------------------------------------------------------------- plain forms


def _codes(x):
    """int8 codes and scales: per row and 64 columns q = round_half_even(
    x * (127 / amax)) and scale = amax / 127, every step rounded to fp32; zeros
    where amax is below 2^-120."""
    M, K = x.shape
    v = x.float().view(M, K // GROUP, GROUP)
    amax = v.abs().amax(dim=2)
    none = amax < TINY
    inv = torch.where(none, torch.zeros_like(amax), torch.full_like(amax, 127.0) / amax)
    q = torch.round(v * inv.unsqueeze(2)).to(torch.int8).view(M, K)
    # a tensor as the divisor: a division by a Python number may become a product with its reciprocal
    scale = torch.where(none, torch.zeros_like(amax), amax / torch.full_like(amax, 127.0))
    return q, scale


def _values(q, scale):
    """What the codes stand for, in fp32."""
    M, K = q.shape
    return (q.view(M, K // GROUP, GROUP).float() * scale.unsqueeze(2)).view(M, K)


def _stats(x):
    mean = x.mean(dim=1)
    var = (x - mean.unsqueeze(1)).square().mean(dim=1)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _layernorm(s):
    x = s["x"].float()
    mean, rstd = _stats(x)
    y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["gain"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _layernorm_backward(dy, x, mean, rstd, gain):
    out = dy.dtype
    dy = dy.float()
    xhat = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    dyg = dy * gain.float()
    m1 = dyg.mean(dim=1, keepdim=True)
    m2 = (dyg * xhat).mean(dim=1, keepdim=True)
    dx = rstd.unsqueeze(1) * (dyg - m1 - xhat * m2)
    return dx.to(out), (dy * xhat).sum(dim=0), dy.sum(dim=0)


def _rmsnorm_backward(dy, x, gain):
    out = dy.dtype
    dy = dy.float()
    r = 1.0 / torch.sqrt(x.square().mean(dim=1, keepdim=True) + EPS)
    xhat = x * r
    dyg = dy * gain.float()
    dx = r * (dyg - xhat * (dyg * xhat).mean(dim=1, keepdim=True))
    return dx.to(out), (dy * xhat).sum(dim=0)


def _gate(u, g):
    r = torch.where(g > 0, g, torch.zeros_like(g)).float()
    return (r * r * u.float()).to(u.dtype)


def _gate_backward(dh, u, g):
    r = torch.where(g > 0, g, torch.zeros_like(g))
    d = dh.float()
    return (d * (r * r)).to(dh.dtype), (d * u * (2.0 * r)).to(dh.dtype)


def _run_plain(s):
    op = s["op"]
    if op == "layernorm_fwd":
        return _layernorm(s)
    if op == "layernorm_bwd":
        x = _values(s["x8"], s["x_scale"]) if s["ckpt"] else s["x"].float()
        return _layernorm_backward(s["dy"], x, s["mean"], s["rstd"], s["gain"])
    if op == "layernorm_step":
        y, mean, rstd = _layernorm(s)
        x8, scale = _codes(s["x"])
        grads = _layernorm_backward(s["dy"], _values(x8, scale), mean, rstd, s["gain"])
        return (y, mean, rstd, scale) + grads
    if op == "rmsnorm_bwd":
        x = _values(s["x8"], s["x_scale"]) if s["ckpt"] else s["x"].float()
        return _rmsnorm_backward(s["dy"], x, s["gain"])
    if op == "checkpoint":
        x8, scale = _codes(s["x"])
        return _values(x8, scale).to(s["x"].dtype), scale
    if op == "gate_step":
        h = _gate(s["u"], s["g"])
        if not s["ckpt"]:
            return (h,) + _gate_backward(s["dh"], s["u"].float(), s["g"].float())
        (u8, us), (g8, gs) = _codes(s["u"]), _codes(s["g"])
        return (h, us, gs) + _gate_backward(s["dh"], _values(u8, us), _values(g8, gs))
    return _gate_backward(s["dh"], _values(s["u8"], s["u_scale"]), _values(s["g8"], s["g_scale"]))


# -------------------------------------------------------- the framework's calls


def _run_own(s):
    import bitlinear_absmean_ternary_b200 as bl

    op = s["op"]
    if op == "layernorm_fwd":
        return bl.bitnet_layernorm(s["x"], s["gain"], s["bias"], EPS)
    if op == "layernorm_bwd":
        if s["ckpt"]:
            return bl.bitnet_layernorm_backward(s["dy"], s["mean"], s["rstd"], x8=s["x8"], x_scale=s["x_scale"],
                                                gain=s["gain"])
        return bl.bitnet_layernorm_backward(s["dy"], s["mean"], s["rstd"], x=s["x"], gain=s["gain"])
    if op == "layernorm_step":
        y, mean, rstd, x8, scale = bl.bitnet_layernorm(s["x"], s["gain"], s["bias"], EPS, checkpoint=True)
        return (y, mean, rstd, scale) + bl.bitnet_layernorm_backward(s["dy"], mean, rstd, x8=x8, x_scale=scale,
                                                                     gain=s["gain"])
    if op == "rmsnorm_bwd":
        if s["ckpt"]:
            return bl.bitnet_rmsnorm_backward(s["dy"], x8=s["x8"], x_scale=s["x_scale"], gain=s["gain"], rms_eps=EPS)
        return bl.bitnet_rmsnorm_backward(s["dy"], x=s["x"], gain=s["gain"], rms_eps=EPS)
    if op == "checkpoint":
        x8, scale = bl.bitnet_act_checkpoint(s["x"])
        return bl.bitnet_act_restore(x8, scale, s["x"].dtype), scale
    if op == "gate_step":
        if not s["ckpt"]:
            h = bl.bitnet_relu2_gate(s["u"], s["g"])
            return (h,) + bl.bitnet_relu2_gate_backward(s["dh"], u=s["u"], g=s["g"])
        h, u8, us, g8, gs = bl.bitnet_relu2_gate(s["u"], s["g"], checkpoint=True)
        return (h, us, gs) + bl.bitnet_relu2_gate_backward(s["dh"], u8=u8, u_scale=us, g8=g8, g_scale=gs)
    return bl.bitnet_relu2_gate_backward(s["dh"], u8=s["u8"], u_scale=s["u_scale"], g8=s["g8"], g_scale=s["g_scale"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------- work


def work(case):
    M, K, op = case["M"], case["K"], case["op"]
    n, b = M * K, _SIZE[case["dtype"]]
    copy = n + 4 * (n // GROUP)  # codes and scales
    kept = copy if case["ckpt"] else n * b
    vec = K * b                  # gain or bias
    if op == "layernorm_fwd":
        return {"bytes": 2 * n * b + 2 * vec + 8 * M, "flops": 8 * n}
    if op == "layernorm_bwd":
        return {"bytes": 2 * n * b + kept + vec + 8 * M + 8 * K, "flops": 13 * n}
    if op == "layernorm_step":
        return {"bytes": (2 * n * b + copy + 2 * vec + 8 * M) + (2 * n * b + copy + vec + 8 * M + 8 * K), "flops": 25 * n}
    if op == "rmsnorm_bwd":
        return {"bytes": 2 * n * b + kept + vec + 4 * K, "flops": 12 * n}
    if op == "checkpoint":
        return {"bytes": 2 * n * b + 2 * copy, "flops": 4 * n}
    if op == "gate_step":
        return {"bytes": 3 * n * b + (2 * copy if case["ckpt"] else 0) + 3 * n * b + 2 * kept, "flops": (16 if case["ckpt"] else 8) * n}
    return {"bytes": 3 * n * b + 2 * copy, "flops": 7 * n}


# ----------------------------------------------------- the definition in 64 bits


def _x64_copy(t):
    """The 8-bit copy of t as 64-bit (values, scales).  The codes' rounding
    border is part of the operator's definition, in fp32 steps."""
    f = t.to(torch.float32).reshape(t.shape[0], -1, GROUP)
    top = f.abs().max(2, keepdim=True).values
    live = top >= TINY
    step = (torch.tensor(127.0, device=t.device).expand_as(top) / top.clamp_min(TINY))
    codes = ((f * step).round() * live).double()
    scale = top.double() / 127.0 * live
    return (codes * scale).reshape(t.shape), scale.squeeze(2)


def _x64_held(s, name):
    """A tensor that the backward pass reads, in 64 bits: from 8 bits as prepare() left them, or as it is."""
    if name + "8" in s:
        q = s[name + "8"].double()
        return (q.reshape(q.shape[0], -1, GROUP) * s[name + "_scale"].double()[:, :, None]).reshape(q.shape)
    return s[name].double()


def _x64_norm_backward(dy, x, centre, r, gain, centred):
    """Gradient of gain * (x - centre) * r for a row: the gradient of a
    normalised vector is the part of gain * dy orthogonal to it (and, with a
    centre, to the vector of ones)."""
    K = x.shape[1]
    n = x.sub(centre).mul_(r)
    gd = dy * gain
    along = torch.einsum("mk,mk->m", gd, n)[:, None] / K
    rest = gd.addcmul(n, along, value=-1.0)
    if centred:
        rest -= gd.sum(1, keepdim=True) / K
    return rest.mul_(r), torch.einsum("mk,mk->k", dy, n)


def exact(case, seed):
    op = case["op"]
    if op == "checkpoint":
        return list(_x64_copy(_inputs(case, seed)["x"]))
    s = prepare(case, seed)
    if op.startswith("gate"):
        dh = s["dh"].double()
        out, held = [], {}
        for name in ("u", "g"):
            if op == "gate_step" and s["ckpt"]:
                held[name], scale = _x64_copy(s[name])
                out.append(scale)
            else:
                held[name] = _x64_held(s, name)
        if op == "gate_step":
            out = [s["g"].double().relu().pow(2) * s["u"].double()] + out
        pos = held["g"].relu()
        return out + [dh * pos.pow(2), dh * held["u"] * pos * 2]
    dy, gain = s["dy"].double(), s["gain"].double()
    if op == "rmsnorm_bwd":
        x = _x64_held(s, "x")
        r = (torch.einsum("mk,mk->m", x, x)[:, None] / x.shape[1] + EPS).rsqrt()
        return list(_x64_norm_backward(dy, x, torch.zeros_like(r), r, gain, False))
    if op == "layernorm_bwd":
        x, centre, r = _x64_held(s, "x"), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        dx, dgain = _x64_norm_backward(dy, x, centre, r, gain, True)
        return [dx, dgain, dy.sum(0)]
    x = s["x"].double()
    var, centre = torch.var_mean(x, dim=1, keepdim=True, correction=0)
    r = (var + EPS).rsqrt()
    y = torch.addcmul(s["bias"].double(), (x - centre) * r, gain)
    if op == "layernorm_fwd":
        return [y, centre[:, 0], r[:, 0]]
    held, scale = _x64_copy(s["x"])
    dx, dgain = _x64_norm_backward(dy, held, centre, r, gain, True)
    return [y, centre[:, 0], r[:, 0], scale, dx, dgain, dy.sum(0)]
