"""The operators around the token mixer: what is timed, and their plain forms.

Three operators of the block, each with its directions:

  short causal convolution   fwd, bwd, one decode token
  selective state space scan fwd, bwd, one decode token
  layer norm                 fwd (with the residual sum), bwd (with the weight's gradient)

Tokens lie as [B, T, channels]; 2048 channels are the 16 heads of 128 of the
1.3B layer whose other workloads bench.py runs, 6144 its q, k and v paths
side by side, 4096 tokens its training length, 32768 its long context, 256
its decode batch.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
DTYPE = {F32: torch.float32, BF16: torch.bfloat16}
BYTES = {F32: 4, BF16: 2}


def listed():
    return [
        # the q, k and v paths of a training batch or a prompt batch, one call
        dict(name="conv_fwd_qkv", op="conv_fwd", B=8, T=4096, C=6144, K=4, dt=BF16, silu=True,
             state=False),
        # a chunk of a prompt of odd length, three sequences continued from their states
        dict(name="conv_fwd_odd_chunk", op="conv_fwd", B=3, T=1025, C=1030, K=3, dt=F32,
             silu=True, state=True),
        # the backward of one path of a training batch
        dict(name="conv_bwd_train", op="conv_bwd", B=8, T=4096, C=2048, K=4, dt=BF16, silu=True,
             state=False),
        # one decode token of a small batch: latency
        dict(name="conv_step_decode", op="conv_step", B=16, C=6144, K=4, dt=BF16, silu=True),
        # the scan of a training batch, x and z halves of one projection, B and C of another
        dict(name="scan_fwd_train", op="scan_fwd", B=8, T=4096, D=2048, G=1, N=16, dt=BF16,
             gate=True, state=False),
        # one long prompt, continued from a state
        dict(name="scan_fwd_long", op="scan_fwd", B=1, T=32768, D=2048, G=1, N=16, dt=BF16,
             gate=True, state=True),
        # a training batch's backward
        dict(name="scan_bwd_train", op="scan_bwd", B=4, T=4096, D=2048, G=1, N=16, dt=BF16,
             gate=True, state=False),
        # a fine-tuning step in fp32 at odd sizes, two groups of B and C
        dict(name="scan_bwd_odd", op="scan_bwd", B=2, T=777, D=500, G=2, N=8, dt=F32, gate=False,
             state=True),
        # one token of the decode batch
        dict(name="scan_step_decode", op="scan_step", B=256, D=2048, G=1, N=16, dt=BF16,
             gate=True),
        # the pre-norm of a training batch with the residual stream's sum
        dict(name="norm_fwd_train", op="norm_fwd", R=32768, C=2048, dt=BF16, residual=True),
        # the last norm of a small decode batch, fp32, an odd width: latency
        dict(name="norm_fwd_decode", op="norm_fwd", R=5, C=2047, dt=F32, residual=False),
        # the pre-norm's backward, with the residual stream's gradient
        dict(name="norm_bwd_train", op="norm_bwd", R=32768, C=2048, dt=BF16, residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step",
                     "norm_fwd", "norm_bwd"])
    dt = rng.choice([F32, BF16])
    if op.startswith("conv"):
        B, K, silu = _log(rng, 1, 256), rng.choice([2, 3, 4]), rng.random() < 0.7
        C = _log(rng, 16, 6144)
        if op == "conv_step":
            return dict(op=op, B=B, C=C, K=K, dt=dt, silu=silu)
        most = (1 << 26) // (B * C)
        T = _log(rng, 1, max(1, min(32768, most)))
        return dict(op=op, B=B, T=T, C=C, K=K, dt=dt, silu=silu, state=rng.random() < 0.5)
    if op.startswith("scan"):
        B, G, N = _log(rng, 1, 64), rng.choice([1, 1, 2, 4]), _log(rng, 1, 64)
        D = G * _log(rng, 8, 4096 // G)
        gate = rng.random() < 0.7
        if op == "scan_step":
            return dict(op=op, B=B, D=D, G=G, N=N, dt=dt, gate=gate)
        most = ((1 << 29) if op == "scan_fwd" else (1 << 28)) // (B * D * N)
        T = _log(rng, 1, max(1, min(32768, most)))
        return dict(op=op, B=B, T=T, D=D, G=G, N=N, dt=dt, gate=gate, state=rng.random() < 0.5)
    R = _log(rng, 1, 32768)
    C = _log(rng, 32, min(16384, (1 << 26) // R))
    return dict(op=op, R=R, C=C, dt=dt, residual=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPE[case["dt"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    s = dict(case=case)
    op = case["op"]
    if op.startswith("conv"):
        B, C, K = case["B"], case["C"], case["K"]
        # a depthwise filter's usual start: uniform in +-1/sqrt(K)
        s["w"] = (2 * rand(C, K) - 1) / math.sqrt(K)
        s["bias"] = 0.1 * randn(C)
        if op == "conv_step":
            s["x"] = randn(B, C).to(dt)
            s["state"] = randn(B, K - 1, C).to(dt)
            return s
        T = case["T"]
        s["x"] = randn(B, T, C).to(dt)
        s["state"] = randn(B, K - 1, C).to(dt) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = randn(B, T, C).to(dt)
            s["ds"] = randn(B, K - 1, C) if case["state"] else None
        return s
    if op.startswith("scan"):
        B, D, G, N = case["B"], case["D"], case["G"], case["N"]
        # the usual start of a diagonal state matrix, -1 .. -N, moved by training
        s["A"] = -(torch.arange(1, N + 1, device=dev) * torch.exp(0.2 * randn(D, N)))
        s["D"] = 1 + 0.1 * randn(D)
        # steps log-uniform in [1e-3, 1e-1] through the softplus
        step = torch.exp(rand(D) * (math.log(1e-1) - math.log(1e-3)) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        lead = (B,) if op == "scan_step" else (B, case["T"])
        xz = randn(*lead, 2 * D).to(dt)          # one projection: x and the gate's branch
        bc = randn(*lead, 2 * G * N).to(dt)      # another: B and C
        s["x"], z = xz[..., :D], xz[..., D:]
        s["z"] = z if case["gate"] else None
        s["Bm"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["Cm"] = bc[..., G * N:].unflatten(-1, (G, N))
        s["dt"] = (0.5 * randn(*lead, D)).to(dt)
        if op == "scan_step":
            s["state"] = 0.1 * randn(B, D, N)
            return s
        s["h0"] = 0.1 * randn(B, D, N) if case["state"] else None
        if op == "scan_bwd":
            s["dout"] = randn(*lead, D).to(dt)
            s["dh"] = 0.1 * randn(B, D, N) if case["state"] else None
        return s
    R, C = case["R"], case["C"]
    s["x"] = (randn(R, C) * torch.exp(0.5 * randn(R, 1)) + 0.3 * randn(R, 1)).to(dt)
    s["w"] = 1 + 0.1 * randn(C)
    s["b"] = 0.1 * randn(C)
    s["eps"] = 1e-5
    s["res"] = randn(R, C).to(dt) if case["residual"] else None
    if op == "norm_bwd":
        s["dy"] = randn(R, C).to(dt)
    return s


# ---- the calls a user makes ---------------------------------------------------


def _own(s):
    import gated_delta_rule_16_amd as gdr
    case = s["case"]
    op, dt = case["op"], DTYPE[case["dt"]]
    if op == "conv_fwd":
        return gdr.gdr_short_conv_fwd(s["x"], s["w"], s["bias"], s["state"], silu=case["silu"])
    if op == "conv_step":
        y = gdr.gdr_short_conv_step(s["x"], s["w"], s["bias"], s["state"], silu=case["silu"])
        return y, s["state"]
    if op == "conv_bwd":
        dx, dw, db, ds0 = gdr.gdr_short_conv_bwd(
            s["x"], s["w"], s["bias"], s["state"], s["dy"], s["ds"], silu=case["silu"],
            grad_dtype=dt, want_ds0=case["state"])
        return (dx, dw, db, ds0) if case["state"] else (dx, dw, db)
    if op == "scan_fwd":
        return gdr.gdr_ssm_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"],
                                    s["dt_bias"], s["h0"])
    if op == "scan_step":
        y = gdr.gdr_ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], s["D"],
                             s["z"], s["dt_bias"])
        return y, s["state"]
    if op == "scan_bwd":
        got = gdr.gdr_ssm_scan_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"],
                                   s["dt_bias"], s["h0"], s["dout"], s["dh"], grad_dtype=dt,
                                   want_dh0=case["state"])
        return {k: v for k, v in zip(SCAN_GRADS, got) if v is not None}
    if op == "norm_fwd":
        return gdr.gdr_layer_norm_fwd(s["x"], s["w"], s["b"], s["eps"], residual=s["res"])
    return gdr.gdr_layer_norm_bwd(s["x"], s["w"], s["dy"], s["eps"], dres=s["res"], grad_dtype=dt)


SCAN_GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


# ---- plain forms: fp32, rounded once at the end -------------------------------


def _windows(s):
    """The K inputs under each output's filter [B, T, C, K], oldest first."""
    x, K = s["x"].float(), s["case"]["K"]
    state = s["state"]
    past = x.new_zeros(x.shape[0], K - 1, x.shape[2]) if state is None else state.float()
    full = torch.cat([past, x], 1)
    return full, full.unfold(1, K, 1)


def _plain_conv_fwd(s):
    case, dt = s["case"], s["x"].dtype
    full, win = _windows(s)
    u = (win * s["w"]).sum(-1) + s["bias"]
    y = u * torch.sigmoid(u) if case["silu"] else u
    return y.to(dt), full[:, case["T"]:].to(dt)


def _plain_conv_step(s):
    case, dt = s["case"], s["x"].dtype
    win = torch.cat([s["state"].float(), s["x"].float().unsqueeze(1)], 1)     # [B, K, C]
    u = (win * s["w"].t()).sum(1) + s["bias"]
    y = u * torch.sigmoid(u) if case["silu"] else u
    s["state"].copy_(win[:, 1:])
    return y.to(dt), s["state"]


def _plain_conv_bwd(s):
    case, dt = s["case"], s["x"].dtype
    K = case["K"]
    _, win = _windows(s)
    du = s["dy"].float()
    if case["silu"]:
        u = (win * s["w"]).sum(-1) + s["bias"]
        sg = torch.sigmoid(u)
        du = du * sg * (1 + u * (1 - sg))
    dw = (win * du.unsqueeze(-1)).sum((0, 1))
    edge = du.new_zeros(du.shape[0], K - 1, du.shape[2])
    back = torch.cat([edge, du, edge], 1).unfold(1, K, 1)
    dfull = (back * s["w"].flip(1)).sum(-1)                  # [B, K - 1 + T, C]
    if s["ds"] is not None:
        dfull[:, case["T"]:] += s["ds"]
    out = (dfull[:, K - 1:].to(dt), dw, du.sum((0, 1)))
    return out + (dfull[:, :K - 1].contiguous(),) if case["state"] else out


def _prefix(a, b, block=64):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, blocks side by side."""
    T = a.shape[1]
    if T <= block:
        h = b.clone()
        for t in range(1, T):
            h[:, t] += a[:, t] * h[:, t - 1]
        return h
    n = -(-T // block)
    pad = (0, 0) * (a.dim() - 2) + (0, n * block - T)
    at = torch.nn.functional.pad(a, pad).unflatten(1, (n, block))
    h = torch.nn.functional.pad(b, pad).unflatten(1, (n, block))
    for t in range(1, block):
        h[:, :, t] += at[:, :, t] * h[:, :, t - 1]
    decay = torch.cumprod(at, 2)
    carry = _prefix(decay[:, :, -1], h[:, :, -1], block)
    h[:, 1:] += decay[:, 1:] * carry[:, :-1].unsqueeze(2)
    return h.flatten(1, 2)[:, :T]


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _per_channel(m, D):
    """B or C [B, T, G, N] for each of D channels [B, T, D, N]."""
    G = m.shape[-2]
    return m.float().unsqueeze(-2).expand(*m.shape[:-1], D // G, m.shape[-1]).flatten(-3, -2)


def _scan_states(s):
    x, step = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    D = x.shape[-1]
    decay = torch.exp(step.unsqueeze(-1) * s["A"])
    h = (step * x).unsqueeze(-1) * _per_channel(s["Bm"], D)
    if s["h0"] is not None:
        h[:, 0] += decay[:, 0] * s["h0"]
    return x, step, decay, _prefix(decay, h)


def _plain_scan_fwd(s):
    x, _, _, h = _scan_states(s)
    y = (h * _per_channel(s["Cm"], x.shape[-1])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype), h[:, -1].contiguous()


def _plain_scan_step(s):
    x, step = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    D = x.shape[-1]
    h = s["state"] * torch.exp(step.unsqueeze(-1) * s["A"])
    h = h + (step * x).unsqueeze(-1) * _per_channel(s["Bm"], D)
    y = (h * _per_channel(s["Cm"], D)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    s["state"].copy_(h)
    return y.to(s["x"].dtype), s["state"]


def _plain_scan_bwd(s):
    dt = s["x"].dtype
    x, step, decay, h = _scan_states(s)
    B, T, D = x.shape
    G, N = s["Bm"].shape[-2:]
    bm, cm = _per_channel(s["Bm"], D), _per_channel(s["Cm"], D)
    dy = s["dout"].float()
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        y = (h * cm).sum(-1) + s["D"] * x
        out["dz"] = (dy * y * sg * (1 + z * (1 - sg))).to(dt)
        dy = dy * z * sg
    # g_t = C_t dy_t + decay_{t+1} g_{t+1}, as a prefix over reversed time
    g = dy.unsqueeze(-1) * cm
    if s["dh"] is not None:
        g[:, -1] += s["dh"]
    later = torch.cat([decay[:, 1:], torch.zeros_like(decay[:, :1])], 1)
    g = _prefix(later.flip(1), g.flip(1)).flip(1)
    out["dC"] = (h * dy.unsqueeze(-1)).unflatten(2, (G, D // G)).sum(3).to(dt)
    out["dB"] = (g * (step * x).unsqueeze(-1)).unflatten(2, (G, D // G)).sum(3).to(dt)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"].unsqueeze(1)
    gah = g * decay * torch.cat([first, h[:, :-1]], 1)
    gb = (g * bm).sum(-1)
    dstep = x * gb + (gah * s["A"]).sum(-1)
    draw_ = dstep * torch.sigmoid(s["dt"].float() + s["dt_bias"])
    out["dx"] = (step * gb + s["D"] * dy).to(dt)
    out["ddt"] = draw_.to(dt)
    out["dA"] = (gah * step.unsqueeze(-1)).sum((0, 1))
    out["dD"] = (dy * x).sum((0, 1))
    out["ddt_bias"] = draw_.sum((0, 1))
    if s["case"]["state"]:
        out["dh0"] = g[:, 0] * decay[:, 0]
    return {k: out[k] for k in SCAN_GRADS if k in out}


def _plain_norm_fwd(s):
    dt = s["x"].dtype
    h = s["x"].float()
    if s["res"] is not None:
        # the norm is of the residual stream as it is stored
        stored = (h + s["res"].float()).to(dt)
        h = stored.float()
    c = h - h.mean(-1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["w"] + s["b"]
    return (y.to(dt), stored) if s["res"] is not None else y.to(dt)


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"])
    n = c * rstd
    dn = dy * s["w"]
    dx = rstd * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_step": _plain_conv_step, "conv_bwd": _plain_conv_bwd,
         "scan_fwd": _plain_scan_fwd, "scan_step": _plain_scan_step, "scan_bwd": _plain_scan_bwd,
         "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    op, e = case["op"], BYTES[case["dt"]]
    if op.startswith("conv"):
        B, C, K = case["B"], case["C"], case["K"]
        state = B * (K - 1) * C
        if op == "conv_step":
            return dict(bytes=2 * B * C * e + 2 * state * e + 4 * C * (K + 1),
                        flops=B * C * (2 * K + 4))
        n = B * case["T"] * C
        kept = state * e if case["state"] else 0
        if op == "conv_fwd":
            return dict(bytes=2 * n * e + 4 * C * (K + 1) + kept + state * e,
                        flops=n * (2 * K + 4))
        return dict(bytes=3 * n * e + 8 * C * (K + 1) + kept + (8 * state if case["state"] else 0),
                    flops=n * (6 * K + 8))
    if op.startswith("scan"):
        B, D, G, N = case["B"], case["D"], case["G"], case["N"]
        gate, state = int(case["gate"]), B * D * N * 4
        consts = 4 * D * (N + 2)
        if op == "scan_step":
            return dict(bytes=B * (D * (3 + gate) + 2 * G * N) * e + 2 * state + consts,
                        flops=B * D * (7 * N + 12))
        tok = B * case["T"]
        if op == "scan_fwd":
            return dict(bytes=tok * (D * (3 + gate) + 2 * G * N) * e + consts +
                        (2 if case["state"] else 1) * state, flops=tok * D * (7 * N + 12))
        return dict(bytes=tok * (D * (5 + 2 * gate) + 4 * G * N) * e + 2 * consts +
                    (3 * state if case["state"] else 0), flops=tok * D * (21 * N + 30))
    R, C, res = case["R"], case["C"], int(case["residual"])
    if op == "norm_fwd":
        return dict(bytes=R * C * e * (2 + 2 * res) + 8 * C, flops=R * C * 8)
    return dict(bytes=R * C * e * (3 + res) + 12 * C, flops=R * C * 16)


# ---- 64 bits, from the definitions, token by token ---------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("conv"):
        return _exact_conv(s, case)
    if op.startswith("scan"):
        return _exact_scan(s, case)
    return _exact_norm(s, case)


def _silu64(u):
    return u / (1 + torch.exp(-u))


def _dsilu64(u):
    e = torch.exp(-u)
    return 1 / (1 + e) + u * e / (1 + e) ** 2


def _exact_conv(s, case):
    K, C = case["K"], case["C"]
    x, w, bias = s["x"].double(), s["w"].double(), s["bias"].double()
    if case["op"] == "conv_step":
        x = x[:, None]
    B, T = x.shape[0], x.shape[1]
    past = torch.zeros(B, K - 1, C, dtype=x.dtype, device=x.device)
    if s["state"] is not None:
        past = s["state"].double()
    full = torch.cat([past, x], 1)
    u = bias.expand(B, T, C).clone()
    for j in range(K):
        u += w[:, j] * full[:, j:j + T]
    if case["op"] != "conv_bwd":
        y = _silu64(u) if case["silu"] else u
        if case["op"] == "conv_step":
            y = y[:, 0]
        return y, full[:, T:]
    du = s["dy"].double()
    if case["silu"]:
        du = du * _dsilu64(u)
    dw = torch.stack([(du * full[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
    dfull = torch.zeros_like(full)
    for j in range(K):
        dfull[:, j:j + T] += w[:, j] * du
    if s["ds"] is not None:
        dfull[:, T:] += s["ds"].double()
    out = (dfull[:, K - 1:], dw, du.sum((0, 1)))
    return out + (dfull[:, :K - 1],) if case["state"] else out


def _exact_scan(s, case):
    op, D, G, N = case["op"], case["D"], case["G"], case["N"]
    x, raw = s["x"].double(), s["dt"].double() + s["dt_bias"].double()
    bm, cm, A, skip = s["Bm"].double(), s["Cm"].double(), s["A"].double(), s["D"].double()
    z = None if s["z"] is None else s["z"].double()
    if op == "scan_step":
        x, raw, bm, cm = x[:, None], raw[:, None], bm[:, None], cm[:, None]
        z = None if z is None else z[:, None]
    B, T = x.shape[0], x.shape[1]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    start = s["state"] if op == "scan_step" else s["h0"]
    h = x.new_zeros(B, D, N) if start is None else start.double()

    def spread(m):          # [B, G, N] -> [B, D, N]
        return m.repeat_interleave(D // G, dim=1)

    back = op == "scan_bwd"
    hs, ys = [h], []
    for t in range(T):
        h = torch.exp(step[:, t, :, None] * A) * h + \
            (step[:, t] * x[:, t])[:, :, None] * spread(bm[:, t])
        ys.append((h * spread(cm[:, t])).sum(-1) + skip * x[:, t])
        if back:
            hs.append(h)
    y = torch.stack(ys, 1)
    if not back:
        if z is not None:
            y = y * _silu64(z)
        return (y[:, 0] if op == "scan_step" else y), h
    dout = s["dout"].double()
    dy = dout if z is None else dout * _silu64(z)
    g = x.new_zeros(B, D, N) if s["dh"] is None else s["dh"].double()
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(skip), torch.zeros_like(skip)
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(bm), torch.empty_like(cm)
    for t in range(T - 1, -1, -1):
        dyt, st, xt = dy[:, t, :, None], step[:, t, :, None], x[:, t, :, None]
        g = g + dyt * spread(cm[:, t])
        dC[:, t] = (hs[t + 1] * dyt).view(B, G, D // G, N).sum(2)
        dB[:, t] = (g * st * xt).view(B, G, D // G, N).sum(2)
        gb = (g * spread(bm[:, t])).sum(-1)
        a = torch.exp(st * A)
        da = g * hs[t] * a                       # dL/d(step A) per state
        dx[:, t] = step[:, t] * gb + skip * dy[:, t]
        dr = ((da * A).sum(-1) + x[:, t] * gb) / (1 + torch.exp(-raw[:, t]))
        ddt[:, t] = dr
        dA += (da * st).sum(0)
        dD += (dy[:, t] * x[:, t]).sum(0)
        dbias += dr.sum(0)
        g = g * a
    out = dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD)
    if z is not None:
        out["dz"] = dout * y * _dsilu64(z)
    out["ddt_bias"] = dbias
    if case["state"]:
        out["dh0"] = g
    return out


def _exact_norm(s, case):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    C = case["C"]
    stored = None
    if case["op"] == "norm_fwd" and s["res"] is not None:
        # the sum is rounded where it is stored, and that value is normalised
        stored = (s["x"].float() + s["res"].float()).to(s["x"].dtype).double()
        x = stored
    mu = x.sum(-1, keepdim=True) / C
    sd = torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / C + s["eps"])
    n = (x - mu) / sd
    if case["op"] == "norm_fwd":
        y = n * w + b
        return y if stored is None else (y, stored)
    dy = s["dy"].double()
    dn = dy * w
    dx = (dn - dn.sum(-1, keepdim=True) / C - n * (dn * n).sum(-1, keepdim=True) / C) / sd
    if s["res"] is not None:
        dx = dx + s["res"].double()
    return dx, (dy * n).sum(0), dy.sum(0)
