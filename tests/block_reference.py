"""Plain fp64 NumPy forms of the operators around the mixer, token by token,
and the error bounds that their tests use.

A bound is c 2^-24 times a majorant: the same formulas with every input
replaced by its absolute value (sums then have no cancellation), which bounds
each intermediate of the fp32 evaluation.  c counts the roundings on the
longest chain.  A store in fewer bits adds half a step of the value.
"""
import numpy as np

U = 2.0 ** -24                      # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of a store


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(x, 0.0)


# ---- short causal convolution ---------------------------------------------------


def conv_full(x, s0, K):
    B, T, C = x.shape
    past = np.zeros((B, K - 1, C)) if s0 is None else s0
    return np.concatenate([past, x], 1)


def conv_fwd(x, w, bias, s0, silu):
    """(y, s_final, u, majorant of u)"""
    K, T = w.shape[1], x.shape[1]
    full = conv_full(x, s0, K)
    u = np.zeros_like(x) + (0.0 if bias is None else bias)
    m = np.zeros_like(x) + (0.0 if bias is None else np.abs(bias))
    for j in range(K):
        u = u + w[:, j] * full[:, j:j + T]
        m = m + np.abs(w[:, j] * full[:, j:j + T])
    return (u * sigmoid(u) if silu else u), full[:, T:], u, m


def conv_fwd_bound(y, u, m, K, silu, out):
    """K fused adds err by K U m; SiLU' is at most 1.1; SiLU itself (exp,
    add, reciprocal, two products, each within a step) by 12 U |y|."""
    b = 1.1 * (K + 1) * U * m + (12 * U * np.abs(y) if silu else 0.0)
    return b * 1.01 + HALF[out] * (np.abs(y) + b)


def conv_bwd(x, w, bias, s0, dy, ds_final, silu):
    """Values and majorants of (dx, dw, dbias, ds0)."""
    K = w.shape[1]
    B, T, C = x.shape
    full = conv_full(x, s0, K)
    _, _, u, m = conv_fwd(x, w, bias, s0, silu)
    sg = sigmoid(u)
    f = sg * (1 + u * (1 - sg)) if silu else np.ones_like(u)
    du = dy * f
    # error of du in units of U: |SiLU''| <= 0.5 times the error of u, and 16
    # roundings of the factor, whose terms are at most 1 + |u|
    edu = np.abs(dy) * ((0.5 * (K + 1) * m + 16 * (1 + np.abs(u))) if silu else 1.0)
    out = []
    for g, aw, ax in ((du, w, full), (edu + (K + 2) * np.abs(du), np.abs(w), np.abs(full))):
        dw = np.stack([(g * ax[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
        df = np.zeros_like(full)
        for j in range(K):
            df[:, j:j + T] += aw[:, j] * g
        if ds_final is not None:
            df[:, T:] += ds_final if g is du else np.abs(ds_final)
        out.append([df[:, K - 1:], dw, g.sum((0, 1)), df[:, :K - 1]])
    # sums over the B T tokens of dw and dbias: one more rounding per term
    vals, bounds = out
    n = B * T
    bounds[1] = bounds[1] + n * np.stack(
        [np.abs(du * full[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
    bounds[2] = bounds[2] + n * np.abs(du).sum((0, 1))
    return vals, [1.01 * U * b for b in bounds]


# ---- selective scan ----------------------------------------------------------------


def _spread(m, D):
    return np.repeat(m, D // m.shape[1], axis=1)


def scan_fwd(x, dt, A, Bm, Cm, D, z, bias, h0, sp=True, majorant=False):
    """(y, h_final, all states [T + 1]); majorant: every term's absolute value."""
    ab = np.abs if majorant else (lambda v: v)
    B, T, Dn = x.shape
    N = A.shape[1]
    raw = dt + (0.0 if bias is None else bias)
    step = softplus(raw) if sp else raw
    h = np.zeros((B, Dn, N)) if h0 is None else ab(h0)
    hs, y = [h], np.zeros_like(x)
    for t in range(T):
        h = np.exp(step[:, t, :, None] * A) * h + \
            ab((step[:, t] * x[:, t])[:, :, None] * _spread(Bm[:, t], Dn))
        hs.append(h)
        y[:, t] = (h * ab(_spread(Cm[:, t], Dn))).sum(-1)
        if D is not None:
            y[:, t] += ab(D * x[:, t])
    if z is not None:
        y = y * ab(z * sigmoid(z))
    return y, h, hs


def scan_bwd(x, dt, A, Bm, Cm, D, z, bias, h0, dout, dh, sp=True, majorant=False):
    """dict of gradients; majorant: every term's absolute value."""
    ab = np.abs if majorant else (lambda v: v)
    B, T, Dn = x.shape
    G, N = Bm.shape[2:]
    raw = dt + (0.0 if bias is None else bias)
    step = softplus(raw) if sp else raw
    dsp = sigmoid(raw) if sp else np.ones_like(raw)
    _, _, hs = scan_fwd(x, dt, A, Bm, Cm, D, None, bias, h0, sp, majorant)
    zs = np.ones_like(x) if z is None else z * sigmoid(z)
    dy = ab(dout * zs)
    skip = np.zeros(Dn) if D is None else D
    g = np.zeros((B, Dn, N)) if dh is None else ab(dh)
    o = {k: np.zeros(s) for k, s in (("dx", x.shape), ("ddt", x.shape), ("dA", A.shape),
                                     ("dB", Bm.shape), ("dC", Bm.shape), ("dD", (Dn,)),
                                     ("dz", x.shape), ("db", (Dn,)))}
    for t in range(T - 1, -1, -1):
        c, b = _spread(Cm[:, t], Dn), _spread(Bm[:, t], Dn)
        g = g + ab(dy[:, t, :, None] * c)
        o["dC"][:, t] = (hs[t + 1] * dy[:, t, :, None]).reshape(B, G, Dn // G, N).sum(2)
        o["dB"][:, t] = (g * ab(step[:, t] * x[:, t])[:, :, None]).reshape(
            B, G, Dn // G, N).sum(2)
        gb = (g * ab(b)).sum(-1)
        a = np.exp(step[:, t, :, None] * A)
        p = g * hs[t] * a
        o["dx"][:, t] = ab(step[:, t]) * gb + ab(skip) * dy[:, t]
        dr = ((p * ab(A)).sum(-1) + ab(x[:, t]) * gb) * dsp[:, t]
        o["ddt"][:, t] = dr
        o["dA"] += (p * ab(step[:, t])[:, :, None]).sum(0)
        o["dD"] += ab(dy[:, t] * x[:, t]).sum(0) if majorant else (dy[:, t] * x[:, t]).sum(0)
        o["db"] += dr.sum(0)
        if z is not None:
            zz, sg = z[:, t], sigmoid(z[:, t])
            y = (hs[t + 1] * ab(c)).sum(-1) + ab(skip * x[:, t])
            f = sg * (1 + zz * (1 - sg))
            # the majorant of 1 + z (1 - sg) has no cancellation either
            o["dz"][:, t] = ab(dout[:, t]) * y * (sg * (1 + ab(zz) * (1 - sg)) if majorant else f)
        g = g * a
    o["dh0"] = g
    return o


def scan_bound(majorant, steps, out="f32", value=None):
    """Each of the `steps` products and sums of a chain adds at most 4 roundings
    (the exponent's product and A log2 e, exp, the fused add), Delta's own 8
    enter through the exponent, whose effect x exp(-x) the majorant of the
    neighbouring token covers; 64 more for SiLU, softplus and the sums over n.
    1e-30: factors below 2^-126 become 0 before their product with others, which
    stay below 2^26."""
    b = 4 * (steps + 16) * U * majorant + 1e-30
    return b if value is None else b + HALF[out] * (np.abs(value) + b)


# ---- layer norm ------------------------------------------------------------------------


def norm_fwd(h, w, b, eps):
    mu = h.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((h - mu) ** 2).mean(-1, keepdims=True) + eps)
    y = (h - mu) * r
    return (y if w is None else y * w) + (0.0 if b is None else b)


def norm_depth(C):
    """Roundings of a row's sum: a thread's own channels one by one, then the
    lanes, then the waves."""
    per = -(-C // 64) if C <= 2048 else -(-C // 256)
    return max(per, 8) + 8


def norm_fwd_bound(h, w, b, eps, out):
    """mean errs by d U mean|h| (d: depth of the sum); the centred value by that
    and U |h - mu|; rstd relatively by the centred values' relative error and
    (d + 4) U."""
    C = h.shape[-1]
    d = norm_depth(C)
    mu = h.mean(-1, keepdims=True)
    c = h - mu
    var = (c * c).mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    ec = U * ((d + 2) * np.abs(h).mean(-1, keepdims=True) + np.abs(c))
    er = (d + 4) * U + r * r * (2 * np.abs(c) * ec + ec * ec).mean(-1, keepdims=True)
    w = 1.0 if w is None else np.abs(w)
    b = 0.0 if b is None else np.abs(b)
    n = np.abs(c) * r
    e = (r * ec + n * (er + 4 * U)) * w * 1.05 + 4 * U * (n * w + b)
    return e + HALF[out] * (n * w + b + e)


def norm_bwd(x, w, dy, eps, dres):
    """Values and bounds of (dx, dw, db)."""
    C = x.shape[-1]
    d = norm_depth(C)
    mu = x.mean(-1, keepdims=True)
    c = x - mu
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n, dn = c * r, dy * (1.0 if w is None else w)
    m1, m2 = dn.mean(-1, keepdims=True), (dn * n).mean(-1, keepdims=True)
    dx = r * (dn - m1 - n * m2) + (0.0 if dres is None else dres)
    ec = U * ((d + 2) * np.abs(x).mean(-1, keepdims=True) + np.abs(c))
    er = (d + 4) * U + r * r * (2 * np.abs(c) * ec + ec * ec).mean(-1, keepdims=True)
    en = r * ec + np.abs(n) * (er + 2 * U)
    adn = np.abs(dn)
    e1 = (d + 4) * U * adn.mean(-1, keepdims=True)
    am2 = (adn * np.abs(n)).mean(-1, keepdims=True)
    e2 = (d + 4) * U * am2 + (adn * en).mean(-1, keepdims=True)
    mag = adn + np.abs(m1) + np.abs(n) * am2
    edx = r * (e1 + en * am2 + np.abs(n) * e2 + (er + 6 * U) * mag) * 1.05
    if dres is not None:
        edx = edx + 2 * U * (np.abs(dres) + r * mag)
    R = x.shape[0]
    dw, db = (dy * n).sum(0), dy.sum(0)
    ew = (np.abs(dy) * en).sum(0) + (R + 4) * U * np.abs(dy * n).sum(0)
    eb = (R + 4) * U * np.abs(dy).sum(0)
    return [dx, dw, db], [edx, 1.05 * ew, 1.05 * eb]
