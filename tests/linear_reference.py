"""Plain fp64 NumPy forms of linear attention, rotary positions and RMS norm, token
by token, and the error bounds that their tests use.

Linear attention's bounds come from two recursions beside the values: a majorant M
(every input by its absolute value, so no sum cancels) and its first moment in the
decay's exponent D = sum |d| e^{-|d|} .. (what a relative error of the exponents
costs).  An output errs by at most U (c M + 8 D), c the number of roundings on the
longest chain, plus half a step of its own type at the store.
"""
import numpy as np

from block_reference import HALF, U, norm_depth

TINY = 1e-30        # terms under 2^-126 count as 0 before their products with others


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


# ---- linear attention ---------------------------------------------------------------


def spread(x, H):
    """[B, T, Hk, D] for each of H heads."""
    return np.repeat(x, H // x.shape[2], axis=2)


def decays(g, B, T, H):
    return np.zeros((B, T, H)) if g is None else np.broadcast_to(np.maximum(g, -1e4), (B, T, H))


def la_fwd(q, k, v, g, s0, scale):
    """(o, s_final, their majorants, their moments)"""
    B, T, H, Dv = v.shape
    q, k, g = spread(q, H), spread(k, H), decays(g, B, T, H)
    S = np.zeros((B, H, Dv, k.shape[-1])) if s0 is None else s0.copy()
    M, D = np.abs(S), np.zeros_like(S)
    o, mo, do = np.zeros_like(v), np.zeros_like(v), np.zeros_like(v)
    for t in range(T):
        x = np.abs(g[:, t, :, None, None])
        a = np.exp(-x) if (g[:, t] <= 0).all() else np.exp(g[:, t, :, None, None])
        S = a * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        D = a * (D + x * M)
        M = a * M + np.abs(v[:, t, :, :, None] * k[:, t, :, None, :])
        o[:, t] = scale * (S * q[:, t, :, None, :]).sum(-1)
        aq = np.abs(q[:, t, :, None, :])
        mo[:, t] = abs(scale) * (M * aq).sum(-1)
        do[:, t] = abs(scale) * (D * aq).sum(-1)
    return (o, S), (mo, M), (do, D)


def la_bwd(q, k, v, g, s0, dout, ds, scale):
    """dicts of values, majorants and moments of dq, dk, dv, dg, ds0"""
    B, T, H, Dv = v.shape
    Hk, Dk = k.shape[2:]
    fq, fk, fg = spread(q, H), spread(k, H), decays(g, B, T, H)
    S = np.zeros((B, H, Dv, Dk)) if s0 is None else s0.copy()
    out = []
    states = [(S, np.abs(S), np.zeros_like(S))]
    a = np.exp(fg)[..., None, None]
    x = np.abs(fg)[..., None, None]
    for t in range(T):
        S, M, D = states[-1]
        vk = v[:, t, :, :, None] * fk[:, t, :, None, :]
        states.append((a[:, t] * S + vk, a[:, t] * M + np.abs(vk), a[:, t] * (D + x[:, t] * M)))
    G = np.zeros_like(S) if ds is None else ds.copy()
    G = (G, np.abs(G), np.zeros_like(G))
    r = [dict(dq=np.zeros_like(fq), dk=np.zeros_like(fk), dv=np.zeros_like(v),
              dg=np.zeros((B, T, H))) for _ in range(3)]
    for t in range(T - 1, -1, -1):
        dq = scale * dout[:, t, :, :, None] * fq[:, t, :, None, :]
        G = (G[0] + dq, G[1] + np.abs(dq), G[2])
        for i in range(3):
            ab = np.abs if i else (lambda z: z)
            sc = abs(scale) if i else scale
            r[i]["dq"][:, t] = sc * (states[t + 1][i] * ab(dout[:, t, :, :, None])).sum(2)
            r[i]["dk"][:, t] = (G[i] * ab(v[:, t, :, :, None])).sum(2)
            r[i]["dv"][:, t] = (G[i] * ab(fk[:, t, :, None, :])).sum(3)
        old = states[t]
        r[0]["dg"][:, t] = (a[:, t] * G[0] * old[0]).sum((2, 3))
        G = (a[:, t] * G[0], a[:, t] * G[1], a[:, t] * (G[2] + x[:, t] * G[1]))
    for i in range(3):
        r[i]["ds0"] = G[i]
        for n, z in (("dq", fq), ("dk", fk)):
            r[i]["e" + n] = (np.abs(z) * r[i][n]).sum(-1) if i else None
            r[i][n] = r[i][n].reshape(B, T, Hk, H // Hk, Dk).sum(3)
    return r


def la_depth(T, Dk, Dv):
    """Roundings on the longest chain: the contractions over Dk (or Dv) and over a
    chunk, a sum over all tokens and a few per factor; the matrix cores may truncate
    where the vector ALU rounds."""
    return 2 * (T + Dk + Dv + 64)


def la_bound(value, major, moment, T, Dk, Dv, out="f32", heads=1):
    b = U * ((la_depth(T, Dk, Dv) + heads) * major + 8 * moment) + TINY
    return b + HALF[out] * (np.abs(value) + b)


def la_dg_bound(r, T, Dk, Dv):
    """dg_t is a sum over the tokens from t on of q . dq - k . dk in 64 bits, each with
    the errors of dq and dk and of its own products, and a product of states at a
    later token, whose majorant that of the whole sum covers."""
    c = la_depth(T, Dk, Dv) + 2 * Dk + 16
    e = U * (c * (r[1]["edq"] + r[1]["edk"]) + 8 * (r[2]["edq"] + r[2]["edk"])) + TINY
    return 2 * np.flip(np.cumsum(np.flip(e, 1), 1), 1)


# ---- rotary positions ----------------------------------------------------------------


def rotary(x, pos, freqs, inter, scale, inverse):
    """(value, majorant): x [..., T, H, D], pos [..., T]"""
    ang = pos.astype(np.float64)[..., None, None] * freqs
    c, s = scale * np.cos(ang), scale * np.sin(ang) * (-1 if inverse else 1)
    n = len(freqs)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + n)
    y, m = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    pair = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    m[..., a] = m[..., b] = pair
    return y, m


def rotary_bound(y, m, out, far=0.0):
    """Sine and cosine within 2^-22 (reduction in 64 bits: far 2^-52 more), the two
    products, their sum and the factor: 4 roundings of each."""
    b = (2.0 ** -22 + far * 2.0 ** -50 + 4 * U) * m
    return b + HALF[out] * (np.abs(y) + b)


# ---- RMS norm --------------------------------------------------------------------------


def rms_fwd(h, w, eps):
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h * r * (1.0 if w is None else w)


def rms_fwd_bound(h, w, eps, out="f32"):
    """The sum of squares errs relatively by its depth (no cancellation), the root by
    half of that, and 6 roundings follow."""
    y = np.abs(rms_fwd(h, w, eps))
    e = (0.5 * (norm_depth(h.shape[-1]) + 2) + 8) * U * y
    return e + HALF[out] * (y + e)


def rms_bwd(x, w, dy, eps, dres):
    """Values and bounds of (dx, dw)."""
    R, C = x.shape
    d = norm_depth(C)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, dn = x * r, dy * (1.0 if w is None else w)
    m2 = (dn * n).mean(-1, keepdims=True)
    dx = r * (dn - n * m2) + (0.0 if dres is None else dres)
    er = (0.5 * (d + 2) + 6) * U
    am2 = (np.abs(dn) * np.abs(n)).mean(-1, keepdims=True)
    mag = np.abs(dn) + np.abs(n) * am2
    edx = r * ((3 * er + 8 * U) * mag + (d + 6) * U * np.abs(n) * am2) * 1.05
    if dres is not None:
        edx = edx + 2 * U * (np.abs(dres) + r * mag)
    dw = (dy * n).sum(0)
    ew = ((er + 2 * U) + (R + 4) * U) * np.abs(dy * n).sum(0) * 1.05
    return [dx, dw], [edx, ew]
