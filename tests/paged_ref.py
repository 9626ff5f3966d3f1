"""Plain 64-bit forms of the rotary tables, the per-head norms with rotation,
the 4-bit pages and paged attention, for the parity tests."""

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
HALF_BF16 = 2.0 ** -8   # half a step, relative to the value
F32 = 2.0 ** -24


def e4m3_values():
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return v


E4M3 = e4m3_values()


def table(M, rot, P, theta, scaling, factor=1.0, orig=8192.0, low=1.0, high=32.0, amp=1.0):
    """(values [M, rot], angles [M, rot/2])"""
    i = np.arange(rot // 2, dtype=np.float64)
    f = np.exp(-np.log(theta) * 2 * i / rot)
    if scaling == 1:
        f = f / factor
    if scaling == 2:
        f = np.exp(-(np.log(theta) + np.log(factor) * rot / (rot - 2)) * 2 * i / rot)
    if scaling == 3:
        keep = np.clip((orig * f / (2 * np.pi) - low) / (high - low), 0, 1)
        f = f * keep + f / factor * (1 - keep)
    a = (P + np.arange(M, dtype=np.float64))[:, None] * f
    out = np.empty((M, rot))
    out[:, 0::2], out[:, 1::2] = amp * np.cos(a), amp * np.sin(a)
    return out, a


def norm_rotate(x, w, eps, tab, pos, rot, half):
    """x [rows, heads, hd] -> (values, the size of what each was summed from)."""
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w
    if rot == 0:
        return x, np.abs(x)
    cs = tab.astype(np.float64)[pos][:, None, :]
    c, s = cs[..., 0::2], cs[..., 1::2]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    y, size = x.copy(), np.abs(x)
    u, v = a * c - b * s, a * s + b * c
    su, sv = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    if half:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, v
        size[..., :rot // 2], size[..., rot // 2:rot] = su, sv
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, v
        size[..., 0:rot:2], size[..., 1:rot:2] = su, sv
    return y, size


def quantise(x, static):
    """x [..., hd] fp32 (bf16 values) -> (codes [..., hd], scale codes [..., hd/16]):
    y = x * fp32(1 / static) in fp32, the rest by exact nearest-even choice."""
    y = (x.astype(np.float32) * np.float32(np.float32(1) / np.float32(static))).astype(np.float64)
    b = y.reshape(y.shape[:-1] + (-1, 16))
    a = np.nanmax(np.where(np.isnan(b), 0, np.abs(b)), -1)
    a6 = (a.astype(np.float32) / np.float32(6)).astype(np.float64)
    fin = E4M3[:127]
    hi = np.clip(np.searchsorted(fin, a6), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = fin[hi] - a6, a6 - fin[lo]
    s8 = np.where(a6 >= 448, 126, np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))))
    s8 = np.where(a6 == 0, 0, s8)
    s = fin[s8][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        t = np.where(s > 0, b / np.where(s > 0, s, 1), 0.0)
    m = np.abs(t)
    c = np.zeros(t.shape, np.int64)
    for border, tie_up in ((.25, 0), (.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5., 0)):
        c += (m >= border) if tie_up else (m > border)
    c += 8 * (np.signbit(t) & (s > 0))
    return c.reshape(x.shape), s8


def pack_codes(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def attention(q, k, v, L, causal, window, scale):
    """One sequence: q [Lq, hq, hd], k and v [hkv, L, hd] in 64 bits ->
    (out [Lq, hq, hd], lse [Lq, hq], bound of |out| error before its own
    rounding, bound of lse error)."""
    Lq, hq, hd = q.shape
    G = hq // k.shape[0]
    out, lse = np.zeros((Lq, hq, hd)), np.full((Lq, hq), -np.inf)
    e_out, e_lse = np.zeros((Lq, hq, hd)), np.zeros((Lq, hq))
    j, p = np.arange(L)[None], (L - Lq + np.arange(Lq))[:, None]
    see = np.ones((Lq, L), bool)
    if causal:
        see &= j <= p
    if window:
        see &= j > p - window
    rows = see.any(1)
    for h in range(hq):
        kk, vv = k[h // G], v[h // G]
        x = np.where(see, q[:, h] @ kk.T * scale, -np.inf)[rows]
        if not len(x):
            continue
        m = x.max(1, keepdims=True)
        w = np.exp(x - m)
        z = w.sum(1, keepdims=True)
        out[rows, h] = (w / z) @ vv
        lse[rows, h] = (m + np.log(z))[:, 0]
        # a score: hd products summed in fp32 (the tensor core truncates:
        # 2^-23 a step), its scaling, the power-of-two fp16 form of q (below
        # 2^-14 of the row's largest it rounds: 2^-25 of it), and the base-2
        # exponential's own 2^-22
        size = (np.abs(q[:, h]) @ np.abs(kk).T * abs(scale))[rows].max(1)
        big = (np.abs(q[:, h]).max(1)[rows] * np.abs(kk).sum(1).max() * abs(scale)) * 2.0 ** -25
        d = (hd + 6) * 2.0 ** -23 * size + big + 2.0 ** -22
        a = (w / z) @ np.abs(vv)
        # the weights' fp16 rounding (2^-11), the sums over the keys
        # (2^-23 a step, a step per 16 keys and one per join)
        e_out[rows, h] = a * (2.0 ** -11 + 2 * d + (L / 16 + 40) * 2.0 ** -23)[:, None]
        # weights below 2^-21 of the largest round by up to 2^-32 of it
        e_out[rows, h] += 2.0 ** -32 * np.abs(vv).sum(0)
        # the output's own rounding is half a step of the computed value v', not
        # of v: |bf16(v') - v| <= e + 2^-8 |v'| <= e (1 + 2^-8) + 2^-8 |v|
        e_out[rows, h] *= 1 + HALF_BF16
        e_lse[rows, h] = d + (L / 16 + 40) * 2.0 ** -23 + np.abs(lse[rows, h]) * 2.0 ** -22
    return out, lse, e_out, e_lse
