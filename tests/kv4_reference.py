"""Plain 64-bit forms of the 4-bit cache, the norm and rotation of rows, and
decode attention, for the tests (numpy and torch on the CPU; none of the
library's code)."""
import math

import numpy as np
import torch

D = 128
U32 = 2.0 ** -24                      # half a step of float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def place(values):
    """(byte, shift) of every channel within a row of 64 bytes, from the format's description."""
    byte, shift = np.zeros(D, np.int64), np.zeros(D, np.int64)
    for c in range(D):
        j, r = divmod(c, 32)
        if values:
            g, r = divmod(r, 4)
            i, h = divmod(r, 2)
            byte[c] = 8 * g + 2 * j + i
        else:
            t, r = divmod(r, 8)
            h, i = divmod(r, 4)
            byte[c] = 16 * t + 4 * j + i
        shift[c] = 4 * h
    return byte, shift


def rows_padded(n_max):
    return -(-n_max // 16) * 16


def split(buf, B, H, n_max, group):
    """(codes [B][H][R][64] uint8, params [B][H][R][D/group][2] float64: scale, middle) of a cache buffer."""
    R = rows_padded(n_max)
    raw = buf.cpu().numpy() if hasattr(buf, "cpu") else buf
    cut = B * H * R * 64
    params = raw[cut:cut + B * H * R * (D // group) * 4].view(np.uint16).astype(np.uint32) << 16
    return raw[:cut].reshape(B, H, R, 64), params.view(np.float32).astype(np.float64).reshape(B, H, R, D // group, 2)


def codes(byte_rows, values):
    b, s = place(values)
    c = (byte_rows[..., b].astype(np.int64) >> s) & 15
    return np.where(c > 7, c - 16, c)


def values_of(buf, B, H, n_max, group, values):
    by, pa = split(buf, B, H, n_max, group)
    c = codes(by, values).reshape(B, H, -1, D // group, group)
    return (pa[..., 1:] + pa[..., :1] * c).reshape(B, H, -1, D)


def to_bf16(x):
    """float32 array rounded to nearest even bfloat16, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def quantise(x, group):
    """(codes, scale, middle) in float64 of float32 rows [..., 128], by the format's formulas."""
    g = x.astype(np.float64).reshape(*x.shape[:-1], D // group, group)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0, g)
    lo, hi = g.min(-1), g.max(-1)
    need = hi - lo
    # all candidates around need / 15: the bfloat16 below and the next two up
    base = (need / 15).astype(np.float32).view(np.uint32) & np.uint32(0xffff0000)
    scale = np.full(need.shape, np.nan)
    for step in (2, 1, 0, -1):
        bits = base.astype(np.int64) + step * 0x10000
        cand = np.where(bits >= 0, bits, 0).astype(np.uint32).view(np.float32).astype(np.float64)
        scale = np.where(15 * cand >= need, cand, scale)
    assert np.isfinite(scale).all()
    middle = to_bf16((lo + 8 * scale).astype(np.float32)).astype(np.float64)
    q = (g - middle[..., None]) / np.where(scale > 0, scale, 1)[..., None]
    c = np.clip(np.rint(q), -8, 7) * (scale > 0)[..., None]
    c[bad], scale[bad], middle[bad] = 0, 0, np.nan
    return c.astype(np.int64).reshape(x.shape), scale, middle


def pack(c, values):
    b, s = place(values)
    out = np.zeros(c.shape[:-1] + (64,), np.uint8)
    for ch in range(D):
        out[..., b[ch]] |= ((c[..., ch] & 15) << s[ch]).astype(np.uint8)
    return out


def cache_of(rows, group, values, n_max):
    """A cache buffer (torch uint8, CPU) that holds float32 rows [B][H][n][128] quantised; the rows behind them are NaN."""
    B, H, n, _ = rows.shape
    R = rows_padded(n_max)
    c, scale, middle = quantise(rows, group)
    by = np.full((B, H, R, 64), 0x5a, np.uint8)
    by[:, :, :n] = pack(c, values)
    pa = np.full((B, H, R, D // group, 2), 0x7fc1, np.uint16)            # NaN scale and middle
    bits = lambda a: (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    pa[:, :, :n, :, 0], pa[:, :, :n, :, 1] = bits(scale), bits(middle)
    return torch.from_numpy(np.concatenate([by.reshape(-1), pa.reshape(-1).view(np.uint8)]))


def rotated(x, pos, weight, eps, inv_freq, interleaved, rot_scale):
    """Rows [B][T][H][128] normalised and rotated in 64 bits, and a bound of the 32-bit error of each channel.

    Counting half steps of float32 (u = 2^-24): the sum of squares is off by at most 9 u relative (a product, 3 + 5 sums),
    its root by half of that, rsqrtf by 2 steps (4 u), eps by u / 2, the two products by 2 u: 11 u.  A rotated channel is
    two products of that with a cosine or sine rounded once (2 u each), and one sum (u): 14 u of |a| + |b|."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    z, bound = y.copy(), 11 * U32 * np.abs(y)
    rot = 2 * len(inv_freq)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = (pos.astype(np.float64) * inv_freq[i])[..., None]
        z[..., a] = rot_scale * (y[..., a] * np.cos(ang) - y[..., b] * np.sin(ang))
        z[..., b] = rot_scale * (y[..., b] * np.cos(ang) + y[..., a] * np.sin(ang))
        bound[..., a] = bound[..., b] = 15 * U32 * abs(rot_scale) * (np.abs(y[..., a]) + np.abs(y[..., b]))
    return z, bound


def parts_of(buf, B, H, n_max, group, values):
    """|middle| + |scale code| of a cache's values: what their two terms can add up to before they cancel."""
    by, pa = split(buf, B, H, n_max, group)
    c = codes(by, values).reshape(B, H, -1, D // group, group)
    return (np.abs(pa[..., 1:]) + np.abs(pa[..., :1] * c)).reshape(B, H, -1, D)


def attend(q, K, V, rows, Kparts=None, Vparts=None):
    """q [heads][128], K and V [R][128] (float64), rows: positions, each as often as listed; Kparts and Vparts: parts_of K and V
    (twice their largest channels where these are not given).

    Returns (out, lse, bound of out, bound of lse).  The bounds count what 32 bits can lose.  A logit is summed from at
    most 4 group terms and 4 middle terms, each rounded a few times: 16 u of sum |q| (|middle| + |scale code|); its queries
    are 28-bit fixed point: 2^-27 of the largest |q| times the sum of those.  A weight is off relatively by twice the largest logit error, by u |z - m| from the
    rounded exponent, and by 2^-20 from the exponential, the product with a scale and its split into two parts.
    Sums of n terms run in 8 chains and a tree: (n / 8 + 64) u."""
    if not len(rows):
        return np.zeros((len(q), D)), np.full(len(q), -math.inf), np.zeros((len(q), D)), np.zeros(len(q))
    k, v = K[rows], V[rows]
    z = q @ k.T / math.sqrt(D)
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    total = p.sum(-1, keepdims=True)
    out = p @ v / total
    lse = (m + np.log(total))[:, 0]
    kp = 2 * np.abs(k).max(-1, keepdims=True) + 0 * k if Kparts is None else Kparts[rows]
    vp = 2 * np.abs(v).max(-1, keepdims=True) + 0 * v if Vparts is None else Vparts[rows]
    zerr = (16 * U32 * (np.abs(q) @ kp.T) + 2.0 ** -27 * np.abs(q).max(-1)[:, None] * kp.sum(-1)) / math.sqrt(D)
    zerr = zerr.max(-1, keepdims=True) + 4 * U32 * np.abs(z).max(-1, keepdims=True)
    rel = 2 * zerr + 2 * U32 * (m - z).clip(max=60) + 2.0 ** -20 + (len(rows) / 8 + 64) * U32
    w = p / total * rel
    err = w @ vp + np.abs(out) * w.sum(-1, keepdims=True) + 2.0 ** -100
    return out, lse, err, (w.sum(-1) + zerr[:, 0]) + 2 * U32 * np.abs(lse)
