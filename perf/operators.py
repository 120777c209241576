"""Cases of the operators around the decode step: the pass that normalises and
rotates queries and keys into the caches, the cache held in 4 bits (written and
read back), and decode attention over that cache, dense and over chosen rows.

`run` computes them in elementary torch operations, or through the library's
entry points where `own` is true; `exact` computes them from their definitions
in 64 bits.

The 4-bit cache of K (or V) is one byte buffer: codes [B][H_kv][R][64], then
(scale, middle) pairs of bfloat16 [B][H_kv][R][128 / group], with R = n_max
rounded up to 16.  A channel's value is middle + scale * code, code in
[-8, 7] as a two's complement nibble; the byte orders of K and V rows are
those of `_pack`.
"""
import math

import torch

own = False

D = 128
SINKS = 4
THETA = 1000000.0
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of four sequences: the call before every decode step of the 8B shape
        dict(name="rope decode b4", op="rope", dtype="bf16", batch=4, tokens=1, q_heads=32, kv_heads=8, n_max=2048,
             norm=True, rot_dim=128, interleaved=False, padded=False, group=0),
        # a whole 16K prompt, queries laid out by head for the prefill graph
        dict(name="rope prompt 16k", op="rope", dtype="bf16", batch=1, tokens=16384, q_heads=32, kv_heads=8,
             n_max=16384, norm=True, rot_dim=128, interleaved=False, padded=False, group=0),
        # float32, no norms, half the channels rotated in adjacent pairs, ragged prompts padded on the right
        dict(name="rope f32 ragged", op="rope", dtype="f32", batch=3, tokens=777, q_heads=8, kv_heads=2, n_max=1000,
             norm=False, rot_dim=64, interleaved=True, padded=True, group=0),
        # prompts straight into the 4-bit cache, and the rows read back
        dict(name="rope to 4 bits", op="rope", dtype="bf16", batch=2, tokens=1000, q_heads=32, kv_heads=8, n_max=1024,
             norm=True, rot_dim=128, interleaved=False, padded=True, group=64),
        # a 16K prompt's keys and values into the 4-bit cache and back
        dict(name="kv4 prompt 16k", op="kv4", dtype="bf16", batch=1, tokens=16384, kv_heads=8, n_max=16384, padded=False,
             group=32),
        # float32 rows, ragged prompts of odd length
        dict(name="kv4 f32 ragged", op="kv4", dtype="f32", batch=3, tokens=1009, kv_heads=2, n_max=1031, padded=True,
             group=128),
        # one short sequence: latency
        dict(name="dense short", op="attend", dtype="bf16", batch=1, q_heads=8, kv_heads=2, n_max=512, n=301, group=32,
             ragged=False, rows=0, per_head=False),
        # the 8B shape at 128K, batch 4: the throughput workload
        dict(name="dense 128k b4", op="attend", dtype="bf16", batch=4, q_heads=32, kv_heads=8, n_max=131200, n=131072,
             group=32, ragged=False, rows=0, per_head=False),
        # a batch of 16 sequences of every length from none to 32K
        dict(name="dense ragged b16", op="attend", dtype="bf16", batch=16, q_heads=32, kv_heads=8, n_max=32800, n=32768,
             group=64, ragged=True, rows=0, per_head=False),
        # float32 queries, eight of them to a KV head
        dict(name="dense f32 group 8", op="attend", dtype="f32", batch=2, q_heads=16, kv_heads=2, n_max=8200, n=8191,
             group=128, ragged=False, rows=0, per_head=False),
        # the rows that a 4096-token budget keeps of 128K
        dict(name="rows 4096 of 128k", op="attend", dtype="bf16", batch=4, q_heads=32, kv_heads=8, n_max=131200,
             n=131072, group=32, ragged=False, rows=4096, per_head=False),
        # a row list for each query head, 256 rows of a short context
        dict(name="rows 256 per head", op="attend", dtype="f32", batch=1, q_heads=8, kv_heads=2, n_max=2064, n=2049,
             group=64, ragged=False, rows=256, per_head=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "kv4", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 8])
    batch = _spread(rng, 1, 16)
    if op != "attend":
        q_heads = kv_heads * rng.choice([1, 2, 4])
        tokens = _spread(rng, 1, max(1, min(16384, 16384 * 8 // (batch * kv_heads * (1 if dtype == "bf16" else 2)))))
        case = dict(op=op, dtype=dtype, batch=batch, tokens=tokens, kv_heads=kv_heads, n_max=tokens + rng.randrange(100),
                    padded=rng.random() < 0.5, group=rng.choice([32, 64, 128]))
        if op == "rope":
            case.update(q_heads=q_heads, norm=rng.random() < 0.7, rot_dim=rng.choice([32, 64, 128, 128]),
                        interleaved=rng.random() < 0.3, group=rng.choice([0, 0, case["group"]]))
        return case
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    per_head = rng.random() < 0.25
    rows = rng.choice([0, 0, _spread(rng, 1, 4096)])
    if rows:
        q_heads = kv_heads * rng.choice([1, 2, 4, 8])
    n = _spread(rng, max(1, rows + SINKS + 1 if rows else 1), min(131072, 131072 * 32 // (batch * kv_heads)))
    return dict(op="attend", dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads, n_max=n + rng.randrange(64), n=n,
                group=rng.choice([32, 64, 128]), ragged=not rows and rng.random() < 0.5, rows=rows,
                per_head=bool(rows) and per_head)


def _units(case):
    return case["batch"] * (case["q_heads"] if case["per_head"] else case["kv_heads"])


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    B, Hkv = case["batch"], case["kv_heads"]
    row4 = 64 + 512 // case["group"] if case["group"] else 0
    if case["op"] == "attend":
        if case["rows"]:
            read = _units(case) * (case["rows"] * 4 + (case["rows"] + SINKS + 1) * 2 * row4)
            pairs = (case["rows"] + SINKS + 1) * B * case["q_heads"]
        else:
            total = sum(_lengths(case))
            read = total * Hkv * 2 * row4
            pairs = total * case["q_heads"]
        return {"bytes": read + B * case["q_heads"] * (D * (esz + 4) + 4), "flops": 4 * D * pairs}
    tokens = B * case["tokens"]
    kv = 2 * tokens * Hkv
    if case["op"] == "kv4":
        return {"bytes": kv * (2 * D * esz + row4) + 4 * tokens, "flops": 8 * kv * D}
    q = tokens * case["q_heads"]
    stored = row4 + D * esz if case["group"] else D * esz      # read back where the cache is 4-bit
    return {"bytes": q * 2 * D * esz + kv * (D * esz + stored) + 4 * tokens, "flops": 10 * (q + kv) * D}


def _lengths(case):
    """The sequences' lengths, in an order of their own: from none to n."""
    B, n = case["batch"], case["n"]
    if not case["ragged"]:
        return [n] * B
    return [n] if B == 1 else [n * b // (B - 1) for b in range(B)]


# -------------------------------------------------------- the 4-bit format
def _pack(code, values):
    """Codes [..., 128] in [-8, 7] as 64 bytes: K rows in the order (t, j, i) of channel 32 j + 8 t + 4 h + i, V rows in the
    order (g, j, i) of channel 32 j + 4 g + 2 i + h; h = 0 is the low nibble."""
    lead = code.shape[:-1]
    c = code.to(torch.int32) & 15
    if values:
        c = c.reshape(*lead, 4, 8, 2, 2).transpose(-4, -3)                # j g i h -> g j i h
    else:
        c = c.reshape(*lead, 4, 4, 2, 4).transpose(-2, -1).transpose(-4, -3)   # j t h i -> t j i h
    return (c[..., 0] | c[..., 1] << 4).reshape(*lead, 64).to(torch.uint8)


def _unpack(byte, values):
    lead = byte.shape[:-1]
    b = byte.to(torch.int16)
    c = torch.stack([b & 15, b >> 4], -1)
    c = ((c ^ 8) - 8).to(torch.int8)
    if values:
        c = c.reshape(*lead, 8, 4, 2, 2).transpose(-4, -3)
    else:
        c = c.reshape(*lead, 4, 4, 4, 2).transpose(-4, -3).transpose(-2, -1)
    return c.reshape(*lead, D)


def _quantise(x, group):
    """Codes, scales and middles (float64) of rows [..., 128]; the decisions next to a border are taken in 64 bits."""
    g = x.double().reshape(*x.shape[:-1], D // group, group)
    lo, hi = g.amin(-1), g.amax(-1)
    least = (hi - lo) / 15
    scale = least.to(torch.bfloat16)
    up = (scale.view(torch.int16) + 1).view(torch.bfloat16)
    scale = torch.where(scale.double() < least, up, scale).double()
    middle = (lo + 8 * scale).to(torch.bfloat16).double()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.round((g - middle[..., None]) / safe[..., None]).clamp(-8, 7)
    code = torch.where(scale[..., None] > 0, code, torch.zeros_like(code))
    return code.reshape(x.shape), scale, middle


def _stored(x, group):
    """The values that rows [..., 128] have in the 4-bit cache."""
    code, scale, middle = _quantise(x, group)
    value = middle[..., None] + scale[..., None] * code.reshape(*x.shape[:-1], D // group, group)
    return value.reshape(x.shape)


def _padded_rows(n_max):
    return (n_max + 15) // 16 * 16


def _values(buf, B, H, n_max, group, values, at=None):
    """The float32 values [B][H][R][128] of a 4-bit cache, or those of its rows at = (b, h, row)."""
    R = _padded_rows(n_max)
    cut = B * H * R * 64
    byte = buf[:cut].reshape(B, H, R, 64)
    params = buf[cut:].view(torch.bfloat16).reshape(B, H, R, D // group, 1, 2)
    if at is not None:
        byte, params = byte[at], params[at]
    params = params.float()
    code = _unpack(byte, values)
    code = code.reshape(*code.shape[:-1], D // group, group).float()
    return torch.addcmul(params[..., 1], params[..., 0], code).flatten(-2)


def _filled(B, H, n_max, group, values, gen):
    """A 4-bit cache of unit normal rows; four channels of the keys are eight times as large."""
    R = _padded_rows(n_max)
    codes = torch.empty((B, H, R, 64), dtype=torch.uint8, device="cuda")
    params = torch.empty((B, H, R, D // group, 2), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        x = torch.randn((H, R, D), generator=gen, device="cuda")
        if not values:
            x[..., 5::32] *= 8
        g = x.reshape(H, R, D // group, group)
        lo, hi = g.amin(-1), g.amax(-1)
        scale = ((hi - lo) / 15 * 1.005).to(torch.bfloat16).float()
        middle = (lo + 8 * scale).to(torch.bfloat16).float()
        code = torch.round((g - middle[..., None]) / scale[..., None]).clamp(-8, 7).reshape(H, R, D)
        codes[b] = _pack(code, values)
        params[b, ..., 0], params[b, ..., 1] = scale, middle
    return torch.cat([codes.reshape(-1), params.reshape(-1).view(torch.uint8)])


# -------------------------------------------------------------- the inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, B, Hkv, n_max = _dtype(case), case["batch"], case["kv_heads"], case["n_max"]
    s = dict(case)
    if case["op"] == "attend":
        Hq, n, group = case["q_heads"], case["n"], case["group"]
        s["q"] = torch.randn((B, Hq, D), generator=gen, device="cuda").to(dt)
        s["K4"] = _filled(B, Hkv, n_max, group, False, gen)
        s["V4"] = _filled(B, Hkv, n_max, group, True, gen)
        order = torch.randperm(B, generator=gen, device="cuda")
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order].contiguous()
        if case["rows"]:
            U, T = _units(case), case["rows"]
            # random positions after the sinks, none twice; the last tenth of the lists is partly empty (-1)
            pick = torch.rand((U, n - 1 - SINKS), generator=gen, device="cuda").argsort(1)[:, :T].sort(1).values + SINKS
            s["n_rows"] = T - (torch.rand(U, generator=gen, device="cuda") * (T / 10)).to(torch.int32)
            keep = torch.arange(T, device="cuda")[None] < s["n_rows"][:, None]
            s["rows_list"] = torch.where(keep, pick, torch.full_like(pick, -1)).to(torch.int32).contiguous()
        s["out"] = torch.empty((B, Hq, D), dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
        return s
    T, Hq = case["tokens"], case.get("q_heads", 0)
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=gen, device="cuda")   # a fused projection's output
    qkv[:, :, Hq:Hq + Hkv, 5::32] *= 4
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    # prompts start where the cache is empty, single tokens behind a context; padding is -1
    first = (torch.rand(B, generator=gen, device="cuda") * (n_max - T + 1)).to(torch.int32)
    pos = first[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")[None]
    if case["padded"]:
        length = T - (torch.rand(B, generator=gen, device="cuda") * (T / 2)).to(torch.int32)
        pos = torch.where(torch.arange(T, device="cuda")[None] < length[:, None], pos, torch.full_like(pos, -1))
    s["pos"] = pos.to(torch.int32).contiguous()
    if case["op"] == "rope":
        s["q_out"] = torch.zeros((B, Hq, T, D), dtype=dt, device="cuda")
        s["q_weight"], s["k_weight"] = ((1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt) for _ in range(2))
        rot = case["rot_dim"]
        s["inv_freq"] = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    s["K"] = torch.zeros((B, Hkv, n_max, D), dtype=dt, device="cuda")
    s["V"] = torch.zeros_like(s["K"])
    if case["group"]:
        size = B * Hkv * _padded_rows(n_max) * (64 + 512 // case["group"])
        s["K4"], s["V4"] = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    return s


# --------------------------------------------------------- the plain forms
def _rotated(x, weight, s, angle):
    """Rows [B][T][H][128] in 32 bits, normalised and rotated; angle [B][T][rot / 2] in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = s["rot_dim"]
    turn = angle[:, :, None]
    cos, sin = turn.cos().float(), turn.sin().float()
    part = x[..., :rot]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([part, x[..., rot:]], -1)


def _put(cache, rows, pos):
    """rows [B][T][H][128] at the positions pos [B][T] of cache [B][H][n_max][128]; a negative position puts nothing."""
    b, t = (pos >= 0).nonzero(as_tuple=True)
    cache[b, :, pos[b, t].long()] = rows[b, t].to(cache.dtype)


def _plain_rope(s):
    norm = s["norm"]
    angle = s["pos"].double()[..., None] * s["inv_freq"].cuda()
    q = _rotated(s["q"], s["q_weight"] if norm else None, s, angle).to(s["q"].dtype)
    k = _rotated(s["k"], s["k_weight"] if norm else None, s, angle).to(s["q"].dtype)
    held = (s["pos"] >= 0)[:, None, :, None]
    s["q_out"] = torch.where(held, q.transpose(1, 2), s["q_out"])
    v = s["v"]
    if s["group"]:
        k, v = _stored(k, s["group"]), _stored(v, s["group"])
    _put(s["K"], k, s["pos"])
    _put(s["V"], v, s["pos"])
    return s["q_out"], s["K"], s["V"]


def _plain_kv4(s):
    _put(s["K"], _stored(s["k"], s["group"]), s["pos"])
    _put(s["V"], _stored(s["v"], s["group"]), s["pos"])
    return s["K"], s["V"]


def _softmax_sum(z, valid, V):
    """softmax(z) V over the last axis where valid, and the log of the sum; rows with nothing valid give 0 and -inf."""
    z = z.masked_fill(~valid, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isfinite(m), m, torch.zeros_like(m))).masked_fill(~valid, 0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, V) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (m + torch.log(total)).squeeze(-1)


def _plain_attend(s):
    B, Hq, Hkv, n = s["batch"], s["q_heads"], s["kv_heads"], s["n"]
    cache = (B, Hkv, s["n_max"], s["group"])
    q = s["q"].float()
    lens = s["lens"].long()
    if not s["rows"]:
        K, V = _values(s["K4"], *cache, False)[:, :, :n], _values(s["V4"], *cache, True)[:, :, :n]
        z = torch.matmul(q.reshape(B, Hkv, Hq // Hkv, D), K.transpose(-1, -2)) * D ** -0.5
        valid = (torch.arange(n, device=q.device) < lens[:, None])[:, None, None]
        out, lse = _softmax_sum(z, valid, V)
        return out.reshape(B, Hq, D), lse.reshape(B, Hq)
    U = _units(s)
    H = U // B                                                     # row lists of a sequence
    rows = s["rows_list"].long().reshape(B, H, -1)
    valid = rows >= 0
    ends = torch.arange(SINKS, device=q.device).expand(B, H, SINKS)
    rows = torch.cat([ends, rows.clamp(min=0), (lens - 1)[:, None, None].expand(B, H, 1)], -1)
    valid = torch.cat([torch.ones_like(ends, dtype=torch.bool), valid, torch.ones((B, H, 1), dtype=torch.bool, device=q.device)], -1)
    b = torch.arange(B, device=q.device)[:, None, None]
    h = (torch.arange(H, device=q.device) // (H // Hkv))[None, :, None]
    K, V = _values(s["K4"], *cache, False, (b, h, rows)), _values(s["V4"], *cache, True, (b, h, rows))
    z = torch.matmul(q.reshape(B, H, Hq // H, D), K.transpose(-1, -2)) * D ** -0.5
    out, lse = _softmax_sum(z, valid[:, :, None], V)
    return out.reshape(B, Hq, D), lse.reshape(B, Hq)


# ------------------------------------------------------------- one pass
def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "kv4": _plain_kv4, "attend": _plain_attend}[state["op"]](state)


def _own(s):
    import long_context_decode_ckv_b200 as ckv
    if "cfg" not in s:                                             # what a program sets up once for its shapes
        cfg = ckv.ckv_config()
        cfg.batch, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim = s["batch"], s.get("q_heads") or s["kv_heads"], s["kv_heads"], D
        cfg.n_max, cfg.n_sinks = s["n_max"], SINKS
        cfg.kv_dtype = ckv.CKV_BF16 if s["dtype"] == "bf16" else ckv.CKV_F32
        cfg.mode = ckv.CKV_PER_HEAD if s.get("per_head") else ckv.CKV_QUERY_GROUP
        cfg.device = s["q"].device.index
        s["cfg"] = cfg
        if s["op"] == "attend":
            s["workspace"] = torch.zeros(ckv.ckv_kv4_workspace(cfg), dtype=torch.uint8, device="cuda")
    cfg, stream = s["cfg"], torch.cuda.current_stream()
    if s["op"] == "attend":
        lens = s["lens"] if s["ragged"] else None
        if s["rows"]:
            ckv.ckv_kv4_attend_rows(cfg, s["group"], s["q"], s["K4"], s["V4"], s["n"], lens, s["rows_list"], s["n_rows"],
                                    s["rows"], s["workspace"], s["out"], s["lse"], stream)
        else:
            ckv.ckv_kv4_dense_decode(cfg, s["group"], s["q"], s["K4"], s["V4"], s["n"], lens, s["workspace"], s["out"],
                                     s["lse"], stream)
        return s["out"], s["lse"]
    if s["op"] == "rope":
        norm, group = s["norm"], s["group"]
        ckv.ckv_qk_norm_rope(cfg, s["q"], s["k"], s["v"], s["pos"], s["q_out"].transpose(1, 2), s["inv_freq"],
                             q_weight=s["q_weight"] if norm else None, k_weight=s["k_weight"] if norm else None, eps=EPS,
                             interleaved=s["interleaved"], K=None if group else s["K"], V=None if group else s["V"],
                             K4=s["K4"] if group else None, V4=s["V4"] if group else None, group=group, stream=stream)
        if group:
            ckv.ckv_kv4_read(cfg, group, s["K4"], s["V4"], 0, s["n_max"], s["K"], s["V"], stream)
        return s["q_out"], s["K"], s["V"]
    ckv.ckv_kv4_write(cfg, s["group"], s["k"], s["v"], s["pos"], s["K4"], s["V4"], stream)
    ckv.ckv_kv4_read(cfg, s["group"], s["K4"], s["V4"], 0, s["n_max"], s["K"], s["V"], stream)
    return s["K"], s["V"]


# ------------------------------------------------- definitions in 64 bits
def _exact_row4(x, group):
    """Rows [..., 128] (float64) through the 4-bit format, by its definition."""
    parts = []
    for c0 in range(0, D, group):
        g = x[..., c0:c0 + group]
        lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
        # the bfloat16 numbers next to (hi - lo) / 15, and the smaller one that is large enough
        want = (hi - lo) / 15
        e = torch.floor(torch.log2(torch.where(want > 0, want, torch.ones_like(want))))
        step = torch.exp2(e - 7)
        scale = torch.ceil(want / step) * step
        middle = (lo + 8 * scale).to(torch.bfloat16).double()
        q = (g - middle) / torch.where(scale > 0, scale, torch.ones_like(scale))
        below = torch.floor(q)
        code = below + (q - below > 0.5).double() + ((q - below == 0.5) & (below % 2 != 0)).double()
        code = code.clamp(-8, 7) * (scale > 0)
        parts.append(middle + scale * code)
    return torch.cat(parts, -1)


def _exact_rotated(x, weight, s):
    y = x.double().clone()
    if weight is not None:
        y = y / ((y * y).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    z = y.clone()
    rot = s["rot_dim"]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + rot // 2)
        turn = (s["pos"].double() * float(s["inv_freq"][i]))[..., None]
        z[..., a] = y[..., a] * turn.cos() - y[..., b] * turn.sin()
        z[..., b] = y[..., b] * turn.cos() + y[..., a] * turn.sin()
    return z


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv = case["batch"], case["kv_heads"]
    if case["op"] != "attend":
        K, V = s["K"].double(), s["V"].double()
        held = s["pos"] >= 0
        k, v, result = s["k"].double(), s["v"].double(), []
        if case["op"] == "rope":
            q = _exact_rotated(s["q"], s["q_weight"] if case["norm"] else None, s)
            k = _exact_rotated(s["k"], s["k_weight"] if case["norm"] else None, s)
            result.append(torch.where(held[:, :, None, None], q, torch.zeros_like(q)).permute(0, 2, 1, 3))
        if case["group"]:
            k = _exact_row4(k.to(s["K"].dtype).double(), case["group"])   # rows enter the cache in the inputs' type
            v = _exact_row4(v, case["group"])
        for b in range(B):
            t = held[b].nonzero()[:, 0]
            K[b, :, s["pos"][b, t].long()] = k[b, t].transpose(0, 1)
            V[b, :, s["pos"][b, t].long()] = v[b, t].transpose(0, 1)
        return (*result, K, V)
    Hq, n, group, R = case["q_heads"], case["n"], case["group"], _padded_rows(case["n_max"])
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    c = torch.arange(D, device="cuda")
    j = c // 32
    place = {"K4": (16 * (c % 32 // 8) + 4 * j + c % 4, c % 8 // 4), "V4": (8 * (c % 32 // 4) + 2 * j + c % 4 // 2, c % 2)}

    def rows_of(name, b, h, rows):
        byte, high = place[name]
        unit = b * Hkv + h
        code = s[name][:B * Hkv * R * 64].view(B * Hkv, R, 64)[unit][rows][:, byte].long() >> (4 * high) & 15
        code = torch.where(code > 7, code - 16, code).double()
        params = s[name][B * Hkv * R * 64:].view(torch.bfloat16).view(B * Hkv, R, D // group, 2)[unit][rows].double()
        return params[:, c // group, 1] + params[:, c // group, 0] * code

    lists = _units(case) // B
    for b in range(B):
        length = int(s["lens"][b])
        for u in range(lists if case["rows"] else Hkv):
            heads = range(u * Hq // lists, (u + 1) * Hq // lists) if case["rows"] else range(u * Hq // Hkv, (u + 1) * Hq // Hkv)
            if case["rows"]:
                listed_rows = s["rows_list"][b * lists + u, :int(s["n_rows"][b * lists + u])].long()
                rows = torch.cat([torch.arange(SINKS, device="cuda"), listed_rows, torch.tensor([length - 1], device="cuda")])
            else:
                rows = torch.arange(length, device="cuda")
            if not len(rows):
                continue
            kv = heads[0] * Hkv // Hq
            k, v = rows_of("K4", b, kv, rows), rows_of("V4", b, kv, rows)
            z = s["q"][b, heads[0]:heads[-1] + 1].double() @ k.T / math.sqrt(D)
            lse[b, heads[0]:heads[-1] + 1] = torch.logsumexp(z, -1)
            out[b, heads[0]:heads[-1] + 1] = torch.softmax(z, -1) @ v
    return out, lse
