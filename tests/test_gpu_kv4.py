"""Rows into the caches and the 4-bit cache on the GPU, against plain 64-bit
forms (kv4_reference.py, which derives the tolerances)."""
import numpy as np
import pytest
import torch

import long_context_decode_ckv_b200 as ckv
from long_context_decode_ckv_b200 import build as ckv_build
from tests import kv4_reference as ref
from tests.conftest import gpu_available
from tests.kv4_reference import D, U32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA device")]

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ckv_build.build()


def config(B, Hq, Hkv, n_max, dtype, sinks=0, per_head=False):
    c = ckv.ckv_config()
    c.batch, c.n_q_heads, c.n_kv_heads, c.head_dim, c.n_max, c.n_sinks = B, Hq, Hkv, D, n_max, sinks
    c.kv_dtype = ckv.CKV_BF16 if dtype == torch.bfloat16 else ckv.CKV_F32
    c.mode = ckv.CKV_PER_HEAD if per_head else ckv.CKV_QUERY_GROUP
    c.device = 0
    return c


def normal(rng, shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape, np.float32)) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


# ---------------------------------------------------------------- the format
def hard_rows(rng, count, dtype):
    """Rows that are hard to quantise: ties, constants, outliers, tiny and huge values, zeros of both signs, every exponent."""
    kinds = []
    for i in range(count):
        k = i % 8
        x = rng.standard_normal(D)
        if k == 1:
            x = rng.integers(-15, 16, D) / 2.0                 # many exact ties
        elif k == 2:
            x = np.full(D, rng.standard_normal())
        elif k == 3:
            x[rng.integers(0, D, 4)] *= 50
        elif k == 4:
            x = x * 2.0 ** rng.integers(-140, -100)            # scales and values down to subnormals
        elif k == 5:
            x = x * 2.0 ** rng.integers(90, 120)
        elif k == 6:
            x = 100.0 + x * 2.0 ** rng.integers(-12, 2)        # far from zero, narrow
        elif k == 7:
            x = np.where(rng.random(D) < 0.5, 0.0, -0.0) if i % 16 == 7 else np.ldexp(x, rng.integers(-30, 30, D))
        kinds.append(x)
    return torch.from_numpy(np.array(kinds, np.float32)).to(dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_codes_and_parameters_are_the_formulas(group, dtype):
    rng = np.random.default_rng(group)
    dt = DTYPES[dtype]
    B, H, T = 2, 3, 200
    c = config(B, H, H, T, dt)
    x = hard_rows(rng, B * T * H, dt).reshape(B, T, H, D).cuda()
    buf = [torch.zeros(ckv.ckv_kv4_bytes(c, group), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ckv.ckv_kv4_write(c, group, x, x, None, *buf)
    want = ref.quantise(f32(x).transpose(0, 2, 1, 3), group)
    for values in (False, True):
        by, pa = ref.split(buf[values], B, H, T, group)
        np.testing.assert_array_equal(pa[:, :, :T, :, 0], want[1])
        np.testing.assert_array_equal(pa[:, :, :T, :, 1], want[2])
        np.testing.assert_array_equal(ref.codes(by[:, :, :T], values), want[0])
        assert not by[:, :, T:].any() and not pa[:, :, T:].any()       # rows behind n_max stay
    back = [torch.empty((B, H, T, D), dtype=dt, device="cuda") for _ in range(2)]
    ckv.ckv_kv4_read(c, group, *buf, 0, T, *back)
    value = torch.from_numpy(want[2][..., None] + want[1][..., None] * want[0].reshape(B, H, T, D // group, group))
    value = value.reshape(B, H, T, D)
    for t in back:
        # the value rounded to float32, then to the cache's type
        assert torch.equal(t.cpu(), value.float().to(dt))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_group_that_is_not_finite_reads_back_as_nan(bad):
    c = config(1, 1, 1, 4, torch.float32)
    x = torch.randn((1, 4, 1, D), device="cuda")
    x[0, 1, 0, 70] = bad
    buf = [torch.zeros(ckv.ckv_kv4_bytes(c, 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ckv.ckv_kv4_write(c, 32, x, x, None, *buf)
    back = [torch.empty((1, 1, 4, D), device="cuda") for _ in range(2)]
    ckv.ckv_kv4_read(c, 32, *buf, 0, 4, *back)
    for t in back:
        nan = torch.isnan(t[0, 0])
        assert nan[1, 64:96].all() and int(nan.sum()) == 32


def test_write_and_read_touch_only_their_rows():
    rng = np.random.default_rng(1)
    B, H, T, n_max, group = 3, 2, 5, 37, 64
    c = config(B, 2 * H, H, n_max, torch.bfloat16)
    fused = normal(rng, (B, T, 4 * H, D), torch.bfloat16)                # k and v within a wider row
    k, v = fused[:, :, H:2 * H], fused[:, :, 3 * H:]
    pos = torch.tensor([[0, 36, 7, -1, 3], [-5, 37, 2 ** 31 - 1, 11, -2 ** 31], [5, 6, 7, 8, 9]], dtype=torch.int32, device="cuda")
    size = ckv.ckv_kv4_bytes(c, group)
    buf = [torch.full((size,), 0xab, dtype=torch.uint8, device="cuda") for _ in range(2)]
    guard = [torch.cat([b, torch.full((4096,), 0xab, dtype=torch.uint8, device="cuda")]) for b in buf]
    ckv.ckv_kv4_write(c, group, k, v, pos, *guard)
    for values, src in ((False, k), (True, v)):
        got = guard[values]
        assert (got[size:] == 0xab).all()
        by, pa = ref.split(got[:size], B, H, n_max, group)
        want_by = np.full_like(by, 0xab)
        want_pa = np.full(pa.shape, np.array([0xabab << 16], np.uint32).view(np.float32)[0], np.float64)
        code, scale, middle = ref.quantise(f32(src), group)
        for b in range(B):
            for t in range(T):
                p = int(pos[b, t])
                if 0 <= p < n_max:
                    want_by[b, :, p] = ref.pack(code[b, t], values)
                    want_pa[b, :, p, :, 0], want_pa[b, :, p, :, 1] = scale[b, t], middle[b, t]
        np.testing.assert_array_equal(by, want_by)
        np.testing.assert_array_equal(pa, want_pa)
    out = [torch.full((B, H, n_max, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ckv.ckv_kv4_read(c, group, *guard, 5, 4, *out)
    ckv.ckv_kv4_read(c, group, guard[0], None, 36, 1, out[0], None)      # one cache alone
    held = torch.zeros(n_max, dtype=torch.bool)
    held[5:9] = True
    assert (out[1][:, :, ~held] == 7.0).all()
    held[36] = True
    assert (out[0][:, :, ~held] == 7.0).all()
    np.testing.assert_array_equal(f64(out[1][2, :, 5:9]),
                                  f64(torch.from_numpy(ref.values_of(guard[1][:size], B, H, n_max, group, True)[2, :, 5:9]).bfloat16()))


# ------------------------------------------------------- norm and rotation
ROPE = [
    # dtype, B, T, Hq, Hkv, rot, interleaved, q norm, k norm, rot_scale
    ("bf16", 1, 1, 1, 1, 128, False, True, True, 1.0),
    ("bf16", 4, 1, 32, 8, 128, False, True, True, 1.0),
    ("f32", 2, 33, 6, 2, 128, False, True, True, 1.25),
    ("f32", 1, 130, 5, 5, 64, True, False, False, 1.0),
    ("bf16", 2, 7, 3, 1, 32, False, True, False, 1.0),
    ("f32", 1, 9, 4, 1, 48, True, False, True, 0.5),
    ("bf16", 3, 500, 8, 2, 112, False, True, True, 1.0),
    ("f32", 1, 3, 2, 1, 16, False, True, True, 1.0),
    ("f32", 1, 17, 1, 1, 0, False, True, True, 1.0),
    ("bf16", 2, 700, 16, 8, 128, True, False, False, 1.0),
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c)))
def test_norm_and_rotation(case):
    dtype, B, T, Hq, Hkv, rot, inter, qn, kn, scale = case
    rng = np.random.default_rng(T + rot)
    dt = DTYPES[dtype]
    n_max = T + 40
    c = config(B, Hq, Hkv, n_max, dt)
    fused = normal(rng, (B, T, Hq + 2 * Hkv, D), dt, 3.0)
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv], fused[:, :, Hq + Hkv:]
    # positions in any order, a few padded
    pos = np.stack([rng.permutation(n_max)[:T] for _ in range(B)]).astype(np.int32)
    pos[rng.random((B, T)) < (0.2 if T > 1 else 0)] = -1
    wq = (1 + 0.2 * normal(rng, (D,), torch.float32)).to(dt) if qn else None
    wk = (1 + 0.2 * normal(rng, (D,), torch.float32)).to(dt) if kn else None
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    out = torch.full((B, Hq, T, D), 5.0, dtype=dt, device="cuda")         # head-major
    K, V = (torch.full((B, Hkv, n_max, D), 5.0, dtype=dt, device="cuda") for _ in range(2))
    dpos = torch.from_numpy(pos).cuda()
    ckv.ckv_qk_norm_rope(c, q, k, v, dpos, out.transpose(1, 2), freq, q_weight=wq, k_weight=wk, eps=1e-5, rot_scale=scale,
                         interleaved=inter, K=K, V=V)
    half = ref.half_step(dt)
    wantK, boundK = np.full(K.shape, 5.0), np.zeros(K.shape)
    wantV = np.full(K.shape, 5.0)
    for x, w, is_q in ((q, wq, True), (k, wk, False)):
        y, bound = ref.rotated(f64(x), pos, None if w is None else f64(w), np.float32(1e-5).astype(np.float64), freq, inter, scale)
        bound = bound + half * (np.abs(y) + bound) + 1e-37
        if is_q:
            y[pos < 0], bound[pos < 0] = 5.0, 0
            err = np.abs(f64(out).transpose(0, 2, 1, 3) - y)
            assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()
        else:
            for b in range(B):
                for t in range(T):
                    if pos[b, t] >= 0:
                        wantK[b, :, pos[b, t]], boundK[b, :, pos[b, t]] = y[b, t], bound[b, t]
                        wantV[b, :, pos[b, t]] = f64(v)[b, t]
    err = np.abs(f64(K) - wantK)
    assert (err <= boundK).all(), (err / np.maximum(boundK, 1e-300)).max()
    np.testing.assert_array_equal(f64(V), wantV)
    # the same through 4-bit caches, alone and beside the others: the rows of K and V, quantised
    for group in (32, 128):
        size = ckv.ckv_kv4_bytes(c, group)
        alone, beside, after = ([torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(3))
        kw = dict(q_weight=wq, k_weight=wk, eps=1e-5, rot_scale=scale, interleaved=inter, group=group)
        ckv.ckv_qk_norm_rope(c, q, k, v, dpos, out.transpose(1, 2), freq, K4=alone[0], V4=alone[1], **kw)
        K2, V2 = K.clone(), V.clone()
        ckv.ckv_qk_norm_rope(c, q, k, v, dpos, out.transpose(1, 2), freq, K=K2, V=V2, K4=beside[0], V4=beside[1], **kw)
        assert torch.equal(K2, K) and torch.equal(V2, V)
        at = [torch.stack([x[b][:, dpos[b].long().clamp(min=0)].transpose(0, 1) for b in range(B)]) for x in (K, V)]
        ckv.ckv_kv4_write(c, group, *at, dpos, *after)
        for i in range(2):
            assert torch.equal(alone[i], after[i]) and torch.equal(beside[i], after[i])


def test_norm_and_rotation_in_place_and_far():
    # q_out is q; positions up to 2 million, where a 32-bit angle is off by 2^-4
    rng = np.random.default_rng(9)
    T, n_max = 50, 1 << 21
    c = config(1, 2, 1, n_max, torch.bfloat16)
    x = normal(rng, (1, T, 4, D), torch.bfloat16)
    q0 = f64(x[:, :, :2])
    pos = np.sort(rng.integers(0, n_max, (1, T)).astype(np.int32))
    pos[0, -1] = n_max - 1
    freq = 1.0e6 ** (-np.arange(0, D, 2) / D)
    K, V = (torch.zeros((1, 1, n_max, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kwant, kb = ref.rotated(f64(x[:, :, 2:3]), pos, None, 0, freq, False, 1.0)
    ckv.ckv_qk_norm_rope(c, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], torch.from_numpy(pos).cuda(), x[:, :, :2], freq, K=K, V=V)
    want, bound = ref.rotated(q0, pos, None, 0, freq, False, 1.0)
    half = 2.0 ** -8
    # the angle itself, pos * f in 64 bits: 2^21 * 2^-52 radians, far below the rest
    assert (np.abs(f64(x[:, :, :2]) - want) <= bound + half * (np.abs(want) + bound)).all()
    got = f64(K[0, 0, torch.from_numpy(pos[0]).long().cuda()])
    assert (np.abs(got - kwant[0, :, 0]) <= kb[0, :, 0] + half * (np.abs(kwant[0, :, 0]) + kb[0, :, 0])).all()


# --------------------------------------------------------------- attention
class Case:
    def __init__(self, rng, B, Hq, Hkv, n_max, n, group, dtype, lens=None, sinks=0, rows=None, n_rows=None, max_rows=0,
                 per_head=False, kscale=1.0, wide=False):
        self.B, self.Hq, self.Hkv, self.n, self.n_max, self.group = B, Hq, Hkv, n, n_max, group
        self.dt = DTYPES[dtype]
        self.cfg = config(B, Hq, Hkv, n_max, self.dt, sinks, per_head)
        held = max([n] if lens is None else [min(max(x, 0), n) for x in lens])
        x = [rng.standard_normal((B, Hkv, held, D)).astype(np.float32) for _ in range(2)]
        x[0][..., 3::40] *= 8
        x[0] *= kscale
        if wide:                                        # groups of very different size beside one another
            x[1] *= 2.0 ** rng.integers(-30, 30, (1, 1, 1, D // 32)).repeat(32, -1).astype(np.float32)
        self.K4, self.V4 = (ref.cache_of(a, group, bool(i), n_max).cuda() for i, a in enumerate(x))
        self.q = normal(rng, (B, Hq, D), self.dt)
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.rows, self.n_rows, self.max_rows = rows, n_rows, max_rows
        self.out = torch.full((B, Hq, D), 9.0, device="cuda")
        self.lse = torch.full((B, Hq), 9.0, device="cuda")
        self.work = torch.zeros(ckv.ckv_kv4_workspace(self.cfg), dtype=torch.uint8, device="cuda")

    def run(self, stream=None, lse=True):
        args = (self.cfg, self.group, self.q, self.K4, self.V4, self.n, self.lens)
        if self.rows is None:
            ckv.ckv_kv4_dense_decode(*args, self.work, self.out, self.lse if lse else None, stream)
        else:
            ckv.ckv_kv4_attend_rows(*args, self.rows, self.n_rows, self.max_rows, self.work, self.out,
                                    self.lse if lse else None, stream)
        return self

    def lists(self):
        """Per (sequence, query head): the positions it attends to."""
        for b in range(self.B):
            n = self.n if self.lens is None else min(max(int(self.lens[b]), 0), self.n)
            for h in range(self.Hq):
                if self.rows is None:
                    yield b, h, np.arange(n)
                    continue
                S, heads = self.cfg.n_sinks, self.Hq if self.cfg.mode == ckv.CKV_PER_HEAD else self.Hkv
                g = b * heads + h * heads // self.Hq
                got = self.rows[g, :min(max(int(self.n_rows[g]), 0), self.max_rows)].cpu().numpy()
                got = got[(got >= S) & (got < n - 1)]
                yield b, h, np.concatenate([np.arange(min(S, n)), got, [n - 1] if n > S else []]).astype(np.int64)

    def check(self):
        K = ref.values_of(self.K4, self.B, self.Hkv, self.n_max, self.group, False)
        V = ref.values_of(self.V4, self.B, self.Hkv, self.n_max, self.group, True)
        Kp = ref.parts_of(self.K4, self.B, self.Hkv, self.n_max, self.group, False)
        Vp = ref.parts_of(self.V4, self.B, self.Hkv, self.n_max, self.group, True)
        out, lse, q = f64(self.out), f64(self.lse), f64(self.q)
        worst = 0.0
        for b, h, rows in self.lists():
            kv = h * self.Hkv // self.Hq
            want, wlse, eo, el = ref.attend(q[b, h:h + 1], K[b, kv], V[b, kv], rows, Kp[b, kv], Vp[b, kv])
            err = np.abs(out[b, h] - want[0])
            assert (err <= eo[0]).all(), (b, h, len(rows), (err / np.maximum(eo[0], 1e-300)).max())
            if len(rows):
                assert abs(lse[b, h] - wlse[0]) <= el[0], (b, h, lse[b, h], wlse[0], el[0])
                # typical, not worst, errors: weights are off by about 2^-22 and sums by less, and a logit of size Z that
                # was rounded twice (2 u Z) moves its weight by as much, against one of the same size in the denominator
                rel = float(np.linalg.norm(err) / np.linalg.norm(want))
                Z = float(np.abs(q[b, h] @ K[b, kv][rows].T).max()) / np.sqrt(D)
                assert rel <= 3e-6 + 4 * U32 * Z, (b, h, rel, Z)
                worst = max(worst, rel)
            else:
                assert lse[b, h] == -np.inf
        return worst


DENSE = [
    # B, Hq, Hkv, n_max, n, group, dtype, lens
    (1, 1, 1, 1, 1, 32, "bf16", None),
    (1, 4, 1, 40, 7, 64, "f32", None),
    (2, 8, 2, 50, 16, 128, "bf16", None),
    (2, 6, 2, 33, 17, 32, "f32", None),
    (1, 5, 1, 300, 255, 64, "bf16", None),
    (1, 7, 1, 300, 257, 32, "bf16", None),
    (2, 16, 2, 1100, 1025, 32, "f32", None),
    (3, 4, 4, 700, 650, 128, "f32", None),
    (1, 2, 1, 6000, 5555, 64, "bf16", None),
    (5, 8, 4, 400, 390, 32, "bf16", [0, 1, 390, 33, 1000]),
    (6, 8, 1, 2100, 2000, 64, "f32", [0, 0, 15, 16, 17, 2000]),
    (4, 3, 3, 64, 40, 128, "bf16", [-7, 0, 0, 0]),
    (3, 32, 8, 1000, 999, 32, "bf16", [999, 500, 2]),
    (2, 8, 2, 3000, 2900, 64, "bf16", [0, 333]),         # fewer tiles than the grid for n has CTAs
]


@pytest.mark.parametrize("case", DENSE, ids=lambda c: "-".join(map(str, c[:7])) + ("-ragged" if c[7] else ""))
def test_dense_attention(case):
    rng = np.random.default_rng(case[4])
    print(Case(rng, *case).run().check())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kscale", [0.0, 1e-4, 8.0])
def test_dense_attention_flat_and_peaked(dtype, kscale):
    # all keys equal, nearly equal, and logits in the tens, one row taking nearly all
    rng = np.random.default_rng(5)
    Case(rng, 2, 8, 2, 900, 813, 32, dtype, kscale=kscale).run().check()


def test_dense_attention_of_groups_of_very_different_size():
    # each group of channels is judged by itself
    rng = np.random.default_rng(6)
    c = Case(rng, 1, 4, 1, 600, 555, 32, "bf16", wide=True).run()
    K = ref.values_of(c.K4, 1, 1, 600, 32, False)
    V = ref.values_of(c.V4, 1, 1, 600, 32, True)
    want, _, bound, _ = ref.attend(f64(c.q[0]), K[0, 0], V[0, 0], np.arange(555))
    for j in range(4):
        part = slice(32 * j, 32 * j + 32)
        _, _, bound, _ = ref.attend(f64(c.q[0]), K[0, 0], np.where((np.arange(D) // 32 == j), V[0, 0], 0), np.arange(555))
        assert (np.abs(f64(c.out[0]) - want)[:, part] <= bound[:, part]).all()


def test_query_of_zeros_and_tiny_and_large_channels():
    rng = np.random.default_rng(7)
    for scale in (0.0, 2.0 ** -100, 2.0 ** 20):
        c = Case(rng, 1, 4, 1, 200, 150, 32, "f32", kscale=1.0 if scale < 1 else 2.0 ** -20)
        c.q = c.q * scale
        c.q[0, 1, 5] = 3.0 * scale
        c.run().check()


def test_rows_that_are_not_finite():
    rng = np.random.default_rng(8)
    c = Case(rng, 2, 4, 2, 120, 100, 32, "bf16", lens=[100, 60])
    R, dev = ref.rows_padded(120), "cuda"
    cut = 2 * 2 * R * 64
    pk = c.K4[cut:].view(torch.int32).view(2, 2, R, 4)
    pv = c.V4[cut:].view(torch.int32).view(2, 2, R, 4)
    nan = 0x7fc00000
    pk[1, 0, 70] = nan                    # behind the length: never used
    pv[1, 1, 60] = nan
    pv[0, 0, 50, 2] = nan                 # a value group of KV head 0 of sequence 0
    pk[0, 1, 30, 1] = nan                 # a key of KV head 1 of sequence 0
    c.run()
    out = c.out
    assert torch.isfinite(out[1]).all() and torch.isfinite(c.lse[1]).all()
    assert torch.isnan(out[0, :2, 64:96]).all() and torch.isfinite(out[0, :2, :64]).all() and torch.isfinite(out[0, :2, 96:]).all()
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(c.lse[0, 2:]).all() and torch.isfinite(c.lse[0, :2]).all()
    c.q[1, 1, 7] = float("inf")
    c.q[1, 2, 7] = float("nan")
    c.run()
    assert torch.isnan(c.out[1, 1:3]).all() and torch.isfinite(c.out[1, 0]).all() and torch.isfinite(c.out[1, 3]).all()
    del dev


ROWS = [
    # B, Hq, Hkv, n, group, dtype, sinks, per_head, max_rows, lens
    (1, 4, 1, 300, 32, "bf16", 4, False, 40, None),
    (2, 8, 2, 2049, 64, "f32", 4, True, 256, None),
    (2, 16, 2, 500, 128, "bf16", 0, False, 133, None),
    (1, 2, 2, 40, 32, "f32", 7, False, 1, None),
    (3, 8, 4, 200, 32, "bf16", 4, False, 64, [200, 4, 0]),
    (3, 12, 4, 200, 64, "bf16", 4, True, 16, [5, 6, 3]),
    (1, 8, 1, 9000, 32, "bf16", 4, False, 4000, None),
    (2, 4, 4, 30, 32, "f32", 30, False, 5, [30, 12]),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c[:9])) + ("-ragged" if c[9] else ""))
def test_attention_over_rows(case):
    B, Hq, Hkv, n, group, dtype, sinks, per_head, max_rows, lens = case
    rng = np.random.default_rng(n + max_rows)
    G = B * (Hq if per_head else Hkv)
    # any order, repeats, padding, sinks, the new token and rows outside the cache among them
    rows = rng.integers(-3, n + 5, (G, max_rows)).astype(np.int32)
    rows[rng.random((G, max_rows)) < 0.1] = -1
    rows[0, 0], rows[-1, -1] = 2 ** 31 - 1, -2 ** 31
    n_rows = rng.integers(0, max_rows + 1, G).astype(np.int32)
    n_rows[0], n_rows[-1] = max_rows + 9, 0 if G > 1 else max_rows
    if G > 2:
        n_rows[1] = -4
    c = Case(rng, B, Hq, Hkv, n + 13, n, group, dtype, lens=lens, sinks=sinks, rows=torch.from_numpy(rows).cuda(),
             n_rows=torch.from_numpy(n_rows).cuda(), max_rows=max_rows, per_head=per_head)
    c.run().check()


def test_rows_equal_dense_over_everything():
    # every position listed once: the dense result of the same cache, up to the order of the sums
    rng = np.random.default_rng(12)
    n = 700
    rows = torch.stack([torch.randperm(n - 5, generator=torch.Generator().manual_seed(s)) + 4 for s in range(2)]).int().cuda()
    c = Case(rng, 1, 8, 2, n, n, 32, "bf16", sinks=4, rows=rows, n_rows=torch.tensor([n - 5] * 2, dtype=torch.int32).cuda(),
             max_rows=n - 5)
    c.run().check()
    sparse = c.out.clone()
    c.rows = None
    c.run().check()
    assert float((sparse - c.out).norm() / c.out.norm()) < 3e-6


def test_repeats_graphs_streams_and_workspaces():
    rng = np.random.default_rng(13)
    a = Case(rng, 2, 8, 2, 3000, 2900, 32, "bf16", lens=[2900, 700])
    rows = torch.from_numpy(rng.integers(4, 2000, (4, 300)).astype(np.int32)).cuda()
    b = Case(rng, 2, 8, 2, 3000, 2900, 64, "f32", sinks=4, rows=rows, n_rows=torch.full((4,), 300, dtype=torch.int32).cuda(),
             max_rows=300)
    a.run().check()
    first = a.out.clone()
    for _ in range(3):                                  # the same bits every time, the workspace as it was left
        a.out.fill_(0)
        a.run()
        assert torch.equal(a.out, first)
    b.work = a.work                                     # another call's workspace, one call after the other
    b.run().check()
    second = b.out.clone()
    a.run(lse=False)
    assert torch.equal(a.out, first)
    # captured, and replayed with other lengths and queries
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a.run(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a.run(side)
            b.run(side)
    for lens in ([2900, 700], [1, 2900], [0, 333]):
        a.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        a.q.copy_(normal(rng, (2, 8, D), a.dt))
        a.out.fill_(0)
        b.out.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        a.check()
        assert torch.equal(b.out, second)
    # two streams at once, a workspace each
    b.work = torch.zeros_like(a.work)
    a.run()
    want = a.out.clone()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(20):
        a.run(side)
        b.run(other)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and torch.equal(b.out, second)
    assert not a.work[:16].any()


def test_offsets_beyond_32_bits():
    # the last unit's rows lie more than 2^31 bytes into the codes
    free = torch.cuda.mem_get_info()[0]
    B, H, n_max, group = 4, 8, 1_200_000, 128
    cfg = config(B, 4 * H, H, n_max, torch.bfloat16)
    size = ckv.ckv_kv4_bytes(cfg, group)
    assert size > 2 ** 31
    if free < 3 * size:
        pytest.skip("not enough device memory")
    buf = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    T = 40
    x = torch.randn((B, T, H, D), device="cuda").bfloat16()
    y = torch.randn((B, T, H, D), device="cuda").bfloat16()
    pos = (torch.arange(T, dtype=torch.int32, device="cuda") + n_max - T).repeat(B, 1)
    ckv.ckv_kv4_write(cfg, group, x, y, pos, *buf)
    # rows before them are zeros: value 0, logit 0; the listed rows are the last ones
    q = torch.randn((B, 4 * H, D), device="cuda").bfloat16()
    out = torch.empty((B, 4 * H, D), device="cuda")
    work = torch.zeros(ckv.ckv_kv4_workspace(cfg), dtype=torch.uint8, device="cuda")
    rows = pos[0, :-1].repeat(B * H, 1).contiguous()
    ckv.ckv_kv4_attend_rows(cfg, group, q, *buf, n_max, None, rows, torch.full((B * H,), T - 1, dtype=torch.int32, device="cuda"),
                            T - 1, work, out)
    last = [ref.cache_of(f32(t)[-1:, :, -1:].transpose(0, 2, 1, 3), group, bool(i), T) for i, t in enumerate((x, y))]
    K, V = (ref.values_of(last[i], 1, 1, T, group, bool(i))[0, 0, :T] for i in range(2))
    want, _, bound, _ = ref.attend(f64(q[-1, -4:]), K, V, np.arange(T))
    assert (np.abs(f64(out[-1, -4:]) - want) <= bound).all()
    # dense over all of it: n_max - T rows of logit 0 and value 0
    ckv.ckv_kv4_dense_decode(cfg, group, q, *buf, n_max, None, work, out)
    z = f64(q[-1, -4:]) @ K.T / np.sqrt(D)
    p = np.exp(z)
    want = p @ V / (p.sum(-1, keepdims=True) + n_max - T)
    off = float(np.linalg.norm(f64(out[-1, -4:]) - want) / np.linalg.norm(want))
    # the sum of the weights is 1.2 million ones in chains of up to 2^13: 2^13 u in the worst case
    assert off <= 2.0 ** -11, off


def test_long_sequences_of_a_full_machine():
    """32 units of 131072 rows: 100 tiles to a warp, where sums that lose a little with every step show it.  The bound is that of
    the short sequences: sums are rounded to nearest, so their errors do not add up in one direction."""
    B, H, n, group = 4, 8, 131072, 32
    cfg = config(B, 4 * H, H, n, torch.bfloat16)
    buf = [torch.zeros(ckv.ckv_kv4_bytes(cfg, group), dtype=torch.uint8, device="cuda") for _ in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for first in range(0, n, n // 4):
        pos = (torch.arange(n // 4, dtype=torch.int32, device="cuda") + first).repeat(B, 1)
        k, v = (torch.randn((B, n // 4, H, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
        ckv.ckv_kv4_write(cfg, group, k, v, pos, *buf)
    del k, v
    q = (1.5 * torch.randn((B, 4 * H, D), generator=gen, device="cuda")).bfloat16()
    out = torch.empty((B, 4 * H, D), device="cuda")
    lse = torch.empty((B, 4 * H), device="cuda")
    work = torch.zeros(ckv.ckv_kv4_workspace(cfg), dtype=torch.uint8, device="cuda")
    ckv.ckv_kv4_dense_decode(cfg, group, q, *buf, n, None, work, out, lse)
    for unit in (0, 19, 31):
        rows = []
        for i, b in enumerate(buf):
            at, cut = unit * n * 64, B * H * n * 64
            one = torch.cat([b[at:at + n * 64], b[cut + unit * n * 16:cut + (unit + 1) * n * 16]])
            rows.append(torch.from_numpy(ref.values_of(one, 1, 1, n, group, bool(i))[0, 0]).cuda())
        b, h = divmod(unit, H)
        z = q[b, 4 * h:4 * h + 4].double() @ rows[0].T / D ** 0.5
        want = torch.softmax(z, -1) @ rows[1]
        err = (out[b, 4 * h:4 * h + 4].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(err.max()) <= 3e-6 + 4 * U32 * float(z.abs().max()), (unit, err)
        assert float((lse[b, 4 * h:4 * h + 4].double() - torch.logsumexp(z, -1)).abs().max()) <= 2e-5


def test_more_units_than_threads_of_a_block():
    rng = np.random.default_rng(31)
    B, Hkv = 40, 8
    lens = rng.integers(0, 70, B).tolist()
    Case(rng, B, 16, Hkv, 70, 69, 64, "bf16", lens=lens).run().check()
    rows = torch.from_numpy(rng.integers(0, 64, (6 * 64, 9)).astype(np.int32)).cuda()
    n_rows = torch.from_numpy(rng.integers(0, 10, 6 * 64).astype(np.int32)).cuda()
    Case(rng, 6, 64, 8, 64, 60, 32, "f32", sinks=3, rows=rows, n_rows=n_rows, max_rows=9, per_head=True,
         lens=[60, 1, 0, 33, 4, 3]).run().check()


def test_no_listed_rows():
    rng = np.random.default_rng(32)
    c = Case(rng, 2, 4, 2, 30, 20, 32, "bf16", sinks=4, rows=torch.empty((4, 0), dtype=torch.int32, device="cuda"),
             n_rows=torch.tensor([5, 0, -1, 0], dtype=torch.int32, device="cuda"), max_rows=0)
    c.run().check()
    first = c.out.clone()
    ckv.ckv_kv4_attend_rows(c.cfg, c.group, c.q, c.K4, c.V4, c.n, None, None, c.n_rows, 0, c.work, c.out)
    assert torch.equal(c.out, first)


def test_a_cache_as_the_source_of_rows():
    # [B][H][n_max][D] caches into 4 bits at rows 0 .. T-1, and many heads
    B, H, n, group = 2, 65, 33, 64
    cfg = config(B, 2 * H, H, n, torch.bfloat16)
    K, V = (torch.randn((B, H, n, D), device="cuda").bfloat16() for _ in range(2))
    buf = [torch.zeros(ckv.ckv_kv4_bytes(cfg, group), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ckv.ckv_kv4_write(cfg, group, K.transpose(1, 2)[:, :20], V.transpose(1, 2)[:, :20], None, *buf)
    for i, t in enumerate((K, V)):
        code, scale, middle = ref.quantise(f32(t[:, :, :20]), group)
        want = (middle[..., None] + scale[..., None] * code.reshape(B, H, 20, D // group, group)).reshape(B, H, 20, D)
        got = ref.values_of(buf[i], B, H, n, group, bool(i))
        np.testing.assert_array_equal(got[:, :, :20], want)
        assert not got[:, :, 20:].any()
    # every head of a token through the norm and rotation as well
    x = torch.randn((B, 3, 4 * H, D), device="cuda").bfloat16()
    pos = torch.tensor([[5, -1, 32], [0, 1, 2]], dtype=torch.int32, device="cuda")
    out = torch.zeros((B, 3, 2 * H, D), dtype=torch.bfloat16, device="cuda")
    freq = 1.0e4 ** (-np.arange(0, D, 2) / D)
    ckv.ckv_qk_norm_rope(cfg, x[:, :, :2 * H], x[:, :, 2 * H:3 * H], x[:, :, 3 * H:], pos, out, freq, K=K, V=V)
    want, bound = ref.rotated(f64(x[:, :, :2 * H]), pos.cpu().numpy(), None, 0, freq, False, 1.0)
    want[0, 1], bound[0, 1] = 0, 0
    assert (np.abs(f64(out) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()
    assert torch.equal(V[1, :, :3], x[1, :, 3 * H:].transpose(0, 1)) and torch.equal(V[0, :, 32], x[0, 2, 3 * H:])


def test_rotated_rows_equal_an_eager_norm_and_rotation():
    # the fixed order of the sum of squares and one rounding a step: the same bits as elementary operations in 32 bits
    B, T, H = 2, 300, 4
    cfg = config(B, H, H, T, torch.float32)
    x = torch.randn((B, T, 3 * H, D), device="cuda")
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    freq = 1.0e6 ** (-np.arange(0, D, 2) / D)
    out, K, V = torch.empty((B, T, H, D), device="cuda"), *(torch.empty((B, H, T, D), device="cuda") for _ in range(2))
    ckv.ckv_qk_norm_rope(cfg, x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], pos, out, freq, q_weight=w, k_weight=w, K=K, V=V)
    y = x[:, :, :H]
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    ang = (pos.double()[..., None] * torch.from_numpy(freq).cuda())[:, :, None]
    c, s = ang.cos().float(), ang.sin().float()
    a, b = y[..., :64], y[..., 64:]
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    # a cosine rounded next to a border may differ by one step of 2^-24: of 600 x 64 cosines, at 2^-49 off, none is expected
    assert float((out != want).float().mean()) < 1e-4
    assert float((out - want).abs().max()) <= 2.0 ** -22 * float(want.abs().max())


# ------------------------------------------------------- as they are used
def test_decode_steps_on_a_4_bit_cache():
    """A prompt's rows into both kinds of cache, then steps of one token: norm and rotation, the append, dense attention and
    attention over the kept rows, captured in one graph, against ckv_dense_decode on the rows read back and the 64-bit form."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, n0, steps, group, S = 2, 8, 2, 333, 4, 32, 4
    n_max = n0 + steps
    dt = torch.bfloat16
    cfg = config(B, Hq, Hkv, n_max, dt, sinks=S)
    cfg.max_communities, cfg.kappa, cfg.budget, cfg.slack = 64, 8, 64, 16
    freq = 1.0e6 ** (-np.arange(0, D, 2) / D)
    wq, wk = ((1 + 0.1 * normal(rng, (D,), torch.float32)).to(dt) for _ in range(2))
    K, V = (torch.zeros((B, Hkv, n_max, D), dtype=dt, device="cuda") for _ in range(2))
    K4, V4 = (torch.zeros(ckv.ckv_kv4_bytes(cfg, group), dtype=torch.uint8, device="cuda") for _ in range(2))
    work = torch.zeros(ckv.ckv_kv4_workspace(cfg), dtype=torch.uint8, device="cuda")

    def rows(x, pos, q_out):
        ckv.ckv_qk_norm_rope(cfg, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], pos, q_out, freq, q_weight=wq,
                             k_weight=wk, K=K, V=V, K4=K4, V4=V4, group=group, stream=torch.cuda.current_stream())

    prompt = normal(rng, (B, n0, Hq + 2 * Hkv, D), dt)
    qp = torch.empty((B, n0, Hq, D), dtype=dt, device="cuda")
    rows(prompt, torch.arange(n0, dtype=torch.int32, device="cuda").repeat(B, 1), qp)
    x = torch.empty((B, 1, Hq + 2 * Hkv, D), dtype=dt, device="cuda")
    pos = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.empty((B, 1, Hq, D), dtype=dt, device="cuda")
    dense, sparse = (torch.empty((B, Hq, D), device="cuda") for _ in range(2))
    kept = torch.from_numpy(np.stack([np.sort(rng.permutation(np.arange(S, n0))[:60]) for _ in range(B * Hkv)]).astype(np.int32)).cuda()
    n_kept = torch.full((B * Hkv,), 60, dtype=torch.int32, device="cuda")

    def step():
        st = torch.cuda.current_stream()
        rows(x, pos, q)
        ckv.ckv_kv4_dense_decode(cfg, group, q[:, 0], K4, V4, n_max, lens, work, dense, stream=st)
        ckv.ckv_kv4_attend_rows(cfg, group, q[:, 0], K4, V4, n_max, lens, kept, n_kept, 60, work, sparse, stream=st)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pos.fill_(-1)                                   # a padded step warms up and writes nothing
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    ctx = ckv.ckv_create(cfg)
    try:
        back = [torch.zeros_like(K) for _ in range(2)]
        out = torch.empty((B, Hq, D), device="cuda")
        for i in range(steps):
            n = n0 + i + 1
            x.copy_(normal(rng, (B, 1, Hq + 2 * Hkv, D), dt))
            pos.fill_(n - 1)
            lens.fill_(n)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want_k, kb = ref.rotated(f64(x[:, :, Hq:Hq + Hkv]), np.full((B, 1), n - 1), f64(wk), 1e-6, freq, False, 1.0)
            err = np.abs(f64(K[:, :, n - 1]) - want_k[:, 0])
            assert (err <= kb[:, 0] + 2.0 ** -8 * (np.abs(want_k[:, 0]) + kb[:, 0])).all()
            # the 4-bit rows are those of K and V
            k4, v4 = (ref.values_of(b, B, Hkv, n_max, group, bool(j)) for j, b in enumerate((K4, V4)))
            for held, t in ((k4, K), (v4, V)):
                code, scale, middle = ref.quantise(f32(t[:, :, :n]), group)
                value = middle[..., None] + scale[..., None] * code.reshape(B, Hkv, n, D // group, group)
                np.testing.assert_array_equal(held[:, :, :n], value.reshape(B, Hkv, n, D))
            for b in range(B):
                for h in range(Hq):
                    kv = h * Hkv // Hq
                    sel = kept[b * Hkv + kv].cpu().numpy()
                    for got, at in ((dense, np.arange(n)), (sparse, np.concatenate([np.arange(S), sel, [n - 1]]))):
                        want, _, eo, _ = ref.attend(f64(q[b, 0, h:h + 1]), k4[b, kv], v4[b, kv], at)
                        assert (np.abs(f64(got[b, h]) - want[0]) <= eo[0]).all()
            # ckv_dense_decode on the rows read back: their rounding to bfloat16 is all that differs
            ckv.ckv_kv4_read(cfg, group, K4, V4, 0, n, *back)
            ckv.ckv_dense_decode(ctx, q[:, 0].contiguous(), *back, n, out)
            assert float((out - dense).norm() / dense.norm()) < 2e-2
    finally:
        ckv.ckv_destroy(ctx)


def test_rows_made_here_feed_the_decode_step():
    """ckv_qk_norm_rope's caches and queries are those of ckv_build_graph and of ckv_decode_step."""
    rng = np.random.default_rng(22)
    B, Hq, Hkv, n0, S = 1, 4, 1, 256, 4
    dt = torch.bfloat16
    cfg = config(B, Hq, Hkv, n0 + 1, dt, sinks=S)
    cfg.max_communities, cfg.kappa, cfg.budget, cfg.slack = 16, 8, 4096, 16
    freq = 1.0e4 ** (-np.arange(0, D, 2) / D)
    K, V = (torch.zeros((B, Hkv, n0 + 1, D), dtype=dt, device="cuda") for _ in range(2))
    x = normal(rng, (B, n0 + 1, Hq + 2 * Hkv, D), dt)
    q = torch.empty((B, Hq, n0 + 1, D), dtype=dt, device="cuda")
    pos = torch.arange(n0 + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    ckv.ckv_qk_norm_rope(cfg, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], pos, q.transpose(1, 2), freq, K=K, V=V)
    want, bound = ref.rotated(f64(x[:, :, :Hq]), pos.cpu().numpy(), None, 0, freq, False, 1.0)
    assert (np.abs(f64(q).transpose(0, 2, 1, 3) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()
    ctx = ckv.ckv_create(cfg)
    try:
        labels = (np.arange(n0, dtype=np.int32) % 16)[None].copy()
        ckv.ckv_init_communities(ctx, labels, 0, 16, K, n0)
        out = torch.empty((B, Hq, D), device="cuda")
        qn = q[:, :, n0].contiguous()
        ckv.ckv_decode_step(ctx, qn, K, V, n0 + 1, out)
        ckv.ckv_assign_update(ctx, K, n0 + 1)
        assert ckv.ckv_last_error(ctx) == ckv.CKV_OK
        # a budget that covers everything: dense attention over the rows written here
        z = f64(qn[0]) @ f64(K[0, 0]).T / np.sqrt(D)
        p = np.exp(z - z.max(-1, keepdims=True))
        want = p @ f64(V[0, 0]) / p.sum(-1, keepdims=True)
        assert (np.abs(f64(out[0]) - want).max(-1) <= 2e-3 * np.abs(want).max(-1)).all()
    finally:
        ckv.ckv_destroy(ctx)
