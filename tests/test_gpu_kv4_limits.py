"""Decode attention over a 4-bit cache and rows into the caches on the GPU, at
the borders of what they take: buffers shared by calls of different shapes,
weights and scales far below the largest, logits and keys far from 1, channels
that are not finite."""
import numpy as np
import pytest
import torch

import long_context_decode_ckv_b200 as ckv
from long_context_decode_ckv_b200 import build as ckv_build
from tests import kv4_reference as ref
from tests.conftest import gpu_available
from tests.kv4_reference import D, U32
from tests.test_gpu_kv4 import Case, config, f64

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ckv_build.build()


# ------------------------------------------------------------ the workspace
def test_one_workspace_over_batches_of_different_size():
    # small and large batches in turn, each with partial results that the next one's counters must not be taken from
    rng = np.random.default_rng(41)
    lists = torch.from_numpy(rng.integers(4, 900, (8, 700)).astype(np.int32)).cuda()
    cases = [
        Case(rng, 1, 32, 8, 3000, 2900, 32, "bf16"),
        Case(rng, 16, 32, 8, 800, 800, 64, "bf16", lens=rng.integers(100, 801, 16).tolist()),
        Case(rng, 2, 16, 2, 3000, 2999, 128, "f32"),
        Case(rng, 1, 8, 2, 1000, 990, 32, "bf16", sinks=4, rows=lists, n_rows=torch.full((8,), 700, dtype=torch.int32).cuda(),
             max_rows=700, per_head=True),
        Case(rng, 40, 16, 8, 400, 400, 32, "f32", lens=rng.integers(0, 401, 40).tolist()),
    ]
    work = torch.zeros(max(ckv.ckv_kv4_workspace(c.cfg) for c in cases), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 4, 3, 1, 0, 4, 2):
        cases[i].work = work
        cases[i].out.fill_(9.0)
        cases[i].lse.fill_(9.0)
        cases[i].run().check()


# --------------------------------------------------------------- refusals
def test_addresses_off_four_bytes_are_refused():
    rng = np.random.default_rng(42)
    rows = torch.full((2, 5), 9, dtype=torch.int32, device="cuda")
    c = Case(rng, 1, 4, 2, 40, 33, 32, "bf16", lens=[33], sinks=4, rows=rows, n_rows=rows[:, 0].contiguous(), max_rows=5)
    good = dict(cfg=c.cfg, group=32, q=c.q, K4=c.K4, V4=c.V4, n=33, lens=c.lens, workspace=c.work, out=c.out, lse=c.lse)
    more = dict(good, rows=rows, n_rows=c.n_rows, max_rows=5)
    for call, args in ((ckv.ckv_kv4_dense_decode, good), (ckv.ckv_kv4_attend_rows, more)):
        for name in ("lens", "lse", "rows", "n_rows"):
            if name in args:
                with pytest.raises(ckv.CkvError) as e:
                    call(**{**args, name: args[name].data_ptr() + 2})
                assert e.value.status == ckv.CKV_ERR_INVALID_ARG
        call(**{**args, "lse": c.lse.data_ptr(), "lens": c.lens.data_ptr()})
    c.check()


# ------------------------------------------------ weights and value scales
def crafted(rng, gaps, vrows, group, dtype="f32", heads=4):
    """One sequence whose row j has a weight of about 2^-gaps[j] of the largest and the values vrows[j]."""
    n = len(gaps)
    w = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    c = Case(rng, 1, heads, 1, n, n, group, dtype)
    a = -np.asarray(gaps, np.float64) * np.log(2) / np.sqrt(D)
    c.K4 = ref.cache_of((a[:, None] * w).astype(np.float32)[None, None], group, False, n).cuda()
    c.V4 = ref.cache_of(vrows.astype(np.float32)[None, None], group, True, n).cuda()
    c.q = torch.from_numpy((w * (1 + 0.01 * rng.standard_normal((1, heads, D)))).astype(np.float32)).to(c.dt).cuda()
    return c


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("heads", [1, 4, 8])
@pytest.mark.parametrize("gap", [4, 12, 20, 24])
def test_many_small_weights_beside_a_few_that_take_nearly_all(gap, heads, group):
    # the large weights' values are zero, or 2^-10 of the others', so that the output is made by the small weights: each of them
    # has to enter with the same relative error as a large one
    rng = np.random.default_rng(gap + heads)
    n = 900
    for small in (0.0, 2.0 ** -10):
        gaps = gap + rng.uniform(-1, 1, n)
        v = rng.standard_normal((n, D))
        gaps[::32] = 0                                  # one in every tile of every warp
        v[::32] *= small
        crafted(rng, gaps, v, group, heads=heads).run().check()


@pytest.mark.parametrize("order", ["first", "last", "mixed"])
@pytest.mark.parametrize("gap,ratio", [(0, 6), (0, 17), (17, 14), (20, 17), (17, 10), (24, 6), (10, 28)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_whose_values_differ_in_size(group, gap, ratio, order):
    # a few rows of values 2^ratio times the others' and of no weight to speak of, before, behind or among rows of weight 2^-gap
    # of the largest, whose own values are zero
    rng = np.random.default_rng(ratio + gap)
    n = 1024
    gaps = gap + rng.uniform(-1, 1, n)
    v = rng.standard_normal((n, D)) * 2.0 ** -ratio
    gaps[5::32] = 0
    v[5::32] = 0
    large = {"first": np.arange(0, 256, 32), "last": np.arange(n - 256, n, 32), "mixed": np.arange(0, n, 96)}[order] + 9
    gaps[large] = gap + ratio + 40
    v[large] *= 2.0 ** ratio
    crafted(rng, gaps, v, group).run().check()


def test_large_values_of_small_weight_and_small_values_of_large_weight():
    # p v is of the same size in every row, p between 1 and 2^-20
    rng = np.random.default_rng(43)
    n = 700
    gaps = rng.uniform(0, 20, n)
    crafted(rng, gaps, rng.standard_normal((n, D)) * 2.0 ** (gaps[:, None] - 20), 32).run().check()


# ------------------------------------------------------- logits far from 0
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("top", [1e6, 5e7, 9.4e7, 1.5e8, 1.8e8, 4e8, 1e10])
def test_large_logits(top, sign):
    # the largest logit, of size `top`, is far enough from the others for any error of 32 bits: it takes all the weight
    rng = np.random.default_rng(44)
    n, best = 300, 211
    c = Case(rng, 1, 4, 1, n, n, 64, "f32")
    w = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    size = rng.uniform(0.5, 0.9, n) if sign > 0 else -rng.uniform(1.1, 1.6, n)
    size[best] = sign
    c.q = torch.from_numpy(np.tile(w, (1, 4, 1)).astype(np.float32)).cuda() * 128.0
    k = (size[:, None] * w * top / (128 * np.sqrt(D))).astype(np.float32)
    c.K4 = ref.cache_of(k[None, None], 64, False, n).cuda()
    c.run()
    K = ref.values_of(c.K4, 1, 1, n, 64, False)[0, 0]
    V = ref.values_of(c.V4, 1, 1, n, 64, True)[0, 0]
    z = f64(c.q[0]) @ K[:n].T / np.sqrt(D)
    order = np.sort(z, -1)
    assert (z.argmax(-1) == best).all() and (order[:, -1] - order[:, -2] > 0.05 * top).all()
    # the weight is 1 but for its two fp16 parts (2^-22), and the value is put together from its two terms (2 half steps)
    parts = ref.parts_of(c.V4, 1, 1, n, 64, True)[0, 0][best]
    assert (np.abs(f64(c.out[0]) - V[best]) <= 2.0 ** -21 * parts).all()
    # the logit's error as in kv4_reference.attend, and its conversion to and from powers of two (4 half steps)
    parts = ref.parts_of(c.K4, 1, 1, n, 64, False)[0, 0][best]
    bound = (16 * U32 + 2.0 ** -27) * np.abs(f64(c.q[0])).max() * parts.sum() / np.sqrt(D) + 8 * U32 * top
    assert (np.abs(f64(c.lse[0]) - z.max(-1)) <= bound).all()


# ------------------------------------------- channels that are not rotated
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 64, 112])
def test_channels_behind_the_rotation_stay(rot, interleaved, dtype):
    # without a norm they keep their bits: infinities, NaN and -0 among them, and their neighbours are not touched
    rng = np.random.default_rng(rot)
    B, T, Hq, Hkv, n_max, group = 2, 9, 3, 1, 20, 32
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    c = config(B, Hq, Hkv, n_max, dt)
    x = torch.from_numpy(rng.standard_normal((B, T, Hq + 2 * Hkv, D)).astype(np.float32)).to(dt)
    x[:, 0, :, rot] = float("inf")
    x[:, 1, :, rot + 1] = float("-inf")
    x[:, 2, :, D - 1] = float("nan")
    x[:, 3, :, rot::2] = -0.0
    x[:, 4, :, rot + 1::2] = -0.0
    x[:, 5, :, rot:] = -0.0
    x = x.cuda()
    pos = torch.arange(3, T + 3, dtype=torch.int32, device="cuda").repeat(B, 1)
    freq = 1.0e4 ** (-np.arange(0, rot, 2) / rot)
    bits = torch.int16 if dt == torch.bfloat16 else torch.int32
    out = torch.zeros((B, T, Hq, D), dtype=dt, device="cuda")
    K, V = (torch.zeros((B, Hkv, n_max, D), dtype=dt, device="cuda") for _ in range(2))
    four = [torch.zeros(ckv.ckv_kv4_bytes(c, group), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want4 = [torch.zeros_like(b) for b in four]
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    ckv.ckv_qk_norm_rope(c, q, k, v, pos, out, freq, interleaved=interleaved, K=K, V=V)

    def same(got, want):
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got.view(bits)[~nan], want.view(bits)[~nan])
    same(out[..., rot:].contiguous(), q[..., rot:].contiguous())
    same(K[:, :, 3:T + 3, rot:].contiguous(), k[..., rot:].transpose(1, 2).contiguous())
    assert torch.isfinite(out[..., :rot]).all() and torch.isfinite(K[..., :rot]).all()
    # the 4-bit rows are those of K, quantised
    out2 = torch.zeros_like(out)
    ckv.ckv_qk_norm_rope(c, q, k, v, pos, out2, freq, interleaved=interleaved, K4=four[0], V4=four[1], group=group)
    ckv.ckv_kv4_write(c, group, K[:, :, 3:T + 3].transpose(1, 2), V[:, :, 3:T + 3].transpose(1, 2), pos, *want4)
    assert torch.equal(four[0], want4[0]) and torch.equal(four[1], want4[1])
    same(out2, out)


# ----------------------------------------------------- errors of other calls
def test_calls_after_another_one_failed():
    # an allocation of a terabyte fails at once; what it leaves behind is not an error of the calls that follow
    rng = np.random.default_rng(46)
    big = config(16, 64, 8, 1024, torch.bfloat16, sinks=4)
    big.max_communities, big.kappa, big.budget, big.slack, big.pool_capacity = 16, 8, 64, 16, 2 ** 31 - 1
    c = Case(rng, 1, 4, 2, 40, 33, 32, "bf16")
    x = torch.randn((1, 5, 8, D), device="cuda").bfloat16()
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[None].contiguous()
    K, V = (torch.zeros((1, 2, 40, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    calls = [
        lambda: ckv.ckv_qk_norm_rope(c.cfg, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], pos, x[:, :, :4], np.ones(64), K=K, V=V),
        lambda: ckv.ckv_kv4_read(c.cfg, 32, c.K4, c.V4, 0, 40, K, V),
        lambda: c.run().check(),
        lambda: ckv.ckv_kv4_write(c.cfg, 32, x[:, :, 4:6], x[:, :, 6:], pos, c.K4, c.V4),
    ]
    for call in calls:
        with pytest.raises(ckv.CkvError) as e:
            ckv.ckv_create(big)
        assert e.value.status == ckv.CKV_ERR_OOM
        call()


# -------------------------------------------------- keys and queries far from 1
@pytest.mark.parametrize("kexp,qexp", [(100, -100), (84, -80), (95, -90), (118, -110), (-100, 100), (-120, 120), (-60, 60), (105, -3),
                                       (110, 10), (122, -122), (0, 115), (10, 100)])
@pytest.mark.parametrize("group", [32, 128])
def test_keys_and_queries_of_any_size(group, kexp, qexp):
    rng = np.random.default_rng(45)
    n = 200
    c = Case(rng, 1, 4, 1, n, n, group, "f32")
    k = rng.standard_normal((n, D)) + 0.5
    q = rng.standard_normal((4, D))
    c.K4 = ref.cache_of((k * 2.0 ** kexp).astype(np.float32)[None, None], group, False, n).cuda()
    c.q = torch.from_numpy((q * 2.0 ** qexp).astype(np.float32))[None].cuda()
    c.run()
    if abs(kexp + qexp) <= 10:
        c.check()
        return
    # logits of 2^20 and more: one row takes all the weight, 1 but for its two fp16 parts
    K = ref.values_of(c.K4, 1, 1, n, group, False)[0, 0]
    z = f64(c.q[0]) @ K[:n].T / np.sqrt(D)
    order = np.sort(z, -1)
    assert (order[:, -1] - order[:, -2] > 2.0 ** -10 * np.abs(z).max(-1)).all()
    want = ref.values_of(c.V4, 1, 1, n, group, True)[0, 0][z.argmax(-1)]
    parts = ref.parts_of(c.V4, 1, 1, n, group, True)[0, 0][z.argmax(-1)]
    assert (np.abs(f64(c.out[0]) - want) <= 2.0 ** -21 * parts).all()


# ------------------------------------------------------- splits of the work
GRIDS = [
    # B, Hq, Hkv, n, group, dtype, lens: units of one length in one share each, in several, in shares that cross units, in two
    # waves of CTAs; units of their own lengths, a tile to a CTA, one CTA to an SM, two
    (10, 32, 8, 3700, 32, "bf16", None),
    (5, 4, 1, 20000, 128, "bf16", None),
    (1, 2, 1, 33000, 64, "f32", None),
    (7, 36, 9, 1500, 64, "bf16", None),
    (25, 48, 12, 100, 128, "bf16", None),
    (37, 16, 16, 70, 32, "f32", None),
    (70, 20, 10, 40, 64, "bf16", None),
    (20, 64, 8, 600, 128, "bf16", None),
    (3, 8, 2, 1300, 32, "bf16", [1300, 11, 700]),
    (12, 8, 8, 1200, 64, "f32", list(range(0, 1200, 100))),
    (11, 32, 8, 4500, 128, "bf16", [4500 - 37 * i for i in range(11)]),
    (90, 8, 8, 65, 32, "bf16", [i % 66 for i in range(90)]),
]


@pytest.mark.parametrize("case", GRIDS, ids=lambda c: "-".join(map(str, c[:6])) + ("-ragged" if c[6] else ""))
def test_splits_of_the_work(case):
    B, Hq, Hkv, n, group, dtype, lens = case
    Case(np.random.default_rng(n), B, Hq, Hkv, n + 3, n, group, dtype, lens=lens).run().check()


def test_splits_of_row_lists():
    rng = np.random.default_rng(47)
    for B, Hq, Hkv, n, max_rows, per_head in ((1, 4, 1, 40000, 30000, False), (5, 8, 4, 700, 200, True), (20, 16, 4, 400, 300, False),
                                              (80, 4, 1, 3000, 2900, False), (50, 16, 4, 64, 20, True)):
        G = B * (Hq if per_head else Hkv)
        rows = torch.from_numpy(rng.integers(4, n - 1, (G, max_rows)).astype(np.int32)).cuda()
        n_rows = torch.from_numpy(rng.integers(0, max_rows + 1, G).astype(np.int32)).cuda()
        Case(rng, B, Hq, Hkv, n, n, 64, "bf16", sinks=4, rows=rows, n_rows=n_rows, max_rows=max_rows, per_head=per_head).run().check()


# ------------------------------------------------------------ long caches
def test_sums_over_a_long_cache():
    # 32 units of 1.2 million rows, the last ones more than 2^31 bytes into the codes: all logits 0, values in 3000 rows from the
    # first to the last.  The weights are equal, so the output is the values' sum over n.
    B, H, n, group, T = 4, 8, 1_200_000, 128, 3000
    cfg = config(B, 4 * H, H, n, torch.bfloat16)
    size = ckv.ckv_kv4_bytes(cfg, group)
    assert size > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 3 * size:
        pytest.skip("not enough device memory")
    K4, V4 = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(48)
    pos = np.stack([np.concatenate([[0, n - 1], 1 + rng.permutation(n - 2)[:T - 2]]) for _ in range(B)]).astype(np.int32)
    v = torch.from_numpy(rng.standard_normal((B, T, H, D)).astype(np.float32)).bfloat16().cuda()
    ckv.ckv_kv4_write(cfg, group, torch.zeros_like(v), v, torch.from_numpy(pos).cuda(), K4, V4)
    q = torch.randn((B, 4 * H, D), device="cuda").bfloat16()
    out, lse = torch.empty((B, 4 * H, D), device="cuda"), torch.empty((B, 4 * H), device="cuda")
    work = torch.zeros(ckv.ckv_kv4_workspace(cfg), dtype=torch.uint8, device="cuda")
    ckv.ckv_kv4_dense_decode(cfg, group, q, K4, V4, n, None, work, out, lse)
    code, scale, middle = ref.quantise(v.float().cpu().numpy(), group)
    want = (middle + scale * code).sum(1) / n                            # one group to a row
    parts = (np.abs(middle) + np.abs(scale * code)).sum(1) / n
    # the weights' sum: a lane adds once for 16 rows of its warp, one of 8 of a share, and a unit has 4 shares at least; the
    # values: a warp meets a few of the 3000 rows (those of value 0 add nothing), then come 8 warps and up to 37 shares: 64 half
    # steps of the sum of all their sizes
    chain = (n / (16 * 8 * 4) + 64) * U32
    bound = 64 * U32 * parts + chain * np.abs(want)
    err = np.abs(f64(out).reshape(B, H, 4, D) - want[:, :, None])
    assert (err <= bound[:, :, None]).all(), (err / bound[:, :, None]).max()
    assert (np.abs(f64(lse) - np.log(n)) <= chain + 2 * U32 * np.log(n)).all()


# ------------------------------------------------------- the order of a sum
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_its_order_written_out(dtype):
    # 32 sums of four neighbouring squares one after the other, these by halves; every step rounded to 32 bits.  The kernel for
    # 4-bit rows holds a row's channels in other lanes and adds in the same order.
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    B, T, H = 2, 150, 3
    cfg = config(B, H, H, T, dt)
    gen = torch.Generator(device="cuda").manual_seed(49)
    x = (2 * torch.randn((B, T, 3 * H, D), generator=gen, device="cuda")).to(dt)
    w = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    four = [torch.zeros(ckv.ckv_kv4_bytes(cfg, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    y = x[:, :, :2 * H].float()
    s = (y * y).unflatten(-1, (32, 4))
    s = ((s[..., 0] + s[..., 1]) + s[..., 2]) + s[..., 3]
    while s.shape[-1] > 1:
        s = s[..., :s.shape[-1] // 2] + s[..., s.shape[-1] // 2:]
    want = (y * torch.rsqrt(s / D + 1e-6) * w.float()).to(dt)
    for more in ({}, dict(K4=four[0], V4=four[1], group=64)):
        out = torch.empty((B, T, H, D), dtype=dt, device="cuda")
        K, V = (torch.empty((B, H, T, D), dtype=dt, device="cuda") for _ in range(2))
        ckv.ckv_qk_norm_rope(cfg, x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], pos, out, None, q_weight=w, k_weight=w, K=K, V=V,
                             **more)
        assert torch.equal(out, want[:, :, :H]) and torch.equal(K.transpose(1, 2), want[:, :, H:])


# ---------------------------------------------------- odd numbers of heads
@pytest.mark.parametrize("heads", [1, 3, 9, 11])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_an_odd_number_of_heads(dtype, heads):
    # half of a warp has no row of its own beside the last head; codes, parameters and rows are those of the formulas
    rng = np.random.default_rng(heads)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    B, T = 3, 700
    c = config(B, heads, heads, T, dt)
    x = torch.from_numpy((rng.standard_normal((B, T, 3 * heads, D)) * 2.0 ** rng.integers(-3, 4, (B, T, 1, 1))).astype(np.float32))
    x = x.to(dt).cuda()
    q, k, v = x[:, :, :heads], x[:, :, heads:2 * heads], x[:, :, 2 * heads:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    for group in (32, 64, 128):
        K, V = (torch.full((B, heads, T, D), 5.0, dtype=dt, device="cuda") for _ in range(2))
        four, alone = ([torch.zeros(ckv.ckv_kv4_bytes(c, group), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2))
        out = torch.full((B, T, heads, D), 5.0, dtype=dt, device="cuda")
        ckv.ckv_qk_norm_rope(c, q, k, v, pos, out, None, K=K, V=V, K4=four[0], V4=four[1], group=group)
        ckv.ckv_kv4_write(c, group, k, v, None, *alone)
        assert torch.equal(out, q) and torch.equal(K.transpose(1, 2), k) and torch.equal(V.transpose(1, 2), v)
        for i, t in enumerate((k, v)):
            assert torch.equal(four[i], alone[i])
            by, pa = ref.split(alone[i], B, heads, T, group)
            code, scale, middle = ref.quantise(t.float().cpu().numpy().transpose(0, 2, 1, 3), group)
            np.testing.assert_array_equal(ref.codes(by[:, :, :T], bool(i)), code)
            np.testing.assert_array_equal(pa[:, :, :T, :, 0], scale)
            np.testing.assert_array_equal(pa[:, :, :T, :, 1], middle)


def test_other_calls_after_a_failed_allocation():
    # a failed ckv_create leaves nothing behind for calls that look at the last error after their launch
    big = config(16, 64, 8, 1024, torch.bfloat16, sinks=4)
    big.max_communities, big.kappa, big.budget, big.slack, big.pool_capacity = 16, 8, 64, 16, 2 ** 31 - 1
    i64, i32, f32 = (dict(dtype=t, device="cuda") for t in (torch.int64, torch.int32, torch.float32))
    rp, col, w = torch.tensor([0, 0, 1, 2], **i64), torch.tensor([0, 1], **i32), torch.ones(2, **f32)
    labels = torch.zeros(3, **i32)
    work = torch.empty(ckv.ckv_modularity_workspace(1), dtype=torch.uint8, device="cuda")
    before = ckv.ckv_modularity(3, rp, col, w, labels, 1, 1.0, work)
    with pytest.raises(ckv.CkvError) as e:
        ckv.ckv_create(big)
    assert e.value.status == ckv.CKV_ERR_OOM
    assert ckv.ckv_modularity(3, rp, col, w, labels, 1, 1.0, work) == before
