"""The 4-bit cache's entry points on a machine without a GPU: sizes, and
arguments refused before any device call."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_decode_ckv_b200 as ckv
from long_context_decode_ckv_b200 import build as ckv_build
from tests import kv4_reference as ref

BAD = ckv.CKV_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    ckv_build.build()
    return ckv.lib()


def config(**kw):
    c = ckv.ckv_config()
    c.batch, c.n_q_heads, c.n_kv_heads, c.head_dim, c.n_max = 2, 8, 2, 128, 100
    c.kv_dtype, c.mode, c.n_sinks, c.device = ckv.CKV_BF16, ckv.CKV_QUERY_GROUP, 4, 0
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_SHAPES = [dict(batch=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(head_dim=64), dict(n_max=0),
              dict(n_max=2 ** 31 - 1), dict(kv_dtype=5), dict(device=-1), dict(device=64), dict(batch=2 ** 20, n_q_heads=8)]


def test_sizes(L):
    for group in (32, 64, 128):
        for n_max in (1, 16, 17, 131200):
            R = ref.rows_padded(n_max)
            assert ckv.ckv_kv4_bytes(config(n_max=n_max), group) == 2 * 2 * R * (64 + 4 * 128 // group)
    for group in (0, 16, 48, 256, -32):
        assert ckv.ckv_kv4_bytes(config(), group) == 0
    assert ckv.ckv_kv4_workspace(config()) > 0
    assert L.ckv_kv4_bytes(None, 32) == 0 and L.ckv_kv4_workspace(None) == 0
    for bad in BAD_SHAPES:
        assert ckv.ckv_kv4_bytes(config(**bad), 32) == 0 and ckv.ckv_kv4_workspace(config(**bad)) == 0


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)           # 8-byte aligned only


def qkv(**kw):
    f = (ctypes.c_double * 64)(*([1.0] * 64))
    x = ckv.ckv_qkv()
    x.n_tokens, x.rot_dim, x.group, x.eps, x.rot_scale = 3, 128, 32, 1e-6, 1.0
    x.inv_freq_host = ctypes.cast(f, ctypes.c_void_p)
    x.keep = f
    for name in ("q", "k", "v", "pos", "q_out", "K", "V", "K4", "V4"):
        setattr(x, name, P)
    for name in ("q_stride", "k_stride", "v_stride", "q_out_stride"):
        setattr(x, name, (ctypes.c_int64 * 3)(4096, 1024, 128))
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def test_norm_rope_arguments_checked(L):
    c = config()
    call = lambda cfg, x: L.ckv_qk_norm_rope(ctypes.byref(cfg), ctypes.byref(x), None)  # noqa: E731
    assert L.ckv_qk_norm_rope(None, ctypes.byref(qkv()), None) == BAD
    assert L.ckv_qk_norm_rope(ctypes.byref(c), None, None) == BAD
    for bad in BAD_SHAPES:
        assert call(config(**bad), qkv()) == BAD
    for name in ("q", "k", "v", "pos", "q_out"):
        assert call(c, qkv(**{name: None})) == BAD
    for name in ("q", "k", "v", "q_out", "K", "V", "K4", "V4", "q_weight", "k_weight"):
        assert call(c, qkv(**{name: ODD})) == BAD
    for name in ("K", "V", "K4", "V4"):
        assert call(c, qkv(**{name: None})) == BAD                      # one of a pair
    assert call(c, qkv(K=None, V=None, K4=None, V4=None)) == BAD        # nowhere to write
    for group in (0, 16, 33, 256):
        assert call(c, qkv(group=group)) == BAD
    for rot in (-16, 8, 40, 144):
        assert call(c, qkv(rot_dim=rot)) == BAD
    assert call(c, qkv(inv_freq_host=None)) == BAD
    assert call(c, qkv(n_tokens=-1)) == BAD and call(c, qkv(n_tokens=2 ** 31 - 1)) == BAD
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(c, qkv(eps=eps)) == BAD
    for scale in (float("nan"), float("inf")):
        assert call(c, qkv(rot_scale=scale)) == BAD
    for name in ("q_stride", "k_stride", "v_stride", "q_out_stride"):
        for stride in ((4, 1024, 128), (4096, 1025, 128), (4096, 1024, 132)):
            assert call(c, qkv(**{name: (ctypes.c_int64 * 3)(*stride)})) == BAD
    # the stride of a single batch, token or head does not matter (the call goes on to look for its device)
    one = config(batch=1, n_q_heads=1, n_kv_heads=1, device=63)
    odd = {name: (ctypes.c_int64 * 3)(5, 7, 9) for name in ("q_stride", "k_stride", "v_stride", "q_out_stride")}
    assert call(one, qkv(n_tokens=0, **odd)) == ckv.CKV_OK
    assert call(one, qkv(n_tokens=0, **{**odd, "q": ODD})) == BAD
    f = (ctypes.c_double * 64)(*([1.0] * 63 + [float("inf")]))
    assert call(c, qkv(inv_freq_host=ctypes.cast(f, ctypes.c_void_p))) == BAD
    assert call(c, qkv(n_tokens=0)) == ckv.CKV_OK                       # nothing to do, nothing launched


def test_write_and_read_arguments_checked(L):
    c, s = config(), (ctypes.c_int64 * 3)(4096, 1024, 128)
    C = ctypes.byref
    good = [C(c), 32, P, s, P, s, 3, P, P, P, None]
    for i in (0, 2, 3, 4, 5, 8, 9):
        assert L.ckv_kv4_write(*[None if k == i else x for k, x in enumerate(good)]) == BAD
    for i in (2, 4, 8, 9):
        assert L.ckv_kv4_write(*[ODD if k == i else x for k, x in enumerate(good)]) == BAD
    assert L.ckv_kv4_write(C(c), 48, *good[2:]) == BAD
    assert L.ckv_kv4_write(*good[:6], -1, *good[7:]) == BAD
    assert L.ckv_kv4_write(*good[:6], 101, None, *good[8:]) == BAD      # rows 0 .. 100 of a cache of 100
    assert L.ckv_kv4_write(*good[:6], 0, *good[7:]) == ckv.CKV_OK
    bad_stride = (ctypes.c_int64 * 3)(4096, 1024, 100)
    assert L.ckv_kv4_write(*good[:3], bad_stride, *good[4:]) == BAD
    for bad in BAD_SHAPES:
        assert L.ckv_kv4_write(C(config(**bad)), *good[1:]) == BAD
    good = [C(c), 32, P, P, 0, 100, P, P, None]
    for first, count in ((-1, 5), (0, 101), (100, 1), (0, -1), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert L.ckv_kv4_read(*good[:4], first, count, *good[6:]) == BAD
    assert L.ckv_kv4_read(*good[:6], None, None, None) == BAD
    assert L.ckv_kv4_read(C(c), 32, None, P, 0, 100, P, P, None) == BAD
    assert L.ckv_kv4_read(C(c), 32, P, None, 0, 100, P, P, None) == BAD
    assert L.ckv_kv4_read(C(c), 0, *good[2:]) == BAD
    for i in (2, 3, 6, 7):
        assert L.ckv_kv4_read(*[ODD if k == i else x for k, x in enumerate(good)]) == BAD
    assert L.ckv_kv4_read(*good[:5], 0, *good[6:]) == ckv.CKV_OK


def test_attention_arguments_checked(L):
    c = config()
    C = ctypes.byref
    dense = [C(c), 32, P, P, P, 100, P, P, P, P, None]
    for i in (0, 2, 3, 4, 7, 8):
        assert L.ckv_kv4_dense_decode(*[None if k == i else x for k, x in enumerate(dense)]) == BAD
    for i in (2, 3, 4, 7, 8):
        assert L.ckv_kv4_dense_decode(*[ODD if k == i else x for k, x in enumerate(dense)]) == BAD
    rows = [C(c), 32, P, P, P, 100, P, P, P, 16, P, P, P, None]
    for i in (0, 2, 3, 4, 7, 8, 10, 11):
        assert L.ckv_kv4_attend_rows(*[None if k == i else x for k, x in enumerate(rows)]) == BAD
    for call, good in ((L.ckv_kv4_dense_decode, dense), (L.ckv_kv4_attend_rows, rows)):
        for n in (0, -1, 101):
            assert call(*good[:5], n, *good[6:]) == BAD
        for group in (0, 31, 256):
            assert call(C(c), group, *good[2:]) == BAD
        for bad in BAD_SHAPES + [dict(n_q_heads=18)]:                   # nine query heads of a KV head
            assert call(C(config(**bad)), *good[1:]) == BAD
    for max_rows in (-1, 2 ** 31 - 1):
        assert L.ckv_kv4_attend_rows(*rows[:9], max_rows, *rows[10:]) == BAD
    for bad in (dict(mode=2), dict(n_sinks=-1)):
        assert L.ckv_kv4_attend_rows(C(config(**bad)), *rows[1:]) == BAD


class FakeTensor:
    """Stands in for a tensor of device 0 on a machine without one."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.bfloat16, device=0, strides=None):
        self.t = torch.empty(shape, dtype=dtype, device="meta")
        if strides:
            self.t = self.t.as_strided(shape, strides)
        self.shape, self.dtype, self.device = self.t.shape, dtype, f"cuda:{device}"
        self.index = device

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_checks_tensors(L):
    c = config()
    F, i32, f32 = FakeTensor, torch.int32, torch.float32
    size = ckv.ckv_kv4_bytes(c, 32)
    good = dict(cfg=c, group=32, q=F((2, 8, 128)), K4=F((size,), torch.uint8), V4=F((size,), torch.uint8), n=50,
                lens=F((2,), i32), workspace=F((ckv.ckv_kv4_workspace(c),), torch.uint8), out=F((2, 8, 128), f32),
                lse=F((2, 8), f32))
    wrong = dict(q=[F((2, 8, 128), f32), F((2, 4, 128)), F((2, 8, 128), device=1), F((2, 8, 128), strides=(1024, 1, 8))],
                 K4=[F((size - 1,), torch.uint8)], V4=[F((size,), torch.uint8, device=1)], lens=[F((3,), i32), F((2,), torch.int64)],
                 workspace=[F((16,), torch.uint8)], out=[F((2, 8, 128))], lse=[F((2, 8, 1), f32)])
    for name, values in wrong.items():
        for value in values:
            with pytest.raises(ValueError):
                ckv.ckv_kv4_dense_decode(**{**good, name: value})
    for name in ("q", "K4", "out", "lens", "workspace"):
        for host in (torch.zeros(4), np.zeros(4, np.float32)):
            with pytest.raises(TypeError):
                ckv.ckv_kv4_dense_decode(**{**good, name: host})
    with pytest.raises(ckv.CkvError) as e:                               # the right kinds reach the C call
        ckv.ckv_kv4_dense_decode(**{**good, "n": 0})
    assert e.value.status == BAD
    more = {**good, "rows": F((4, 16), i32), "n_rows": F((4,), i32), "max_rows": 16}
    for name, value in (("rows", F((2, 16), i32)), ("rows", F((4, 8), i32)), ("n_rows", F((2,), i32))):
        with pytest.raises(ValueError):
            ckv.ckv_kv4_attend_rows(**{**more, name: value})

    freq = np.ones(64)
    rows = dict(cfg=c, q=F((2, 3, 8, 128)), k=F((2, 3, 2, 128)), v=F((2, 3, 2, 128)), pos=F((2, 3), i32),
                q_out=F((2, 3, 8, 128)), inv_freq_host=freq, K4=F((size,), torch.uint8), V4=F((size,), torch.uint8), group=32)
    wrong = dict(q=[F((2, 3, 8, 128), f32), F((2, 3, 4, 128)), F((3, 8, 128))], k=[F((2, 3, 8, 128))], v=[F((2, 4, 2, 128))],
                 q_out=[F((2, 3, 8, 128), device=1), F((2, 3, 8, 128), strides=(4096, 1024, 1, 8))], pos=[F((2, 4), i32)],
                 K4=[F((8,), torch.uint8)], q_weight=[F((64,)), F((128,), f32)], K=[F((2, 2, 99, 128))])
    for name, values in wrong.items():
        for value in values:
            with pytest.raises(ValueError):
                ckv.ckv_qk_norm_rope(**{**rows, name: value})
    for name, value in (("q", torch.zeros(4)), ("k", F((2, 3, 2, 128)).t), ("inv_freq_host", np.ones(64, np.float32)),
                        ("inv_freq_host", np.ones(128)[::2]), ("inv_freq_host", F((64,), torch.float64)), ("q", 4096), ("v", None)):
        with pytest.raises(TypeError):
            ckv.ckv_qk_norm_rope(**{**rows, name: value})
    with pytest.raises(ckv.CkvError):
        ckv.ckv_qk_norm_rope(**{**rows, "group": 48, "K4": 4096, "V4": 4096})


def test_reference_format_round_trip():
    rng = np.random.default_rng(3)
    x = ref.to_bf16(rng.standard_normal((2, 3, 20, 128)) * 3)
    for group in (32, 64, 128):
        for values in (False, True):
            buf = ref.cache_of(x, group, values, 21)
            got = ref.values_of(buf, 2, 3, 21, group, values)[:, :, :20]
            c, scale, middle = ref.quantise(x, group)
            bound = np.repeat(scale / 2 + 2.0 ** -9 * np.abs(middle), group, -1)
            assert (np.abs(got - x) <= bound * (1 + 1e-12)).all()


def test_integers_and_lse_on_four_bytes(L):
    # a kernel faults on an address off its type's alignment, so the call refuses it
    c, s, off = config(device=63), (ctypes.c_int64 * 3)(4096, 1024, 128), ctypes.c_void_p(4098)
    C = ctypes.byref
    assert L.ckv_qk_norm_rope(C(c), C(qkv(n_tokens=0)), None) == ckv.CKV_OK
    assert L.ckv_qk_norm_rope(C(c), C(qkv(n_tokens=0, pos=off)), None) == BAD
    write = [C(c), 32, P, s, P, s, 0, P, P, P, None]
    assert L.ckv_kv4_write(*write) == ckv.CKV_OK
    assert L.ckv_kv4_write(*write[:7], off, *write[8:]) == BAD
    for i in (6, 9):
        dense = [C(c), 32, P, P, P, 100, P, P, P, P, None]
        assert L.ckv_kv4_dense_decode(*[off if k == i else x for k, x in enumerate(dense)]) == BAD
    for i in (6, 7, 8, 12):
        rows = [C(c), 32, P, P, P, 100, P, P, P, 16, P, P, P, None]
        assert L.ckv_kv4_attend_rows(*[off if k == i else x for k, x in enumerate(rows)]) == BAD


class EmptyTensor(FakeTensor):
    """A tensor without elements has no address."""

    def data_ptr(self):
        return 0


def test_no_tokens(L):
    # a chunk of no tokens is an empty tensor, and nothing to do
    c, E = config(), EmptyTensor
    size = ckv.ckv_kv4_bytes(c, 32)
    four = [FakeTensor((size,), torch.uint8) for _ in range(2)]
    q, k, pos = E((2, 0, 8, 128)), E((2, 0, 2, 128)), E((2, 0), torch.int32)
    ckv.ckv_qk_norm_rope(c, q, k, k, pos, q, np.ones(64), K4=four[0], V4=four[1], group=32)
    ckv.ckv_kv4_write(c, 32, k, k, pos, *four)
    ckv.ckv_kv4_write(c, 32, k, k, None, *four)
    x = {name: None for name in ("q", "k", "v", "pos", "q_out")}
    assert L.ckv_qk_norm_rope(ctypes.byref(c), ctypes.byref(qkv(n_tokens=0, **x)), None) == ckv.CKV_OK
    assert L.ckv_qk_norm_rope(ctypes.byref(c), ctypes.byref(qkv(n_tokens=0, group=48, **x)), None) == BAD


def test_binding_names_what_is_wrong_with_rows_and_types(L):
    # the kinds of error that the other arguments raise
    c, F, i32 = config(), FakeTensor, torch.int32
    size = ckv.ckv_kv4_bytes(c, 32)
    four = [F((size,), torch.uint8) for _ in range(2)]
    q, k, pos = F((2, 3, 8, 128)), F((2, 3, 2, 128)), F((2, 3), i32)
    for bad, error in ((None, TypeError), (4096, TypeError), (np.zeros((2, 3, 2, 128)), TypeError), (torch.zeros((2, 3, 2, 128)), TypeError),
                       (F((128,)), ValueError), (F(()), ValueError)):
        with pytest.raises(error):
            ckv.ckv_qk_norm_rope(c, q, bad, k, pos, q, np.ones(64), K4=four[0], V4=four[1], group=32)
        with pytest.raises(error):
            ckv.ckv_kv4_write(c, 32, bad, k, pos, *four)
    c = config(kv_dtype=7)
    f32 = torch.float32
    out, work = F((2, 8, 128), f32), F((1 << 20,), torch.uint8)
    for call in (lambda: ckv.ckv_qk_norm_rope(c, q, k, k, pos, q, np.ones(64), K4=four[0], V4=four[1], group=32),
                 lambda: ckv.ckv_kv4_write(c, 32, k, k, pos, *four),
                 lambda: ckv.ckv_kv4_read(c, 32, *four, 0, 1, F((2, 2, 100, 128)), None),
                 lambda: ckv.ckv_kv4_dense_decode(c, 32, F((2, 8, 128)), *four, 50, None, work, out),
                 lambda: ckv.ckv_kv4_attend_rows(c, 32, F((2, 8, 128)), *four, 50, None, F((4, 16), i32), F((4,), i32), 16, work, out)):
        with pytest.raises(ValueError):
            call()


def test_queries_over_themselves(L):
    # rows written by one warp while another still has to read them, or twice: refused, not raced
    c = config()
    Q, S3 = ctypes.c_void_p(8192), ctypes.c_int64 * 3
    call = lambda **kw: L.ckv_qk_norm_rope(ctypes.byref(c), ctypes.byref(qkv(n_tokens=0, **kw)), None)  # noqa: E731
    assert call() == ckv.CKV_OK                                          # in place
    assert call(q_out=Q, q_out_stride=S3(4096, 1024, 256)) == ckv.CKV_OK  # elsewhere, other strides
    for stride in ((8192, 1024, 128), (4096, 1024, 256)):
        assert call(q_out_stride=S3(*stride)) == BAD
    for stride in ((0, 1024, 128), (4096, 1024, 0)):
        assert call(q_out=Q, q_out_stride=S3(*stride)) == BAD
    assert call(q_out_stride=S3(4096, 0, 128)) == ckv.CKV_OK              # one that takes no part: there are no two tokens
