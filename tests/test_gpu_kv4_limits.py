"""Decode attention over a 4-bit cache and rows into the caches on the GPU, at
the borders of what they take: buffers shared by calls of different shapes,
weights and scales far below the largest, logits and keys far from 1, channels
that are not finite."""
import numpy as np
import pytest
import torch

import long_context_decode_ckv_b200 as ckv
from long_context_decode_ckv_b200 import build as ckv_build
from tests.conftest import gpu_available
from tests.test_gpu_kv4 import Case

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
