"""Values and arguments at the edges of kv_attention's contract, on both of its
kernels: one query row goes through k_kv_decode, forty a key/value head through
k_kv_prefill."""
import math

import pytest
import torch

from kv_reference import attention, cache_sides, check, seeded
from test_gpu_kv_attention import compare, i32, make, nv  # noqa: F401 (nv is a fixture)

pytestmark = pytest.mark.gpu

bf16, f16 = torch.bfloat16, torch.float16
MODES = ["nvfp4", "mxfp4", "mxfp8"]


def no_workspace():
    return torch.empty(0, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("L", [90, 5000])
def test_a_nan_query_gives_nan_and_leaves_the_others(nv, mode, dtype, n, L):
    lens, G = [L, 50], 4
    c, table = make(nv, mode, lens, 2, 64, 16, 91)
    q = seeded((2 * n, 2 * G, 64), 5, dtype)
    starts = [0, n, 2 * n]
    want, want_lse = compare(nv, c, table, lens, q, starts, n, L)
    for element in (3, slice(None)):
        p = q.clone()
        p[n // 2, 1, element] = float("nan")
        for kw in ({}, {"workspace": no_workspace()}):
            out, lse = nv.kv_attention(c, p, table, i32(lens), i32(starts), n, L, return_lse=True, **kw)
            nv.check_device_errors()
            assert torch.isnan(out[n // 2, 1]).all() and torch.isnan(lse[n // 2, 1])
            rest = torch.ones(2 * n, 2 * G, dtype=torch.bool, device="cuda")
            rest[n // 2, 1] = False
            assert torch.isfinite(out[rest].float()).all() and torch.isfinite(lse[rest]).all()
            if not kw:
                assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
