"""The give-up path of the attention kernels over the key/value cache.

A wait that runs out ends the CTA, not the GPU's usefulness: every warp of it
comes to the end, whatever the others have given up, the error word is set and
the other CTAs' results stand.  A small test library (kv_give_up.cu, low wait
limit) never hands over one unit or value tile of CTA 0.
"""
import ctypes
import os
import subprocess

import pytest
import torch

from kv_reference import seeded

pytestmark = pytest.mark.gpu

TIMEOUT = 2  # kDevErrTimeout


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


@pytest.fixture(scope="module")
def give_up(tmp_path_factory):
    from mxfp8_block_scaled_nvfp4_b200 import build
    out = str(tmp_path_factory.mktemp("give_up") / "libkv_give_up.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.check_call([build.NVCC, *build.FLAGS, "-DNVFP4_WAIT_LIMIT=1048576u", "-DNVFP4_TEST_WITHHOLD_STAGE=g_withheld",
                           "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(here, "kv_give_up.cu"), "-o", out])
    L = ctypes.CDLL(out)
    L.kv_give_up.argtypes = [ctypes.c_int] * 3 + [ctypes.c_void_p] * 10 + [ctypes.c_uint32] * 6 + [ctypes.c_void_p]
    return L


# (queries, tokens): k_kv_decode, k_kv_prefill with one and two query tiles a CTA and one to four value tiles
@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("n,L", [(1, 300), (1, 320), (25, 100), (25, 500), (64, 100), (64, 500)])
def test_a_wait_that_runs_out_ends_in_the_error_word(nv, give_up, mode, n, L):
    B, heads, G, D = 3, 2, 4, 64
    cache = nv.KvCache.empty(mode, B, heads, L, D)
    nv.kv_cache_write(cache, seeded((B * L, heads, D), 1), seeded((B * L, heads, D), 2),
                      torch.arange(B * L, dtype=torch.int32, device="cuda"))
    q = seeded((B * n, heads * G, D), 3)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    kv_len = torch.full((B,), L, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    want, want_lse = nv.kv_attention(cache, q, table, kv_len, starts, n, L, causal=False, return_lse=True,
                                     workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    nv.check_device_errors()
    prefill = n * G > 32
    mine = torch.zeros(B * n, heads * G, dtype=torch.bool, device="cuda")  # CTA 0: sequence 0, head 0, the last row tile
    mine[:n, :G] = True

    def run(withheld):
        out, lse = torch.full_like(q, 7.0), torch.full((B * n, heads * G), 7.0, device="cuda")
        st = give_up.kv_give_up(prefill, mode == "mxfp8", withheld, *(t.data_ptr() for t in (
            cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, q, starts, kv_len, table, out, lse)),
            B, n, L, heads, G, L, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        return give_up.kv_give_up_word(), out, lse

    word, out, lse = run(-1)
    assert word == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    tiles = -(-L // 128)
    for withheld in {0, tiles - 1}:
        word, out, lse = run(withheld)
        assert word == TIMEOUT
        assert torch.equal(out[~mine], want[~mine]) and torch.equal(lse[~mine], want_lse[~mine])
    word, out, lse = run(-1)  # the device serves on
    assert word == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
