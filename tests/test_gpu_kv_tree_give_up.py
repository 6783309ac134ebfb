"""A wait that runs out in the attention kernel for trees of drafts ends in the
device error word; the other CTAs' results stay right (as
test_gpu_kv_give_up.py has it for the kernels without masks)."""
import ctypes
import os
import subprocess

import pytest
import torch

from kv_reference import seeded
from tree_reference import ancestors, pack

pytestmark = pytest.mark.gpu

TIMEOUT = 2


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


@pytest.fixture(scope="module")
def give_up(tmp_path_factory):
    from mxfp8_block_scaled_nvfp4_b200 import build
    out = str(tmp_path_factory.mktemp("tree_give_up") / "libkv_tree_give_up.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.check_call([build.NVCC, *build.FLAGS, "-DNVFP4_WAIT_LIMIT=1048576u", "-DNVFP4_TEST_WITHHOLD_STAGE=g_withheld",
                           "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(here, "kv_tree_give_up.cu"), "-o", out])
    L = ctypes.CDLL(out)
    L.kv_give_up.argtypes = [ctypes.c_int] * 2 + [ctypes.c_void_p] * 11 + [ctypes.c_uint32] * 6 + [ctypes.c_void_p]
    return L


# one query tile (25 x 4 rows) of one token tile, of two and of four in two slots; two query tiles
@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("n,L", [(25, 100), (25, 200), (25, 500), (64, 500)])
def test_a_wait_that_runs_out_ends_in_the_error_word(nv, give_up, mode, n, L):
    B, heads, G, D = 3, 2, 4, 64
    cache = nv.KvCache.empty(mode, B, heads, L, D)
    nv.kv_cache_write(cache, seeded((B * L, heads, D), 1), seeded((B * L, heads, D), 2), torch.arange(B * L, dtype=torch.int32, device="cuda"))
    q = seeded((B * n, heads * G, D), 3)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    kv_len = torch.full((B,), L, dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    mask = pack([m for b in range(B) for m in ancestors(n, b)], 2).cuda()
    want, want_lse = nv.kv_attention_tree(cache, q, table, kv_len, mask, starts, n, L, return_lse=True,
                                          workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    nv.check_device_errors()
    mine = torch.zeros(B * n, heads * G, dtype=torch.bool, device="cuda")  # CTA 0: sequence 0, head 0
    mine[:n, :G] = True

    def run(withheld):
        out, lse = torch.full_like(q, 7.0), torch.full((B * n, heads * G), 7.0, device="cuda")
        st = give_up.kv_give_up(mode == "mxfp8", withheld, *(t.data_ptr() for t in (
            cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, q, starts, kv_len, table, mask, out, lse)),
            B, n, L, heads, G, 2, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        return give_up.kv_give_up_word(), out, lse

    word, out, lse = run(-1)
    assert word == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    for withheld in range(-(-L // 128)):
        word, out, lse = run(withheld)
        assert word == TIMEOUT
        assert torch.equal(out[~mine], want[~mine]) and torch.equal(lse[~mine], want_lse[~mine])
    word, out, lse = run(-1)  # the device serves on
    assert word == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
