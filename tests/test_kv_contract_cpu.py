"""Host-side contract of the key/value cache calls that no GPU is needed for."""
import pytest
import torch

from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv
from test_kv_cpu import A, L, attend, cache, msg, needs_device  # noqa: F401 (L is a fixture)


def test_max_q_beyond_all_queries_is_all_queries(L):
    size = nv.kv_attention_workspace_size
    for T in (9, 100, 300):
        for loose in (T + 1, 1 << 20, 1 << 30):
            assert size(1, T, 32, 8, 128, loose, 8192) == size(1, T, 32, 8, 128, T, 8192) > 0
            # the grids' limits
            assert needs_device(attend(L, cache(heads=64), q_start=A, T=T, Hq=256, stride=256 * 64, max_q=loose)), msg(L)
            assert needs_device(attend(L, cache(mode=1), dt=1, q_start=A, T=T, max_q=loose, max_kv=1024, max_pages=64)), msg(L)
