"""Host-side contract of the key/value cache calls that no GPU is needed for."""
import importlib.util
import types

import pytest
import torch

from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv
from test_kv_cpu import A, L, attend, cache, msg, needs_device, write  # noqa: F401 (L is a fixture)


def test_max_q_beyond_all_queries_is_all_queries(L):
    size = nv.kv_attention_workspace_size
    for T in (9, 100, 300):
        for loose in (T + 1, 1 << 20, 1 << 30):
            assert size(1, T, 32, 8, 128, loose, 8192) == size(1, T, 32, 8, 128, T, 8192) > 0
            # the grids' limits
            assert needs_device(attend(L, cache(heads=64), q_start=A, T=T, Hq=256, stride=256 * 64, max_q=loose)), msg(L)
            assert needs_device(attend(L, cache(mode=1), dt=1, q_start=A, T=T, max_q=loose, max_kv=1024, max_pages=64)), msg(L)


def decode_bytes(rows, D):
    """k_kv_decode: 592 workers, two partial results of a row tile and 32 bytes each."""
    tile = 8 if rows <= 8 or D > 128 else 16
    return 592 * (2 * tile * (4 * D + 8) + 32)


@pytest.mark.parametrize("args,want", [
    # B, T, Hq, heads, D, max_q, max_kv, window
    ((1, 1, 32, 8, 128, 1, 64), 0),                                    # one unit of tokens: nothing to split
    ((1, 1, 32, 8, 128, 1, 65), decode_bytes(4, 128)),
    ((32, 32, 32, 8, 128, 1, 32768), decode_bytes(4, 128)),            # the same for any batch and length
    ((8, 8, 16, 8, 256, 1, 6000), decode_bytes(2, 256)),
    ((2, 6, 32, 8, 128, 3, 5000), decode_bytes(12, 128)),
    # one sequence of 100 queries, group 4: 8 heads x 2 tiles of 256 rows, 8192 * 16 / 148 = 885.6 tokens a CTA, so
    # chunks of 896: 10 of them
    ((1, 100, 32, 8, 128, 100, 8192), 10 * 100 * 32 * (4 * 128 + 8)),
    # 8 x 300 over 2500 and the like: 320 tiles, more than there are SMs, so not split
    ((8, 2400, 32, 8, 128, 300, 2500), decode_bytes(1200, 128)),
    # a window of 1024 leaves 1024 + 100 + 30 tokens, at least 512 a chunk
    ((1, 100, 32, 8, 128, 100, 8192, 1024), max(3 * 100 * 32 * (4 * 128 + 8), decode_bytes(400, 128))),
])
def test_workspace_sizes(L, args, want):
    assert nv.kv_attention_workspace_size(*args) == want


def test_token_strides_end_at_2_to_the_31(L):
    c = cache()
    for big, ok in ((2 ** 31 - 8, True), (2 ** 31, False), (2 ** 62, False)):
        assert needs_device(write(L, c, ks=big, vs=big)) == ok and needs_device(attend(L, c, stride=big)) == ok
        assert needs_device(write(L, c, T=1, ks=big, vs=big)) and needs_device(attend(L, c, q_start=A, B=1, T=1, stride=big))


def host_cache(monkeypatch, mode="nvfp4"):
    """A handle over host tensors (no call is made with it)."""
    monkeypatch.setattr(nv, "_need_cuda", lambda *ts: None)
    g = [torch.ones(1), torch.ones(1)] if mode == "nvfp4" else [None, None]
    return nv.KvCache.empty(mode, 4, 2, 16, 64, *g, device="cpu")


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
def test_a_cache_handle_cannot_be_given_other_tensors(monkeypatch, mode):
    """The library reads the addresses the handle was made with."""
    c = host_cache(monkeypatch, mode)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "g_k", "g_v", "mode", "num_pages", "page_size", "heads", "D",
                 "device", "_args", "_ref", "anything"):
        before = getattr(c, name, None)
        with pytest.raises(AttributeError, match="cannot be set"):
            setattr(c, name, torch.ones(1))
        assert getattr(c, name, None) is before
    with pytest.raises(AttributeError):
        del c.k_codes
    assert c._args.k_codes == c.k_codes.data_ptr() and c._args.v_scales == c.v_scales.data_ptr()
    assert c._args.g_k == (c.g_k.data_ptr() if mode == "nvfp4" else None)
    assert (c._args.D, c._args.heads, c._args.page_size, c._args.num_pages) == (64, 2, 16, 4)


def test_the_stream_without_torchs_private_accessor(monkeypatch):
    """_stream() serves every call of the binding and must not depend on a name
    that torch does not promise."""
    spec = importlib.util.find_spec(nv.__name__)
    for private in (True, False):
        if private:
            monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
        else:
            monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
            monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=2000 + device))
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
        assert m._stream().value == (1003 if private else 2003)
