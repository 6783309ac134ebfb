"""Host-side checks of the key/value cache calls (no GPU): bad arguments are
refused before any device call, good ones reach the device query."""
import ctypes

import pytest
import torch

from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv

A = 0x10000  # a fake, 16-byte aligned device address: never dereferenced
N0 = None
INF = float("inf")


@pytest.fixture(scope="module")
def L():
    from mxfp8_block_scaled_nvfp4_b200 import build
    build.build()
    return nv.lib()


def msg(L):
    return L.nvfp4_last_error_message().decode()


def cache(mode=0, pages=8, page_size=16, heads=2, D=64, k=A, ks=A, v=A, vs=A, g_k=N0, g_v=N0):
    return ctypes.byref(nv.KvCacheArgs(mode, pages, page_size, heads, D, k, ks, v, vs, g_k, g_v))


def write(L, c, k=A, v=A, dt=2, T=3, ks=128, vs=128, slots=A):
    return L.kv_cache_write(c, k, v, dt, T, ks, vs, slots, N0)


def attend(L, c, q=A, dt=2, stride=256, q_start=N0, kv_len=A, table=A, B=2, T=2, Hq=4, max_q=1, max_kv=64, max_pages=4,
           scale=0.1, causal=1, window=0, out=A, lse=N0, ws=N0, ws_bytes=0):
    return L.kv_attention(c, q, dt, stride, q_start, kv_len, table, B, T, Hq, max_q, max_kv, max_pages, scale, causal,
                          window, out, lse, ws, ws_bytes, N0)


def needs_device(st):
    return st not in (0, 1, 2)


@pytest.mark.parametrize("call", [write, attend, lambda L, c: L.kv_cache_read(c, A, 3, A, A, 2, N0)])
def test_the_cache_handle_is_checked(L, call):
    assert needs_device(call(L, cache()))
    assert needs_device(call(L, cache(g_k=A, g_v=A)))
    assert call(L, N0) == 1 and "null cache" in msg(L)
    assert call(L, cache(mode=3)) == 1 and "mode" in msg(L)
    assert call(L, cache(mode=1, g_k=A, g_v=A)) == 1 and "only supported for 'nvfp4'" in msg(L)
    assert call(L, cache(g_k=A)) == 1 and "or neither" in msg(L)
    assert call(L, cache(page_size=0)) == 1
    assert call(L, cache(pages=-1)) == 1
    assert call(L, cache(pages=1 << 27, page_size=16)) == 1 and "2^31" in msg(L)
    assert call(L, cache(pages=1 << 62, page_size=4)) == 1  # the product would wrap
    assert call(L, cache(heads=0)) == 1 and call(L, cache(heads=65536)) == 1
    assert call(L, cache(D=0)) == 1 and call(L, cache(D=48)) == 1 and "multiple of 32" in msg(L)
    assert call(L, cache(D=288)) == 2 and "at most 256" in msg(L)
    assert call(L, cache(k=N0)) == 1 and call(L, cache(vs=N0)) == 1 and "null" in msg(L)
    assert call(L, cache(v=A + 8)) == 1 and "16-byte" in msg(L)
    assert call(L, cache(g_k=A + 2, g_v=A)) == 1


def test_write_and_read_arguments(L):
    c = cache()
    assert write(L, c, dt=7) == 2
    assert write(L, c, T=-1) == 1 and write(L, c, T=1 << 62) == 1
    assert write(L, c, k=N0) == 1 and write(L, c, slots=N0) == 1
    assert write(L, c, v=A + 4) == 1 and write(L, c, slots=A + 2) == 1
    assert write(L, c, ks=127) == 1 and write(L, c, vs=130) == 1 and "stride" in msg(L)
    assert needs_device(write(L, c, ks=136)) and needs_device(write(L, c, T=1, ks=0, vs=5))
    assert needs_device(write(L, c, dt=0, ks=132, vs=132))
    assert write(L, c, dt=0, ks=130) == 1
    assert write(L, c, T=0, k=N0, v=N0, slots=N0) == 0
    assert L.kv_cache_read(c, N0, 0, N0, N0, 2, N0) == 0
    assert L.kv_cache_read(c, A, 3, A, A, 9, N0) == 2
    assert L.kv_cache_read(c, A, 3, N0, A, 2, N0) == 1
    assert L.kv_cache_read(c, A, 3, A, A + 8, 2, N0) == 1
    assert L.kv_cache_read(c, A, -3, A, A, 2, N0) == 1
    assert write(L, cache(pages=0, k=N0, ks=N0, v=N0, vs=N0), T=0, k=N0, v=N0, slots=N0) == 0


def test_attention_arguments(L):
    c = cache()
    assert attend(L, c, dt=0) == 2 and "float16 or bfloat16" in msg(L)
    assert attend(L, c, Hq=3) == 1 and "multiple" in msg(L)
    assert attend(L, c, Hq=0) == 1 and attend(L, c, B=65536, T=65536) == 1 and attend(L, c, T=-1) == 1
    assert attend(L, c, T=3) == 1 and "q_start" in msg(L)
    assert attend(L, c, max_q=2) == 1
    assert attend(L, c, max_kv=65) == 1 and "max_kv" in msg(L)
    assert attend(L, cache(page_size=1 << 20), max_kv=(1 << 30) + 1, max_pages=2048) == 2 and "2^30" in msg(L)
    assert attend(L, c, max_kv=-1) == 1 and attend(L, c, window=-1) == 1
    assert attend(L, c, scale=INF) == 1 and attend(L, c, scale=float("nan")) == 1
    assert attend(L, c, stride=255) == 1 and attend(L, c, stride=260) == 1
    for bad in ("q", "out", "kv_len", "table"):
        assert attend(L, c, **{bad: N0}) == 1 and "null" in msg(L)
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(kv_len=A + 1), dict(table=A + 2), dict(q_start=A + 2),
                dict(ws=A + 8, ws_bytes=64)):
        assert attend(L, c, **bad) == 1 and "aligned" in msg(L)
    assert attend(L, c, ws_bytes=64) == 1
    assert attend(L, c, T=1 << 30, q_start=A, B=1, max_q=1, Hq=65534) == 1  # T*Hq*D
    assert attend(L, c, B=0, T=0, q=N0, out=N0, kv_len=N0, table=N0) == 0
    assert attend(L, c, q_start=A, max_q=0) == 0
    assert needs_device(attend(L, c)) and needs_device(attend(L, c, q_start=A, T=9, max_q=4))
    assert needs_device(attend(L, c, max_kv=0, max_pages=0, table=N0))
    assert needs_device(attend(L, c, window=1 << 40)) and needs_device(attend(L, c, max_pages=(1 << 31) - 1))


def test_workspace_size(L):
    size = nv.kv_attention_workspace_size
    for bad in ((-1, 1, 4, 1, 64, 1, 100), (1, 1, 4, 3, 64, 1, 100), (1, 1, 4, 1, 48, 1, 100), (1, 1, 4, 1, 288, 1, 100),
                (1, 1, 4, 1, 64, 1, -1), (1, 1, 4, 0, 64, 1, 100), (1, 1 << 62, 4, 1, 64, 1, 100), (1, 1, 4, 1, 64, 1, 100, -1)):
        assert size(*bad) == 0
    assert size(1, 1, 32, 8, 128, 1, 16) == 0  # nothing to split
    assert size(512, 512, 32, 8, 128, 1, 1 << 20) <= 1 << 32


def e(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype)


def test_binding_refuses_what_a_pointer_would_hide():
    i32, bf16 = torch.int32, torch.bfloat16
    with pytest.raises(ValueError, match="mode"):
        nv.KvCache("fp4", e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 4), e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 4))
    with pytest.raises(ValueError, match="k_scales"):
        nv.KvCache("nvfp4", e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 2), e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 4))
    with pytest.raises(ValueError, match="v_codes"):
        nv.KvCache("mxfp4", e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 2), e(4, 2, 16, 16, dtype=i32), e(4, 2, 16, 2))
    with pytest.raises(ValueError, match="int32"):
        nv.KvCache("mxfp4", e(4, 2, 16, 8), e(4, 2, 16, 2), e(4, 2, 16, 8, dtype=i32), e(4, 2, 16, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        nv.KvCache("mxfp8", e(4, 2, 16, 16, dtype=i32), e(4, 2, 16, 2), e(4, 2, 16, 16, dtype=i32), e(4, 2, 16, 2))
    with pytest.raises(ValueError, match="heads and D"):
        nv._need_rows(_OnDevice((3, 2, 64), (256, 128, 1)), (3, 2, 64), "k", 0)
    nv._need_rows(_OnDevice((3, 2, 64), (999, 64, 1)), (3, 2, 64), "k", 0)
    with pytest.raises(ValueError, match=r"must be \(3, 2, 64\)"):
        nv._need_rows(_OnDevice((3, 2, 32), (64, 32, 1)), (3, 2, 64), "k", 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        nv._need_rows(_OnDevice((3, 2, 64), (128, 64, 1), 1), (3, 2, 64), "k", 0)


class _OnDevice:
    """Stand-in for a CUDA tensor (no GPU here)."""
    is_cuda = True

    def __init__(self, shape, strides, index=0):
        self.shape, self._strides, self.device = shape, strides, torch.device("cuda", index)

    def numel(self):
        return self.shape[0] * self.shape[1] * self.shape[2]

    def stride(self):
        return self._strides


@pytest.fixture(autouse=True)
def _device_zero(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
