"""GPU parity of kv_cache_write and kv_cache_read with the oracle's quantizers
and dequantizers, row by row: same bytes, same values."""
import numpy as np
import pytest
import torch

from helpers import NAME_DT, raw
from kv_reference import distinct_slots, seeded

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
G_K, G_V = 9.0, 3.5


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def new_cache(nv, mode, pages, heads, page_size, D, use_g=True, fill=0xA5):
    g = [torch.tensor([x], device="cuda") for x in (G_K, G_V)] if mode == "nvfp4" and use_g else [None, None]
    c = nv.KvCache.empty(mode, pages, heads, page_size, D, *g)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.view(torch.uint8).fill_(fill)
    return c


def oracle_rows(orc, mode, x, g):
    """(codes [T, heads, words], scales [T, heads, blocks]) as raw numpy."""
    T, H, D = x.shape
    r, dt = np.ascontiguousarray(raw(x.contiguous())).reshape(T * H, D), NAME_DT[x.dtype]
    if mode == "nvfp4":
        c, s = orc.nvfp4_quantize(r, dt, g)
    else:
        c, s = (orc.mxfp8_quantize if mode == "mxfp8" else orc.mxfp4_quantize)(r, dt)
    return c.reshape(T, H, -1), s.reshape(T, H, -1)


def rows_of(t, slots, page_size):
    """numpy [T, heads, ...] of a cache tensor at slots (numpy)."""
    n = raw(t)
    return n[slots // page_size, :, slots % page_size]


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("T,heads,D,page_size", [(1, 8, 128, 16), (37, 3, 96, 24), (130, 1, 32, 7), (65, 5, 256, 64),
                                                 (300, 2, 64, 1)])
def test_write_gives_the_quantizers_bytes(nv, orc, mode, dtype, T, heads, D, page_size):
    pages = (2 * T) // page_size + 2
    c = new_cache(nv, mode, pages, heads, page_size, D, use_g=T != 65)
    k, v = seeded((T, heads, D), T, dtype, 3.0), seeded((T, heads, D), T + 1, dtype)
    k[0, 0, :32] = 0  # a block of zeros
    v[T // 2, -1, 5] = 700.0  # far beyond g: saturates
    slots = distinct_slots(T, pages * page_size, T)
    nv.kv_cache_write(c, k, v, slots.cuda())
    nv.check_device_errors()
    s = slots.numpy()
    for x, codes, scales, g in ((k, c.k_codes, c.k_scales, c.g_k), (v, c.v_codes, c.v_scales, c.g_v)):
        oc, os_ = oracle_rows(orc, mode, x, None if g is None else float(g))
        assert np.array_equal(rows_of(codes, s, page_size), oc)
        assert np.array_equal(rows_of(scales, s, page_size), os_)
        rest = np.ones(pages * page_size, dtype=bool)
        rest[s] = False
        rest = np.nonzero(rest)[0]
        assert (rows_of(codes, rest, page_size) == 0xA5A5A5A5).all()  # every other row as it was
        assert (rows_of(scales, rest, page_size) == 0xA5).all()


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
def test_read_gives_the_dequantizers_values(nv, orc, mode, dtype):
    T, heads, D, page_size, pages = 83, 3, 96, 24, 9
    c = new_cache(nv, mode, pages, heads, page_size, D)
    k, v = seeded((T, heads, D), 4, bf16, 3.0), seeded((T, heads, D), 5, bf16)
    slots = distinct_slots(T, pages * page_size, 6)
    nv.kv_cache_write(c, k, v, slots.cuda())
    again = torch.cat([slots[:10], slots.flip(0), slots[:1]])  # any order, repeated
    ko, vo = nv.kv_cache_read(c, again.cuda(), dtype)
    nv.check_device_errors()
    name = NAME_DT[dtype]
    for x, o, g in ((k, ko, c.g_k), (v, vo, c.g_v)):
        oc, os_ = oracle_rows(orc, mode, x, None if g is None else float(g))
        oc, os_ = oc.reshape(T * heads, -1), os_.reshape(T * heads, -1)
        want = (orc.nvfp4_dequantize(oc, os_, float(g), name) if mode == "nvfp4" else
                (orc.mxfp8_dequantize if mode == "mxfp8" else orc.mxfp4_dequantize)(oc, os_, name)).reshape(T, heads, D)
        at = np.concatenate([np.arange(10), np.arange(T)[::-1], [0]])
        assert np.array_equal(raw(o).view(np.uint8), np.ascontiguousarray(want[at]).view(np.uint8))


def test_parts_of_a_projection_are_taken_as_they_lie(nv):
    T, heads, D, page_size = 45, 4, 64, 16
    qkv = seeded((T, 4 * heads, D), 8, bf16)
    k, v = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
    slots = distinct_slots(T, 8 * page_size, 9).cuda()
    a, b = new_cache(nv, "nvfp4", 8, heads, page_size, D), new_cache(nv, "nvfp4", 8, heads, page_size, D)
    nv.kv_cache_write(a, k, v, slots)
    nv.kv_cache_write(b, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    assert torch.equal(a.k_scales, b.k_scales) and torch.equal(a.v_scales, b.v_scales)
    # rows that begin at odd multiples of 16 bytes
    odd = torch.empty(T, heads * D + 8, dtype=bf16, device="cuda")
    ko, vo = odd[:, 8:].unflatten(1, (heads, D)), odd.clone()[:, 8:].unflatten(1, (heads, D))
    ko.copy_(k)
    vo.copy_(v)
    nv.kv_cache_write(a, ko, vo, slots)
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes)
    flat = torch.empty(2 * T * heads * D + 8, dtype=bf16, device="cuda")[8:]
    outs = flat[:T * heads * D].view(T, heads, D), flat[T * heads * D:].view(T, heads, D)
    nv.kv_cache_read(a, slots, k_out=outs[0], v_out=outs[1])
    want = nv.kv_cache_read(b, slots, bf16)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # every second token of a longer tensor, and one token broadcast over T
    nv.kv_cache_write(a, k[::2], v[::2], slots[::2].contiguous())
    assert torch.equal(a.k_codes, b.k_codes)
    with pytest.raises(nv.Nvfp4Error, match="strides"):
        nv.kv_cache_write(a, k[:1].expand(T, heads, D), v, slots)


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
def test_skipped_and_out_of_range_slots(nv, mode):
    heads, D, page_size, pages = 2, 64, 16, 3
    c = new_cache(nv, mode, pages, heads, page_size, D)
    k, v = seeded((5, heads, D), 1, bf16), seeded((5, heads, D), 2, bf16)
    nv.kv_cache_write(c, k, v, torch.tensor([-1, 3, -7, -2 ** 31, 47], dtype=torch.int32, device="cuda"))
    nv.check_device_errors()
    touched = (c.k_scales != 0xA5).any(-1).any(1)  # [pages, page_size]
    assert touched.nonzero().tolist() == [[0, 3], [2, 15]]
    ko, vo = nv.kv_cache_read(c, torch.tensor([3, -1, 47], dtype=torch.int32, device="cuda"), f32)
    nv.check_device_errors()
    assert ko[1].abs().sum() == 0 and vo[1].abs().sum() == 0 and ko[0].abs().sum() > 0 and vo[2].abs().sum() > 0
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    nv.kv_cache_write(c, k[:2], v[:2], torch.tensor([48, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.check_device_errors()
    assert e.value.status == nv.ERR_DEVICE_INDEX
    assert all(torch.equal(x, y) for x, y in zip(before, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)))
    ko, vo = nv.kv_cache_read(c, torch.tensor([48, 3], dtype=torch.int32, device="cuda"), f32)
    with pytest.raises(nv.Nvfp4Error):
        nv.check_device_errors()
    assert ko[0].abs().sum() == 0 and vo[0].abs().sum() == 0 and ko[1].abs().sum() > 0


def test_no_tokens(nv):
    c = new_cache(nv, "mxfp4", 2, 2, 16, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 2, 64, dtype=bf16, device="cuda")
    nv.kv_cache_write(c, x, x, none)
    ko, vo = nv.kv_cache_read(c, none)
    assert ko.shape == (0, 2, 64) and vo.shape == (0, 2, 64)


def test_rows_past_four_gigabytes(nv):
    """9 GB of cache: the last page's rows lie past 2^32 bytes of codes."""
    heads, D, page_size = 8, 128, 64
    pages = (1 << 32) // (heads * page_size * D // 2) + 3
    c = nv.KvCache.empty("nvfp4", pages, heads, page_size, D)
    T = 2 * page_size
    k, v = seeded((T, heads, D), 1, bf16), seeded((T, heads, D), 2, bf16)
    slots = torch.arange((pages - 2) * page_size, pages * page_size, dtype=torch.int32, device="cuda")
    low = torch.arange(T, dtype=torch.int32, device="cuda")
    nv.kv_cache_write(c, v, k, low)  # what a wrapped offset would hit
    nv.kv_cache_write(c, k, v, slots)
    small = nv.KvCache.empty("nvfp4", 2, heads, page_size, D)
    nv.kv_cache_write(small, k, v, low)
    got, want = nv.kv_cache_read(c, slots, f32), nv.kv_cache_read(small, low, f32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(nv.kv_cache_read(c, low, f32)[0], want[1])
    q = seeded((1, 32, D), 3, bf16)
    args = dict(kv_len=torch.tensor([T], dtype=torch.int32, device="cuda"))
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    assert torch.equal(nv.kv_attention(c, q, table, **args), nv.kv_attention(small, q, table - (pages - 2), **args))
    nv.check_device_errors()
