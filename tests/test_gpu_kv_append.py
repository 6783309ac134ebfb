"""GPU parity of kv_cache_append and kv_cache_move: rotated queries and the
cache's bytes are those of the definition's fp32 steps and the oracle's
quantizers; moves are compared with the same moves made one by one."""
import numpy as np
import pytest
import torch

from helpers import raw
from kv_reference import distinct_slots, seeded
from test_gpu_kv_cache import G_K, G_V, new_cache, oracle_rows, rows_of

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def table(rot, most=300, base=10000.0):
    a = torch.arange(most, dtype=torch.float64)[:, None] * base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return a.cos().float().cuda(), a.sin().float().cuda()


def turned(x, cos, sin, positions, interleaved):
    """fp32 on the CPU, every product and sum rounded."""
    x, p = x.float().cpu(), positions.cpu().long()
    c, s, rot = cos.cpu()[p][:, None], sin.cpu()[p][:, None], 2 * cos.shape[1]
    out = x.clone()
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    out[..., i], out[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return out


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,heads,D,rot,page_size", [(1, 32, 8, 128, 128, 16), (37, 6, 3, 96, 48, 24), (130, 1, 1, 32, 16, 7),
                                                        (65, 10, 5, 256, 64, 64), (300, 14, 2, 64, 64, 1), (9, 3, 3, 192, 176, 100)])
def test_append(nv, orc, mode, dtype, interleaved, T, Hq, heads, D, rot, page_size):
    pages = (2 * T) // page_size + 2
    c = new_cache(nv, mode, pages, heads, page_size, D, use_g=T != 65)
    # parts of one projection's rows; of T == 37, rows that begin at a multiple of 16 bytes only
    pad = 8 if T == 37 else 0
    qkv = torch.zeros(T, (Hq + 2 * heads) * D + pad, dtype=dtype, device="cuda")
    qkv[:, pad:] = seeded((T, (Hq + 2 * heads) * D), T, dtype, 2.0)
    if T > 1:
        qkv[T // 2, pad + Hq * D + 5] = 700.0  # a key far beyond g
        qkv[0, pad:] = 0
    at = [pad, pad + Hq * D, pad + (Hq + heads) * D, pad + (Hq + 2 * heads) * D]
    q, k, v = (qkv[:, x:y].unflatten(1, (-1, D)) for x, y in zip(at, at[1:]))
    cos, sin = table(rot)
    g = torch.Generator().manual_seed(T)
    positions = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    positions[0] = 299
    slots = distinct_slots(T, pages * page_size, T)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    out = nv.kv_cache_append(c, q, k, v, cos, sin, positions.cuda(), slots.cuda(), interleaved)
    nv.check_device_errors()
    assert out.shape == (T, Hq, D) and out.is_contiguous()
    assert torch.equal(out.cpu(), turned(q, cos, sin, positions, interleaved).to(dtype))
    n = slots.numpy()
    for x, codes, scales, gl in ((turned(k, cos, sin, positions, interleaved), c.k_codes, c.k_scales, G_K), (v.float().cpu(), c.v_codes, c.v_scales, G_V)):
        oc, os_ = oracle_rows(orc, mode, x, gl if c.g_k is not None else None)
        assert np.array_equal(rows_of(codes, n, page_size), oc) and np.array_equal(rows_of(scales, n, page_size), os_)
    rest = torch.ones(pages * page_size, dtype=torch.bool)
    rest[slots.long()] = False
    m = rest.nonzero()[:, 0].numpy()
    for t, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
        assert np.array_equal(rows_of(t, m, page_size), rows_of(b, m, page_size))


def test_append_is_kv_cache_write_at_position_zero(nv):
    """At angle zero nothing turns: the bytes are kv_cache_write's."""
    T, heads, D = 50, 2, 64
    k, v, q = seeded((T, heads, D), 1), seeded((T, heads, D), 2), seeded((T, 4, D), 3)
    slots = distinct_slots(T, 64, 4).cuda()
    a, b = (new_cache(nv, "nvfp4", 4, heads, 16, D) for _ in range(2))
    out = nv.kv_cache_append(a, q, k, v, *table(64), torch.zeros(T, dtype=torch.int32, device="cuda"), slots)
    nv.kv_cache_write(b, k, v, slots)
    assert torch.equal(out, q)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a, name), getattr(b, name))


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
def test_append_skips_tokens(nv, mode):
    T, heads, D = 9, 2, 64
    c = new_cache(nv, mode, 2, heads, 16, D)
    q, k, v = seeded((T, 4, D), 1), seeded((T, heads, D), 2), seeded((T, heads, D), 3)
    cos, sin = table(32)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    out = torch.full((T, 4, D), 7.0, dtype=bf16, device="cuda")

    def run(positions, slots):
        out.fill_(7.0)
        for t, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
            t.copy_(b)
        nv.kv_cache_append(c, q, k, v, cos, sin, i32(positions), i32(slots), q_out=out)

    good_p, good_s = list(range(9)), list(range(9))
    run(good_p, good_s)
    nv.check_device_errors()
    want, cache_want = out.clone(), [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    # padding: slots below zero, whatever their positions
    run([0, 1, -5, 3, 999, 5, 6, 7, 8], [0, 1, -1, 3, -2 ** 31, 5, 6, 7, 8])
    nv.check_device_errors()
    skipped = [2, 4]
    for bad_p, bad_s in (([0, 1, -1, 3, 300, 5, 6, 7, 8], good_s), (good_p, [0, 1, 32, 3, 2 ** 31 - 1, 5, 6, 7, 8]),
                         ([0, 1, 2 ** 31 - 1, 3, -2 ** 31, 5, 6, 7, 8], good_s), (None, None)):
        if bad_p is not None:
            run(bad_p, bad_s)
            with pytest.raises(nv.Nvfp4Error) as err:
                nv.check_device_errors()
            assert err.value.status == nv.ERR_DEVICE_INDEX
        else:
            run(good_p, [0, 1, -1, 3, -1, 5, 6, 7, 8])
        assert (out[skipped] == 7).all()
        kept = [i for i in range(9) if i not in skipped]
        assert torch.equal(out[kept], want[kept])
        for t, b, w in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before, cache_want):
            assert torch.equal(t[0, :, kept], w[0, :, kept]) and torch.equal(t[0, :, skipped], b[0, :, skipped])
            assert torch.equal(t[1], b[1]) and torch.equal(t[0, :, 9:], b[0, :, 9:])
    nv.check_device_errors()
    assert nv.kv_cache_append(c, q[:0], k[:0], v[:0], cos, sin, i32([]), i32([])).shape == (0, 4, D)


def filled(nv, mode, pages, heads, page_size, D, seed):
    c = nv.KvCache.empty(mode, pages, heads, page_size, D, *([torch.ones(1, device="cuda")] * 2 if mode == "nvfp4" else []))
    g = torch.Generator().manual_seed(seed)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, dtype=torch.uint8))
    return c


def sequential(t, page_size, src, dst):
    t = t.cpu().clone()
    total = t.shape[0] * page_size
    for s, d in zip(src, dst):
        if 0 <= s < total and 0 <= d < total:
            t[d // page_size, :, d % page_size] = t[s // page_size, :, s % page_size]
    return t


def check_moves(nv, c, src, dst, starts, order=None):
    names = ("k_codes", "k_scales", "v_codes", "v_scales")
    o = range(len(src)) if order is None else order
    want = [sequential(getattr(c, n), c.page_size, [src[i] for i in o], [dst[i] for i in o]) for n in names]
    nv.kv_cache_move(c, i32(src), i32(dst), None if starts is None else i32(starts))
    for n, w in zip(names, want):
        assert torch.equal(getattr(c, n).cpu(), w), n


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("heads,D,page_size", [(8, 128, 16), (3, 96, 24), (1, 32, 7), (2, 256, 64), (2, 160, 5), (2, 224, 1)])
def test_moves(nv, mode, heads, D, page_size):
    total = 200
    pages = -(-total // page_size)
    c = filled(nv, mode, pages, heads, page_size, D, D)
    total = pages * page_size
    perm = distinct_slots(total, total, 5).tolist()
    check_moves(nv, c, perm[:60], perm[60:120], None)                      # every one for itself
    check_moves(nv, c, perm[:60] + [-1, 3], perm[60:120] + [4, -7], None)  # and some skipped
    # accepted drafts of three sequences close up in place
    src, dst, starts = [], [], [0]
    for first, path in ((0, [0, 2, 3, 7, 9, 12, 13, 20, 21, 22, 30]), (60, [1, 2]), (120, [0])):
        src += [first + p for p in path]
        dst += [first + i for i in range(len(path))]
        starts.append(len(src))
    check_moves(nv, c, src, dst, starts)
    # chains: what one move writes the next ones read, over more than one group of moves; the same slot written twice
    check_moves(nv, c, [5] + list(range(50, 80)) + [5, 6, 79], list(range(50, 81)) + [90, 90, 91], [0, 34])
    check_moves(nv, c, [10, 11, 12, 11, 10], [11, 12, 13, 10, 11], [0, 5, 5])
    check_moves(nv, c, [], [], [0, 0])
    check_moves(nv, c, [], [], None)
    nv.check_device_errors()


def test_move_refuses_what_is_past_the_cache(nv):
    c = filled(nv, "nvfp4", 4, 2, 16, 64, 1)
    for src, dst in (([0, 64, 1], [10, 11, 12]), ([0, 2 ** 31 - 1, 1], [10, 11, 12]), ([0, 5, 1], [10, 64, 12])):
        for starts in (None, [0, 3]):
            check_moves(nv, c, src, dst, starts)
            with pytest.raises(nv.Nvfp4Error) as err:
                nv.check_device_errors()
            assert err.value.status == nv.ERR_DEVICE_INDEX
    # sequences whose starts are out of order or past the moves are skipped, the others made
    for starts, order in (([0, 2, 1, 3], [0, 1, 1, 2]), ([0, 2, 4], [0, 1]), ([-1, 2, 3], [2])):
        check_moves(nv, c, [0, 1, 2], [20, 21, 22], starts, order)
        with pytest.raises(nv.Nvfp4Error):
            nv.check_device_errors()
    nv.check_device_errors()
