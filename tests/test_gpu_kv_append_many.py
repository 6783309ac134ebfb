"""kv_cache_append where a thread turns four heads of a token, from
T * Hq * D / 16 = 148 * 2048 on: rotated queries against the definition's fp32
steps and the cache's bytes against kv_cache_write's for the rotated keys (which
test_gpu_kv_cache.py holds to the oracle's), on both sides of that border."""
import pytest
import torch

from kv_reference import distinct_slots
from test_gpu_kv_append import i32, table
from test_gpu_kv_cache import new_cache

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("k_codes", "k_scales", "v_codes", "v_scales")


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def four_heads(T, Hq, D):
    return T * Hq * D // 16 >= 148 * 2048


def parts(T, Hq, heads, D, dtype, pad):
    """q, k, v as parts of one projection's rows, which begin `pad` elements into their storage's."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(T, (Hq + 2 * heads) * D + pad, generator=gen, device="cuda").mul_(2.0).to(dtype)
    at = [pad, pad + Hq * D, pad + (Hq + heads) * D, pad + (Hq + 2 * heads) * D]
    return [qkv[:, x:y].unflatten(1, (-1, D)) for x, y in zip(at, at[1:])]


def turned(x, cos, sin, positions, interleaved):
    """fp32: every product and every sum is an operation of its own, and rounded."""
    x, p = x.float(), positions.long()
    c, s, rot = cos[p][:, None], sin[p][:, None], 2 * cos.shape[1]
    out = x.clone()
    i = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    j = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    out[..., i], out[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return out


def check(nv, mode, dtype, T, Hq, heads, D, rot, page_size, interleaved, pad=0):
    pages = T // page_size + 3
    a, b = (new_cache(nv, mode, pages, heads, page_size, D) for _ in range(2))
    q, k, v = parts(T, Hq, heads, D, dtype, pad)
    cos, sin = table(rot)
    positions = torch.randint(0, 300, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    slots = distinct_slots(T, pages * page_size, T).cuda()
    out = nv.kv_cache_append(a, q, k, v, cos, sin, positions, slots, interleaved)
    nv.kv_cache_write(b, turned(k, cos, sin, positions, interleaved), v.float(), slots)
    nv.check_device_errors()
    assert torch.equal(out, turned(q, cos, sin, positions, interleaved).to(dtype))
    for name in NAMES:  # slots that are not named as well
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_both_sides_of_the_border(nv, mode, dtype, interleaved):
    assert not four_heads(1183, 32, 128) and four_heads(1184, 32, 128)
    for T in (1183, 1184):
        check(nv, mode, dtype, T, 32, 2, 128, 128, 16, interleaved)


# the last group of heads of one, two and three; fewer heads than a group; a part of each head turning
@pytest.mark.parametrize("mode,dtype", [("nvfp4", bf16), ("mxfp8", f16), ("mxfp4", f32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,heads,D,rot,page_size,pad", [(8503, 6, 3, 96, 48, 24, 0), (10901, 7, 1, 64, 64, 7, 8), (1403, 14, 2, 256, 64, 64, 0),
                                                            (1203, 33, 1, 128, 112, 100, 8), (151553, 1, 1, 32, 16, 256, 0)])
def test_heads_that_four_do_not_divide(nv, mode, dtype, interleaved, T, Hq, heads, D, rot, page_size, pad):
    assert four_heads(T, Hq, D)
    check(nv, mode, dtype, T, Hq, heads, D, rot, page_size, interleaved, pad)


@pytest.mark.parametrize("Hq", [32, 31])
def test_skipped_tokens(nv, Hq):
    """The queries' loads are under way when a token turns out to be skipped."""
    T, heads, D = 1300, 2, 128
    assert four_heads(T, Hq, D)
    c = new_cache(nv, "nvfp4", T // 16 + 2, heads, 16, D)
    total = c.num_pages * 16
    q, k, v = parts(T, Hq, heads, D, bf16, 0)
    cos, sin = table(64)
    before = [getattr(c, n).clone() for n in NAMES]
    good_p, good_s = [i % 300 for i in range(T)], list(range(T))

    def run(positions, slots):
        for name, b in zip(NAMES, before):
            getattr(c, name).copy_(b)
        out = torch.full((T, Hq, D), 7.0, dtype=bf16, device="cuda")
        nv.kv_cache_append(c, q, k, v, cos, sin, i32(positions), i32(slots), q_out=out)
        return out, [getattr(c, n).clone() for n in NAMES]

    def changed(x, at):
        x = list(x)
        for i, value in at.items():
            x[i] = value
        return x

    want, cache_want = run(good_p, good_s)
    nv.check_device_errors()
    skipped = [0, 700, T - 1]
    for positions, slots, bad in ((good_p, {0: -1, 700: -2 ** 31, T - 1: -7}, False),
                                  (changed(good_p, {0: 999, 700: -5, T - 1: 2 ** 31 - 1}), {0: -1, 700: -1, T - 1: -1}, False),
                                  (good_p, {0: total, 700: 2 ** 31 - 1, T - 1: total + 1}, True),
                                  (changed(good_p, {0: -1, 700: 300, T - 1: -2 ** 31}), {}, True)):
        out, cache = run(positions, changed(good_s, slots))
        if bad:
            with pytest.raises(nv.Nvfp4Error) as err:
                nv.check_device_errors()
            assert err.value.status == nv.ERR_DEVICE_INDEX
        else:
            nv.check_device_errors()
        kept = [i for i in range(T) if i not in skipped]
        assert (out[skipped] == 7).all() and torch.equal(out[kept], want[kept])
        for t, b, w in zip(cache, before, cache_want):
            t, b, w = (x.transpose(1, 2).flatten(0, 1) for x in (t, b, w))  # by slots
            assert torch.equal(t[kept], w[kept]) and torch.equal(t[skipped], b[skipped]) and torch.equal(t[T:], b[T:])
