"""Values and arguments at the edges of kv_attention's contract, on both of its
kernels: one query row goes through k_kv_decode, forty a key/value head through
k_kv_prefill."""
import math

import pytest
import torch

import kv_reference
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


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 10])
@pytest.mark.parametrize("power", [20.0, 25.7, 27.0])
def test_many_light_tokens_beside_heavy_ones(nv, mode, dtype, n, power):
    """131072 tokens of weight 2^-power beside four of weight 1 whose values are
    zero: all of the output comes from weights far below the largest.

    Tolerance, relative to the largest weight 1.  The kernels hold weights as
    16-bit floats times at least 2^7 (fp16: half a step of its subnormals is
    2^-25, so 2^-32 a weight) or in two bf16 terms (2^-16 relative): with
    A = sum w |v| = out, sum w = l,
      u out + (2^-11 + 2 dz + sums) A + 2^-32 sum |v| / l.
    The logits of the light tokens are 0 and exact but for the reference's
    2^-22 * power ln 2."""
    D, L, page = 64, 131072, 1024
    g = [torch.tensor([2688.0], device="cuda")] * 2 if mode == "nvfp4" else [None] * 2
    c = nv.KvCache.empty(mode, L // page, 1, page, D, *g)
    k, v = torch.zeros(L, 1, D, dtype=bf16, device="cuda"), torch.full((L, 1, D), 6.0, dtype=bf16, device="cuda")
    heavy = torch.tensor([0, 32, 64, 96], device="cuda")  # one for each warp of a CTA
    k[heavy, :, 0] = 6.0
    v[heavy] = 0.0
    nv.kv_cache_write(c, k, v, torch.arange(L, dtype=torch.int32, device="cuda"))
    q = torch.zeros(n, 4, D, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    scale = power * math.log(2.0) / 6.0
    table = torch.arange(L // page, dtype=torch.int32, device="cuda")[None]
    ko, vo = nv.kv_cache_read(c, i32([0, 1]), torch.float32)
    assert ko[0, 0, 0] == 6 and ko[1].abs().sum() == 0 and vo[0].abs().sum() == 0 and (vo[1] == 6).all()
    light = 2.0 ** (-scale * 6.0 / math.log(2.0))
    l = 4 + (L - 4) * light
    want, total = (L - 4) * light * 6.0 / l, math.log(l) + scale * 6.0
    dz = 2.0 ** -21 * scale * 6.0 + 2.0 ** -22
    sums = (L / 4 + 160) * 2.0 ** -23
    tol = torch.finfo(dtype).eps / 2 * want + (2.0 ** -11 + 2 * dz + sums) * want + 2.0 ** -32 * L * 6.0 / l
    assert tol < want / 20
    for kw in ({}, {"workspace": no_workspace()}):
        out, lse = nv.kv_attention(c, q, table, i32([L]), i32([0, n]), n, L, scale=scale, causal=False, return_lse=True, **kw)
        nv.check_device_errors()
        assert ((out.double() - want).abs() <= tol).all(), (out.double().min(), out.double().max(), want, tol)
        assert ((lse.double() - total).abs() <= dz + 2.0 ** -22 * total + sums).all()


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("kexp,vexp", [(-70, (-64, -70, -76, -84)), (-100, (-100, -110, -118, 0)), (50, (60, 58, -118, 0))])
def test_mx_blocks_far_from_one(nv, mode, dtype, n, kexp, vexp):
    """Value blocks of the given powers of two beside one another, keys of
    2^kexp with a scale that brings the logits back to order one."""
    L, D = 300, 128
    c, table = make(nv, mode, [L], 1, D, 16, 47)
    j = torch.arange(L)
    slots = (table[0].cpu()[j // 16] * 16 + j % 16).to(torch.int32).cuda()
    k = seeded((L, 1, D), 1, torch.float32) * 2.0 ** kexp
    v = seeded((L, 1, D), 2, torch.float32)
    v = (v.unflatten(-1, (-1, 32)) * torch.exp2(torch.tensor([float(x) for x in vexp], device="cuda"))[:, None]).flatten(-2)
    nv.kv_cache_write(c, k.contiguous(), v.contiguous(), slots)
    q = seeded((n, 4, D), 3, dtype)
    scale = D ** -0.5 * 2.0 ** -kexp
    out, lse = torch.empty_like(q, dtype=dtype), torch.empty(n, 4, device="cuda")
    for kw in ({}, {"workspace": no_workspace()}):
        nv.kv_attention(c, q, table, i32([L]), i32([0, n]), n, L, scale=scale, out=out, lse=lse, **kw)
        nv.check_device_errors()
        o, l, tol, ltol = attention(cache_sides(c), q, table, torch.tensor([L]), torch.tensor([0, n]), scale)
        lost = o.abs() > torch.finfo(dtype).max  # beyond fp16
        assert torch.isinf(out.cpu()[lost]).all()
        o[lost] = float("nan")
        check(out, o, tol, "out")
        check(lse, l, ltol, "lse")
        if dtype == bf16:
            assert (out.abs().amax((0, 1)).view(4, 32) > 0).all()


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_mx_scale_bytes_from_the_smallest_on(nv, mode, dtype, n, D):
    """Value blocks with the scale bytes 0, 1, 2, ... in the outputs' elements
    beside one another, and around the border of one factor (2 for MXFP4, whose
    keys have theirs at 2^25)."""
    L = 150
    c, table = make(nv, mode, [L], 1, D, 16, 48)
    q = seeded((n, 4, D), 4, dtype)
    blocks = D // 32
    for first in (0, 60, 126, 187):
        c.v_scales.copy_((first + torch.arange(blocks, device="cuda") % 5).to(torch.uint8).expand_as(c.v_scales))
        sides = cache_sides(c)
        out = nv.kv_attention(c, q, table, i32([L]), i32([0, n]), n, L)
        nv.check_device_errors()
        o, _, tol, _ = attention(sides, q, table, torch.tensor([L]), torch.tensor([0, n]), D ** -0.5)
        if dtype == f16:  # beyond fp16
            o[o.abs() > 60000] = float("nan")
        check(out, o, tol, "out")
    for byte in (90, 152, 153):
        c.v_scales.fill_(127)
        c.k_scales.fill_(byte)
        scale = D ** -0.5 * 2.0 ** (127 - byte) / 8
        compare(nv, c, table, [L], q, [0, n], n, L, scale=scale)


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("n", [1, 40])
def test_mx_largest_values_over_a_long_range(nv, mode, n):
    """Values of 2^64 times the largest code, equal weights after a rise of the
    logits that the running maximum does not follow (less than 2^8)."""
    D, L, page = 32, 1 << 17, 1024
    c = nv.KvCache.empty(mode, L // page, 1, page, D)
    most = {"mxfp4": 6.0, "mxfp8": 448.0}[mode]
    k = torch.ones(L, 1, D, dtype=bf16, device="cuda")
    k[:256] = 0
    v = torch.full((L, 1, D), most * 2.0 ** 64, dtype=bf16, device="cuda")
    nv.kv_cache_write(c, k, v, torch.arange(L, dtype=torch.int32, device="cuda"))
    assert (nv.kv_cache_read(c, i32([5]))[1] == most * 2.0 ** 64).all()
    q = torch.ones(n, 1, D, dtype=bf16, device="cuda")
    table = torch.arange(L // page, dtype=torch.int32, device="cuda")[None]
    for kw in ({}, {"workspace": no_workspace()}):
        out = nv.kv_attention(c, q, table, i32([L]), i32([0, n]), n, L, scale=7.0 * math.log(2.0) / D, causal=False, **kw)
        nv.check_device_errors()
        # half a bf16 step, the weights' 2^-16 and the fp32 sums of 2^17 terms in four chains
        tol = 2.0 ** -9 + 2.0 ** -16 + (L / 4 + 160) * 2.0 ** -23
        assert ((out.double() / (most * 2.0 ** 64) - 1).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n,D,page", [(1, 128, 16), (1, 96, 7), (1, 256, 64), (13, 64, 16), (40, 128, 16), (40, 96, 7), (70, 256, 64)])
@pytest.mark.parametrize("L", [130, 2500])
def test_nan_codes_count_as_480(nv, dtype, n, D, page, L, monkeypatch):
    """kv_attention carries no NaN of an MXFP8 cache into its results: the codes
    are +-480, for the queries that see their tokens and for no others;
    kv_cache_read gives the NaN."""
    heads, G, lens = 2, 3, [L, 120]
    c, table = make(nv, "mxfp8", lens, heads, D, page, 93)
    starts = [0, n, 2 * n]
    q = seeded((2 * n, heads * G, D), 6, dtype)

    def poison(side, b, j, head, element, code):
        codes = (c.k_codes if side == "k" else c.v_codes).view(torch.uint8)
        codes[int(table[b, j // page]), head, j % page, element] = code

    poison("v", 0, L - 2 if n > 1 else L - 1, 0, 5, 0x7F)  # the last two tokens: few queries see them
    poison("v", 0, L - n // 2 - 1, 0, 0, 0xFF)
    poison("v", 0, 40, 1, D - 1, 0xFF)                     # all queries see it
    poison("k", 1, 120 - n // 2 - 1, 1, 7, 0x7F)
    at = int(table[0, 40 // page]) * page + 40 % page
    assert torch.isnan(nv.kv_cache_read(c, i32([at]), dtype)[1][0, 1, D - 1])
    table480 = kv_reference.E4M3.clone()
    table480[0x7F], table480[0xFF] = 480.0, -480.0
    monkeypatch.setattr(kv_reference, "E4M3", table480)
    for window in (0, 60):
        for kw in ({}, {"workspace": no_workspace()}):
            compare(nv, c, table, lens, q, starts, n, L, window=window, **kw)


@pytest.mark.parametrize("heads,G,n", [(1, 8, 40), (2, 4, 3)])
def test_a_loose_bound_on_the_queries(nv, heads, G, n):
    """max_q may be any upper bound; no sequence has more than T queries."""
    lens = [3000, 700]
    c, table = make(nv, "nvfp4", lens, heads, 64, 16, 95)
    q = seeded((2 * n, heads * G, 64), 7, bf16)
    for starts in ([0, n, 2 * n], [0, 2 * n - 1, 2 * n]):
        want = compare(nv, c, table, lens, q, starts, 2 * n, 3000)
        for loose in (2 * n + 1, 1 << 20, 1 << 30):
            got = compare(nv, c, table, lens, q, starts, loose, 3000)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("n,D,page", [(1, 128, 16), (1, 96, 24), (1, 64, 7), (40, 128, 64), (40, 96, 24), (40, 256, 7)])
def test_rows_without_a_name_have_no_effect(nv, mode, n, D, page):
    lens, heads = [150, 37], 2
    c, table = make(nv, mode, lens, heads, D, page, 97)
    q = seeded((2 * n, heads * 4, D), 8, bf16)
    named = torch.zeros(c.num_pages, page, dtype=torch.bool)
    for b, length in enumerate(lens):
        j = torch.arange(length)
        named[table[b].cpu().long()[j // page], j % page] = True
    other = ~named[:, None, :, None].cuda()
    results = []
    for byte in (0xFF, 0x7F, 0x00, 0x5A):
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.copy_(torch.where(other, torch.full_like(t.view(torch.uint8), byte).view(t.dtype), t))
        results.append(nv.kv_attention(c, q, table, i32(lens), i32([0, n, 2 * n]), n, 150, return_lse=True))
        nv.check_device_errors()
    assert torch.isfinite(results[0][0].float()).all()
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("page", [16, 24])
def test_tokens_on_bad_pages_count_as_unseen(nv, mode, dtype, n, page):
    lens, heads, G, D = [170, 90], 2, 4, 64
    c, table = make(nv, mode, lens, heads, D, page, 61)
    q = seeded((2 * n, heads * G, D), 1, dtype)
    starts = [0, n, 2 * n]
    sides = cache_sides(c)
    for bad in ([0], [2, 4], list(range(-(-170 // page)))):
        for entry in (c.num_pages, -1, 2 ** 31 - 1):
            t = table.clone()
            t[0, bad] = entry
            out, lse = nv.kv_attention(c, q, t, i32(lens), i32(starts), n, 170, return_lse=True)
            with pytest.raises(nv.Nvfp4Error) as e:
                nv.check_device_errors()
            assert e.value.status == nv.ERR_DEVICE_INDEX
            # the reference without those tokens: softmax over the rest
            o, l, tol, ltol = seen_without(sides, q, table, lens, starts, D ** -0.5, {0: bad})
            check(out, o, tol, "out")
            check(lse, l, ltol, "lse")


def seen_without(sides, q, table, lens, starts, scale, bad):
    """attention() with the tokens of pages bad[b] of sequence b left out: a
    query at position p over the tokens that are left is the last query over the
    cache that holds only those."""
    page = sides[0].shape[2]
    rows = [attention(sides, q, table, torch.tensor(lens), torch.tensor(starts), scale)]
    out, lse, tol, ltol = rows[0]
    for b, pages in bad.items():
        for i in range(starts[b + 1] - starts[b]):
            t, p = starts[b] + i, lens[b] - (starts[b + 1] - starts[b]) + i
            kept = [j for j in range(max(0, p + 1)) if j // page not in pages]
            at = table[b].cpu().long()
            j = torch.tensor(kept, dtype=torch.long)
            K, V = (s[at[j // page], :, j % page].transpose(0, 1)[None] for s in sides)  # one page [1, H, kept, D]
            r = attention((K, V), q[t:t + 1], torch.zeros(1, 1), torch.tensor([len(kept)]), None, scale)
            out[t], lse[t], tol[t], ltol[t] = (x[0] for x in r)
    return out, lse, tol, ltol


@pytest.mark.parametrize("mode,dtype", [("nvfp4", bf16), ("mxfp4", f16), ("mxfp8", bf16)])
@pytest.mark.parametrize("lens,n", [([5000, 700], [1, 1]), ([4097], [3]), ([2047, 4100], [130, 40])])
def test_a_workspace_of_the_stated_size_is_enough(nv, mode, dtype, lens, n):
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    c, table = make(nv, mode, lens, 2, 128, 64, 31)
    q = seeded((starts[-1], 8, 128), 7, dtype)
    size = nv.kv_attention_workspace_size(len(lens), starts[-1], 8, 2, 128, max(n), max(lens), 0)
    assert size > 0
    for part in (size, size // 2 // 16 * 16, size // 5 // 16 * 16):
        guard = 1 << 20
        both = torch.full((part + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        compare(nv, c, table, lens, q, starts, max(n), max(lens), workspace=both[:part])
        assert (both[part:] == 0xA5).all()


@pytest.mark.parametrize("mode,dtype", [("nvfp4", bf16), ("nvfp4", f16), ("mxfp4", bf16), ("mxfp8", bf16)])
@pytest.mark.parametrize("D,border", [(32, 48), (64, 48), (96, 32), (128, 32), (160, 16), (256, 16)])
def test_both_sides_of_the_border_between_the_kernels(nv, mode, dtype, D, border):
    """The most rows a key/value head that k_kv_decode takes, and one query more."""
    lens = [700, 90]
    c, table = make(nv, mode, lens, 2, D, 16, 99)
    for n in (border // 4, border // 4 + 1):
        q = seeded((2 * n, 8, D), 9, dtype)
        compare(nv, c, table, lens, q, [0, n, 2 * n], n, 700)
        compare(nv, c, table, lens, q, [0, 2 * n - 1, 2 * n], 2 * n - 1, 700, window=50)
