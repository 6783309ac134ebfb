"""GPU parity of kv_attention with a 64-bit reference on the cache's own
values; the tolerance is derived in kv_reference.py."""
import pytest
import torch

from kv_reference import attention, cache_sides, check, distinct_slots, seeded

pytestmark = pytest.mark.gpu

bf16, f16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(nv, mode, lens, heads, D, page_size, seed, use_g=True, k_std=1.0, v_std=1.0, spare=2):
    """A cache holding `lens` tokens of each sequence on shuffled pages; every
    other byte is 0xFF (NaN scales and codes) and the page table's unused
    entries name no page."""
    need = [-(-n // page_size) for n in lens]
    pages = sum(need) + spare
    g = [torch.tensor([x], device="cuda") for x in (5.0 * k_std, 4.0 * v_std)] if mode == "nvfp4" and use_g else [None] * 2
    c = nv.KvCache.empty(mode, pages, heads, page_size, D, *g)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.view(torch.uint8).fill_(0xFF)
    perm = distinct_slots(pages, pages, seed)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, (n, L) in enumerate(zip(need, lens)):
        table[b, :n] = perm[at:at + n]
        at += n
        if L:
            j = torch.arange(L)
            slots = (table[b][j // page_size] * page_size + j % page_size).to(torch.int32).cuda()
            nv.kv_cache_write(c, seeded((L, heads, D), seed + 2 * b + 1, bf16, k_std),
                              seeded((L, heads, D), seed + 2 * b + 2, bf16, v_std), slots)
    return c, table.cuda()


def compare(nv, c, table, lens, q, q_start=None, max_q=None, max_kv=None, causal=True, window=0, scale=None, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    nv.kv_attention(c, q, table, i32(lens), None if q_start is None else i32(q_start), max_q, max_kv, scale=scale,
                    causal=causal, window=window, out=out, lse=lse, **kw)
    nv.check_device_errors()
    o, l, tol, ltol = attention(cache_sides(c), q, table, torch.tensor(lens),
                                None if q_start is None else torch.tensor(q_start),
                                c.D ** -0.5 if scale is None else scale, causal, window)
    check(out, o, tol, "out")
    check(lse, l, ltol, "lse")
    unnamed = torch.isnan(l).cuda()
    assert (out[unnamed] == 7).all() and (lse[unnamed] == 7).all()  # left as they were
    return out, lse


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("heads,G,D,page_size", [(8, 4, 128, 64), (3, 1, 96, 24), (1, 16, 64, 16), (2, 8, 256, 32),
                                                 (2, 7, 32, 7), (1, 3, 192, 100), (1, 71, 128, 16)])
def test_one_token_a_sequence(nv, mode, dtype, heads, G, D, page_size):
    lens = [1, 0, 17, 300, 64, 129]
    c, table = make(nv, mode, lens, heads, D, page_size, 11, use_g=heads != 3)
    q = seeded((len(lens), heads * G, D), 5, dtype)
    compare(nv, c, table, lens, q)
    compare(nv, c, table, lens, q, window=40, max_kv=300)
    compare(nv, c, table, lens, q, causal=False, scale=0.3)


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("n", [1, 11])
def test_scale_of_any_sign(nv, mode, n):
    lens = [90, 33]
    c, table = make(nv, mode, lens, 2, 64, 16, 13)
    q = seeded((2 * n, 8, 64), 5, bf16)
    for scale in (-0.2, 0.0):
        compare(nv, c, table, lens, q, [0, n, 2 * n], n, scale=scale)


@pytest.mark.parametrize("B", [32, 33, 75, 161, 500])
@pytest.mark.parametrize("most,window", [(60, 0), (700, 100)])
def test_many_sequences(nv, B, most, window):
    """More sequences than a warp, or all of a CTA's, take at a time; some of
    them empty, some without a query."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, most, (B,), generator=g).tolist()
    lens[B // 2:B // 2 + 3] = [0, 0, 0]
    n = torch.randint(0, 3, (B,), generator=g).clamp(max=torch.tensor(lens)).tolist()
    n[0] = n[B - 1] = 1
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    c, table = make(nv, "nvfp4", lens, 2, 64, 16, 15)
    q = seeded((starts[-1], 6, 64), 6, bf16)
    compare(nv, c, table, lens, q, starts, 2, max(lens), window=window)
    compare(nv, c, table, lens, seeded((B, 6, 64), 7, f16), workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("heads,G,D,page_size", [(2, 4, 128, 64), (3, 1, 96, 24), (1, 16, 64, 16), (2, 3, 256, 100),
                                                 (1, 1, 32, 7)])
def test_many_tokens_a_sequence(nv, mode, dtype, heads, G, D, page_size):
    lens, n = [150, 3, 0, 200, 33, 64], [70, 5, 2, 1, 33, 0]  # 5 queries over 3 tokens: two see nothing when causal
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    c, table = make(nv, mode, lens, heads, D, page_size, 21)
    q = seeded((starts[-1] + 3, heads * G, D), 6, dtype)  # three rows behind the last sequence
    compare(nv, c, table, lens, q, starts, 70, 200)
    compare(nv, c, table, lens, q, starts, window=19)
    compare(nv, c, table, lens, q, starts, 100, causal=False)
    compare(nv, c, table, lens, q, starts, 70, 200, causal=False, window=50)


@pytest.mark.parametrize("mode,dtype", [("nvfp4", bf16), ("nvfp4", f16), ("mxfp4", f16), ("mxfp8", bf16)])
@pytest.mark.parametrize("lens,n", [([5000, 700], [1, 1]), ([4097], [3]), ([2047, 4100], [130, 40])])
def test_long_axes_are_split_and_joined(nv, mode, dtype, lens, n):
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    c, table = make(nv, mode, lens, 2, 128, 64, 31)
    q = seeded((starts[-1], 8, 128), 7, dtype)
    whole, _ = compare(nv, c, table, lens, q, starts, max(n), max(lens))
    # without a workspace and with a part of one: the same sums in another order
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    compare(nv, c, table, lens, q, starts, max(n), max(lens), workspace=small)
    size = nv.kv_attention_workspace_size(len(lens), starts[-1], 8, 2, 128, max(n), max(lens), 0)
    compare(nv, c, table, lens, q, starts, max(n), max(lens),
            workspace=torch.empty(size // 2, dtype=torch.uint8, device="cuda"))
    # the same call gives the same bits
    again, _ = compare(nv, c, table, lens, q, starts, max(n), max(lens))
    assert torch.equal(whole, again)


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 40])
def test_sharp_and_large_logits(nv, mode, dtype, n):
    """Logits of hundreds: the running maximum moves by more than exp's range
    from tile to tile, and single tokens carry all the weight."""
    lens = [257, 90]
    c, table = make(nv, mode, lens, 2, 64, 16, 41, k_std=20.0, v_std=0.02)
    q = seeded((2 * n, 8, 64), 8, dtype, 6.0)
    compare(nv, c, table, lens, q, [0, n, 2 * n], n, 257)


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("n", [1, 40])
def test_small_and_uneven_queries(nv, mode, dtype, n):
    """Elements of one query over 20 octaves, and queries of 2^-10."""
    lens = [130, 50]
    c, table = make(nv, mode, lens, 1, 128, 16, 43, v_std=30.0)
    q = seeded((2 * n, 4, 128), 9, torch.float32)
    q = q * torch.exp2(torch.randint(-14, 7, q.shape, generator=torch.Generator().manual_seed(3)).float()).cuda()
    q[n:] = q[n:] * 2.0 ** -10
    compare(nv, c, table, lens, q.to(dtype), [0, n, 2 * n], n, 130)


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("n", [1, 40])
def test_mx_scales_over_their_range(nv, mode, n):
    """Value blocks from 2^-60 to 2^60 beside one another, keys far from 1 with
    a scale that brings the logits back."""
    L, D = 100, 128
    c, table = make(nv, mode, [L], 1, D, 16, 47)
    j = torch.arange(L)
    slots = (table[0].cpu()[j // 16] * 16 + j % 16).to(torch.int32).cuda()
    k = seeded((L, 1, D), 1, torch.float32) * 2.0 ** 40
    v = seeded((L, 1, D), 2, torch.float32)
    v = (v.unflatten(-1, (-1, 32)) * torch.exp2(torch.tensor([-60.0, 0.0, 60.0, 20.0], device="cuda"))[:, None]).flatten(-2)
    nv.kv_cache_write(c, k.contiguous(), v.contiguous(), slots)
    compare(nv, c, table, [L], seeded((n, 4, D), 3, bf16), [0, n], n, L, scale=D ** -0.5 * 2.0 ** -40)


def test_queries_as_parts_of_a_projection(nv):
    lens = [70, 40]
    c, table = make(nv, "nvfp4", lens, 2, 64, 16, 51)
    qkv = seeded((12, 12, 64), 1, bf16)
    for starts, n in ((None, 1), ([0, 9, 12], 9)):
        q = (qkv[:2] if starts is None else qkv)[:, :8]
        s = None if starts is None else i32(starts)
        a = nv.kv_attention(c, q, table, i32(lens), s, n)
        assert torch.equal(a, nv.kv_attention(c, q.contiguous(), table, i32(lens), s, n))


def test_a_contiguous_cache_is_one_page_a_sequence(nv):
    B, H, L, D = 3, 2, 75, 64
    c = nv.KvCache.empty("mxfp4", B, H, L, D)
    slots = torch.arange(B * L, dtype=torch.int32, device="cuda")
    nv.kv_cache_write(c, seeded((B * L, H, D), 1), seeded((B * L, H, D), 2), slots)
    compare(nv, c, torch.arange(B, dtype=torch.int32, device="cuda")[:, None], [75, 1, 40], seeded((B, 4, D), 3))


def test_bad_entries_set_the_error_word_and_touch_nothing_else(nv):
    lens = [40, 40, 40, 40]
    c, table = make(nv, "nvfp4", lens, 2, 64, 16, 61)
    for n in (1, 20):
        q = seeded((4 * n, 8, 64), 1, bf16)
        starts = [0, n, 2 * n, 3 * n, 4 * n]
        good = nv.kv_attention(c, q, table, i32(lens), i32(starts), n, 48)
        nv.check_device_errors()

        def bad(kv_len=lens, q_start=starts, page_table=table, rows=slice(0, 0)):
            out = torch.full_like(q, 7.0)
            nv.kv_attention(c, q, page_table, i32(kv_len), i32(q_start), n, 48, out=out)
            with pytest.raises(nv.Nvfp4Error) as e:
                nv.check_device_errors()
            assert e.value.status == nv.ERR_DEVICE_INDEX
            left = torch.ones(4 * n, dtype=torch.bool, device="cuda")
            left[rows] = False
            assert (out[rows] == 7).all() and torch.equal(out[left], good[left])

        bad(kv_len=[40, 49, 40, 40], rows=slice(n, 2 * n))
        bad(kv_len=[40, 40, -1, 40], rows=slice(2 * n, 3 * n))
        bad(q_start=[0, n, 2 * n, 3 * n, 4 * n + 1], rows=slice(3 * n, 4 * n))  # past T, more than max_q
        bad(q_start=[0, n, 2 * n, 3 * n, 2 * n], rows=slice(3 * n, 4 * n))
        bad(q_start=[-1, n, 2 * n, 3 * n, 4 * n], rows=slice(0, n))
        # a page out of range: its 16 tokens count as unseen
        t = table.clone()
        t[1, 0] = c.num_pages
        out = nv.kv_attention(c, q, t, i32(lens), i32(starts), n, 48)
        with pytest.raises(nv.Nvfp4Error):
            nv.check_device_errors()
        seen = nv.kv_attention(c, q, table, i32(lens), i32(starts), n, 48, window=24 if n == 1 else 0)
        nv.check_device_errors()
        if n == 1:  # one query at position 39: tokens 16 .. 39 are its last 24
            assert torch.allclose(out[1].float(), seen[1].float(), rtol=2 ** -6, atol=2 ** -8)
        assert torch.isfinite(out.float()).all() and torch.equal(out[0], good[0]) and torch.equal(out[2 * n:], good[2 * n:])


def test_pages_behind_a_window_are_not_read(nv):
    """A server that frees the pages a sliding window has left may keep any
    entry for them."""
    L, window = 400, 50
    c, table = make(nv, "nvfp4", [L], 2, 128, 16, 71)
    q = seeded((1, 8, 128), 1, bf16)
    want, _ = compare(nv, c, table, [L], q, window=window)
    t = table.clone()
    t[0, : (L - window) // 16] = -5
    got = nv.kv_attention(c, q, t, i32([L]), window=window)
    nv.check_device_errors()
    assert torch.equal(got, want)


def test_empty_calls(nv):
    c, table = make(nv, "mxfp8", [5], 2, 64, 16, 1)
    q = torch.zeros(0, 4, 64, dtype=bf16, device="cuda")
    assert nv.kv_attention(c, q, table[:0], i32([])).shape == (0, 4, 64)
    out, lse = nv.kv_attention(c, q, table, i32([5]), i32([0, 0]), 0, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no cache at all: every query sees nothing
    none = nv.KvCache.empty("mxfp8", 0, 2, 16, 64)
    out, lse = nv.kv_attention(none, seeded((2, 4, 64), 1), torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                               i32([0, 0]), return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    nv.check_device_errors()


def test_on_another_stream_and_two_at_once(nv):
    lens = [3000, 900]
    c, table = make(nv, "nvfp4", lens, 2, 128, 64, 81)
    qs = [seeded((2, 8, 128), s, bf16) for s in (1, 2)]
    kv = i32(lens)
    want = [nv.kv_attention(c, q, table, kv) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(nv.kv_attention(c, q, table, kv))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    nv.check_device_errors()


@pytest.mark.parametrize("mode,D,G", [("nvfp4", 128, 4), ("mxfp8", 64, 8)])
def test_serving_steps_in_one_graph(nv, mode, D, G):
    """A prompt in two chunks, then decoding steps captured once (write, then
    attention) and replayed with new tokens, lengths and slots in the same
    buffers: each step against the reference on the cache as it then is."""
    heads, page_size, most = 2, 16, 96
    lens = [50, 21]
    B, pages = len(lens), 2 * most // page_size
    g = [torch.tensor([x], device="cuda") for x in (5.0, 4.0)] if mode == "nvfp4" else [None] * 2
    c = nv.KvCache.empty(mode, pages, heads, page_size, D, *g)
    table = distinct_slots(pages, pages, 3).view(B, -1).cuda()

    def slot(b, j):
        return int(table[b, j // page_size]) * page_size + j % page_size

    def chunk(lo, hi, seed):
        """Tokens lo[b] .. hi[b] - 1 of each sequence, written and attended."""
        slots = i32([slot(b, j) for b in range(B) for j in range(lo[b], hi[b])])
        T = slots.shape[0]
        qkv = seeded((T, heads * (G + 2), D), seed, bf16)
        q, k, v = qkv[:, :heads * G], qkv[:, heads * G:heads * (G + 1)], qkv[:, heads * (G + 1):]
        nv.kv_cache_write(c, k, v, slots)
        starts = [0]
        for b in range(B):
            starts.append(starts[-1] + hi[b] - lo[b])
        compare(nv, c, table, hi, q, starts, max(h - l for l, h in zip(lo, hi)), max(hi))

    c.k_scales.fill_(0)
    c.v_scales.fill_(0)
    c.k_codes.fill_(0)
    c.v_codes.fill_(0)
    chunk([0, 0], [30, 20], 1)
    chunk([30, 20], lens, 2)
    qkv = seeded((B, heads * (G + 2), D), 3, bf16)
    q, k, v = qkv[:, :heads * G], qkv[:, heads * G:heads * (G + 1)], qkv[:, heads * (G + 1):]
    slots, kv = i32([slot(b, lens[b]) for b in range(B)]), i32([n + 1 for n in lens])
    out, lse = torch.empty(B, heads * G, D, dtype=bf16, device="cuda"), torch.empty(B, heads * G, device="cuda")
    ws = torch.empty(max(16, nv.kv_attention_workspace_size(B, B, heads * G, heads, D, 1, most)), dtype=torch.uint8,
                     device="cuda")

    def step():
        nv.kv_cache_write(c, k, v, slots)
        nv.kv_attention(c, q, table, kv, max_kv=most, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        now = [x + 1 + n for x in lens]
        qkv.copy_(seeded(qkv.shape, 10 + n, bf16))
        slots.copy_(i32([slot(b, now[b] - 1) for b in range(B)]))
        kv.copy_(i32(now))
        ws.fill_(0xFF)
        graph.replay()
        nv.check_device_errors()
        o, l, tol, ltol = attention(cache_sides(c), q, table, torch.tensor(now), None, D ** -0.5)
        check(out, o, tol, "out")
        check(lse, l, ltol, "lse")
