"""GPU parity of kv_attention_tree with a 64-bit reference (tree_reference.py),
and one decoder step with drafts through all of the calls together."""
import pytest
import torch

from kv_reference import attention, cache_sides, check, distinct_slots, seeded
from test_gpu_kv_append import table
from test_gpu_kv_attention import compare, i32, make
from tree_reference import ancestors, attention_tree, pack

pytestmark = pytest.mark.gpu

bf16, f16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def starts_of(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def compare_tree(nv, c, table_, lens, n, q, masks, words=None, junk=0, window=0, max_kv=None, spare=2, **kw):
    """q has `spare` rows more than the sequences name."""
    starts = starts_of(n)
    words = -(-max(n) // 32) if words is None else words
    mask = pack(masks + [0] * (q.shape[0] - len(masks)), words, junk).cuda()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    nv.kv_attention_tree(c, q, table_, i32(lens), mask, i32(starts), max(n), max_kv, window=window, out=out, lse=lse, **kw)
    nv.check_device_errors()
    o, l, tol, ltol = attention_tree(cache_sides(c), q, table_, lens, starts, masks, c.D ** -0.5, window)
    check(out, o, tol, "out")
    check(lse, l, ltol, "lse")
    unnamed = torch.isnan(l).cuda()
    assert (out[unnamed] == 7).all() and (lse[unnamed] == 7).all()
    return out, lse


# rows of a key/value head: 1 to 130 drafts x G, through both kernels and every number of tiles
@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [bf16, f16])
@pytest.mark.parametrize("heads,G,D,page_size", [(2, 4, 128, 64), (3, 1, 96, 24), (1, 8, 64, 16), (2, 3, 256, 100), (1, 2, 32, 7)])
def test_trees(nv, mode, dtype, heads, G, D, page_size):
    for n, lens in (([1, 5, 8, 0], [40, 5, 130, 9]), ([17, 33, 64], [300, 33, 190]), ([130, 31], [131, 517])):
        c, t = make(nv, mode, lens, heads, D, page_size, 11, use_g=heads != 3)
        q = seeded((sum(n) + 2, heads * G, D), 5, dtype)
        masks = [m for b, x in enumerate(n) for m in ancestors(x, b, blank=0.1)]
        compare_tree(nv, c, t, lens, n, q, masks)
        compare_tree(nv, c, t, lens, n, q, masks, window=37)


# 24 rows; 80 and 128 (one query tile, whose tokens two slots take in turn); 160
@pytest.mark.parametrize("mode,n,G", [("nvfp4", 6, 4), ("nvfp4", 20, 4), ("nvfp4", 32, 4), ("nvfp4", 40, 4), ("mxfp8", 6, 4), ("mxfp8", 20, 4),
                                      ("mxfp4", 32, 4), ("mxfp4", 40, 4)])
def test_long_contexts_split_and_whole(nv, mode, n, G):
    """Contexts cut over many workers, with all, some and none of the workspace."""
    lens = [3000, 1033]
    c, t = make(nv, mode, lens, 2, 128, 16, 3)
    q = seeded((2 * n, 2 * G, 128), 5, bf16)
    masks = ancestors(n, 1) + ancestors(n, 2)
    size = nv.kv_attention_tree_workspace_size(2, 2 * n, 2 * G, 2, 128, n, 3000)
    assert size > 0
    for b in (size, size // 2, 0):
        compare_tree(nv, c, t, lens, [n, n], q, masks, max_kv=3000, workspace=torch.empty(b, dtype=torch.uint8, device="cuda"))
    compare_tree(nv, c, t, lens, [n, n], q, masks, max_kv=3000, window=1000)


@pytest.mark.parametrize("n,G", [(7, 2), (50, 4)])
def test_masks_at_their_edges(nv, n, G):
    lens = [n, n + 1, 200, n - 3]  # no context, one token of it, and fewer tokens than drafts
    c, t = make(nv, "nvfp4", lens, 2, 64, 16, 3)
    B = len(lens)
    q = seeded((B * n, 2 * G, 64), 5, bf16)
    full = (1 << n) - 1
    for masks in ([0] * (B * n), [full] * (B * n), [1 << (n - 1)] * (B * n), [1 << i for i in range(n)] * B):
        # bits behind the drafts have no effect, on the depth neither
        words = n // 32 + 2
        junk = ((1 << (32 * words)) - 1) ^ full
        for window in (0, 5, 1, 1 << 40):
            a = compare_tree(nv, c, t, lens, [n] * B, q, masks, words=words, junk=junk, window=window)
            b = compare_tree(nv, c, t, lens, [n] * B, q, masks, words=words, window=window)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("n,G,D", [(6, 2, 64), (6, 2, 96), (9, 2, 256), (30, 4, 128), (60, 4, 64), (60, 4, 256)])
def test_drafts_that_no_mask_names_hold_anything(nv, mode, n, G, D):
    """Places of a tree that were never written: NaN scales, the largest ones
    and infinities of every kind must not reach the queries."""
    lens = [n + 70, n, 300]
    c, t = make(nv, mode, lens, 2, D, 16, 3)
    holes = [1, n // 2, n - 1]
    dead = sum(1 << x for x in holes)
    masks = [m & ~dead for b in range(3) for m in ancestors(n, b)]
    q = seeded((3 * n + 2, 2 * G, D), 5, bf16)
    want = compare_tree(nv, c, t, lens, [n] * 3, q, masks)
    for fill in (0xFF, 0x7F, 0xFE, 0x7E):
        for b, L in enumerate(lens):
            for x in holes:
                j = L - n + x
                page, row = int(t[b, j // 16]), j % 16
                for s in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
                    s.view(torch.uint8)[page, :, row] = fill
        out, lse = torch.full(q.shape, 7.0, dtype=bf16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
        nv.kv_attention_tree(c, q, t, i32(lens), pack(masks + [0, 0], 2).cuda(), i32(starts_of([n] * 3)), n, out=out, lse=lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    nv.check_device_errors()


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8"])
@pytest.mark.parametrize("n,G", [(3, 4), (16, 2), (64, 4)])
def test_a_chain_is_causal_attention(nv, mode, n, G):
    """A tree without branches sees what kv_attention's queries do: within the
    same tolerance, window and all."""
    lens = [n, 400, 77 + n]
    c, t = make(nv, mode, lens, 2, 128, 64, 3)
    q = seeded((3 * n, 2 * G, 128), 5, bf16)
    masks = [(2 << i) - 1 for i in range(n)] * 3
    for window in (0, n + 50):  # (within the drafts kv_attention's window would hide some)
        got = compare_tree(nv, c, t, lens, [n] * 3, q, masks, window=window)
        want = compare(nv, c, t, lens, q, starts_of([n] * 3), n, window=window)
        _, _, tol, ltol = attention(cache_sides(c), q, t, torch.tensor(lens), torch.tensor(starts_of([n] * 3)), 128 ** -0.5, True, window)
        assert ((got[0].double() - want[0].double()).abs().cpu() <= 2 * tol).all()
        assert ((got[1].double() - want[1].double()).abs().cpu() <= 2 * ltol).all()


def test_bad_sequences_and_pages(nv):
    lens, n = [100, 90, 80], [8, 8, 8]
    c, t = make(nv, "nvfp4", lens, 2, 64, 16, 3)
    for G in (2, 8):
        q = seeded((24, 2 * G, 64), 5, bf16)
        masks = [m for b in range(3) for m in ancestors(8, b)]
        mask = pack(masks, 1).cuda()
        want = nv.kv_attention_tree(c, q, t, i32(lens), mask, i32([0, 8, 16, 24]), 8)

        def run(**kw):
            a = dict(page_table=t, kv_len=i32(lens), q_start=i32([0, 8, 16, 24]), max_q=8)
            a.update(kw)
            out = torch.full(q.shape, 7.0, dtype=bf16, device="cuda")
            nv.kv_attention_tree(c, q, tree_mask=mask, out=out, **a)
            with pytest.raises(nv.Nvfp4Error) as err:
                nv.check_device_errors()
            assert err.value.status == nv.ERR_DEVICE_INDEX
            return out

        out = run(kv_len=i32([100, -1, 80]))
        assert (out[8:16] == 7).all() and torch.equal(out[:8], want[:8]) and torch.equal(out[16:], want[16:])
        out = run(kv_len=i32([100, 90, 10 ** 6]))
        assert (out[16:] == 7).all() and torch.equal(out[:16], want[:16])
        out = run(q_start=i32([0, 8, 7, 24]))  # a negative number of queries, then more than max_q
        assert (out[8:] == 7).all() and torch.equal(out[:8], want[:8])
        bad = t.clone()
        bad[1, 5] = c.num_pages  # the page with the last context and the drafts: they count as unseen
        out = run(page_table=bad)
        assert torch.equal(out[:8], want[:8]) and torch.equal(out[16:], want[16:])
        k, v = cache_sides(c)
        # what is left is the context of the first five pages, the same for all drafts
        x = attention((k, v), q[8:16], t[1:2], torch.tensor([80]), torch.tensor([0, 8]), 64 ** -0.5, causal=False)
        check(out[8:16], x[0], x[2], "out")
    nv.check_device_errors()


@pytest.mark.parametrize("n,kv", [(8, 600), (20, 600), (64, 600), (64, 6000)])
def test_outputs_and_queries_at_16_bytes(nv, n, kv):
    """Rows that begin at 16 bytes and not at 32, of queries, results and partial results."""
    G, D = 4, 128
    c, t = make(nv, "nvfp4", [kv], 2, D, 64, 3)
    q = seeded((n, 2 * G, D), 5, bf16)
    mask = pack(ancestors(n, 1), 2).cuda()
    size = nv.kv_attention_tree_workspace_size(1, n, 2 * G, 2, D, n, kv)
    want = nv.kv_attention_tree(c, q, t, i32([kv]), mask, i32([0, n]), n, kv, return_lse=True)

    def shifted(x, by):
        s = torch.zeros(x.numel() + by, dtype=x.dtype, device="cuda")
        s[by:] = x.reshape(-1)
        return s[by:].view(x.shape)

    out = shifted(torch.zeros_like(q), 8)
    got = nv.kv_attention_tree(c, shifted(q, 8), t, i32([kv]), mask, i32([0, n]), n, kv, out=out, return_lse=True,
                               workspace=torch.empty(size + 16, dtype=torch.uint8, device="cuda")[16:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    nv.check_device_errors()


def test_many_sequences(nv):
    g = torch.Generator().manual_seed(1)
    B = 75
    n = torch.randint(0, 4, (B,), generator=g).tolist()
    n[0] = 3
    lens = [x + int(torch.randint(0, 90, (1,), generator=g)) for x in n]
    c, t = make(nv, "mxfp4", lens, 2, 64, 16, 15)
    q = seeded((sum(n), 6, 64), 6, bf16)
    compare_tree(nv, c, t, lens, n, q, [m for b, x in enumerate(n) for m in ancestors(x, b)], window=20)


def step(nv, s):
    """One layer's step over drafts: norm, projection, append, attention, output projection, the next norm."""
    c, sc, h = nv.rms_norm_quantize(s["x"], s["w1"], "nvfp4", s["g1"], 1e-5, s["stream"], "swizzled")
    qkv = nv.qqmm(c, sc, *s["wqkv"], s["K"], "nvfp4", s["g1"], s["g_qkv"])
    T, Hq, H, D = qkv.shape[0], s["Hq"], s["cache"].heads, s["cache"].D
    rows = qkv.view(T, Hq + 2 * H, D)
    q = nv.kv_cache_append(s["cache"], rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:], s["cos"], s["sin"], s["positions"], s["slots"])
    o = nv.kv_attention_tree(s["cache"], q, s["table"], s["kv_len"], s["mask"], s["q_start"], s["n"], s["max_kv"])
    oc, os_ = nv.nvfp4_quantize(o.view(T, Hq * D), s["g_o"], "swizzled")
    y = nv.qqmm(oc, os_, *s["wo"], Hq * D, "nvfp4", s["g_o"], s["g_wo"])
    z, h2, r = nv.rms_norm(y, s["w2"], 1e-5, h, return_rstd=True)
    return q, o, z, h2, r


def test_one_step_with_drafts(nv):
    """Every call on what the call before it gave; then the accepted branch
    closes up and plain attention over it gives what the tree's did."""
    B, n, Hq, H, D, K, page = 3, 12, 8, 2, 64, 256, 16
    lens = [40 + n, 17 + n, 100 + n]
    T = B * n
    pages = [-(-L // page) for L in lens]
    ones = [torch.tensor([x], device="cuda") for x in (6.0, 6.0)]
    cache = nv.KvCache.empty("nvfp4", sum(pages), H, page, D, *ones)
    order = distinct_slots(sum(pages), sum(pages), 1).tolist()
    t = torch.zeros(B, max(pages), dtype=torch.int32)
    for b, p in enumerate(pages):
        t[b, :p] = torch.tensor(order[sum(pages[:b]):sum(pages[:b + 1])])

    def slot(b, j):
        return int(t[b, j // page]) * page + j % page

    for b, L in enumerate(lens):  # the context
        m = L - n
        nv.kv_cache_append(cache, seeded((m, Hq, D), b), seeded((m, H, D), 10 + b), seeded((m, H, D), 20 + b), *table(D),
                           torch.arange(m, dtype=torch.int32, device="cuda"), i32([slot(b, j) for j in range(m)]))
    masks = [m for b in range(B) for m in ancestors(n, 30 + b, near=3)]
    depth = [bin(m).count("1") - 1 for m in masks]

    def weight(N, Kw, seed):
        w = seeded((N, Kw), seed, bf16, Kw ** -0.5)
        g = nv.amax(w)
        return nv.nvfp4_quantize(w, g, "swizzled"), g

    s = dict(x=seeded((T, K), 1), stream=seeded((T, K), 2), w1=seeded((K,), 3, bf16, 0.1) + 1, w2=seeded((K,), 4, bf16, 0.1) + 1,
             g1=torch.tensor([6.0], device="cuda"), g_o=torch.tensor([3.0], device="cuda"), K=K, Hq=Hq, n=n, max_kv=max(lens), cache=cache,
             positions=i32([lens[i // n] - n + depth[i] for i in range(T)]),
             slots=i32([slot(i // n, lens[i // n] - n + i % n) for i in range(T)]), table=t.cuda(), kv_len=i32(lens), mask=pack(masks, 1).cuda(),
             q_start=i32([b * n for b in range(B + 1)]))
    s["cos"], s["sin"] = table(D)
    (s["wqkv"], s["g_qkv"]), (s["wo"], s["g_wo"]) = weight((Hq + 2 * H) * D, K, 5), weight(K, Hq * D, 6)
    got = step(nv, s)
    nv.check_device_errors()
    q, o, z, h2, _ = got
    want, _, tol, _ = attention_tree(cache_sides(cache), q, t, lens, [b * n for b in range(B + 1)], masks, D ** -0.5)
    check(o, want, tol, "drafts")
    assert torch.isfinite(z.float()).all() and torch.isfinite(h2.float()).all()

    # captured into a graph and replayed on other inputs: the eager step's bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(nv, s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = step(nv, s)
        s["x"].copy_(seeded((T, K), 77))
        graph.replay()
        side.synchronize()
        replayed = [x.clone() for x in again]
        for x, y in zip(replayed, step(nv, s)):
            assert torch.equal(x, y)
        side.synchronize()
    torch.cuda.current_stream().wait_stream(side)
    q, o = replayed[:2]

    # the longest branch of each sequence is accepted
    path = []
    for b in range(B):
        best = max(range(n), key=lambda i: depth[b * n + i])
        path.append([d for d in range(n) if masks[b * n + best] >> d & 1])
    src = [slot(b, lens[b] - n + d) for b in range(B) for d in path[b]]
    dst = [slot(b, lens[b] - n + i) for b in range(B) for i in range(len(path[b]))]
    starts = [0]
    for p in path:
        starts.append(starts[-1] + len(p))
    nv.kv_cache_move(cache, i32(src), i32(dst), i32(starts))
    rows = [b * n + d for b in range(B) for d in path[b]]
    now = [lens[b] - n + len(path[b]) for b in range(B)]
    plain = nv.kv_attention(cache, q[rows].contiguous(), s["table"], i32(now), i32(starts), max(len(p) for p in path), max(lens))
    nv.check_device_errors()
    _, _, tol, _ = attention(cache_sides(cache), q[rows], t, torch.tensor(now), torch.tensor(starts), D ** -0.5)
    assert ((plain.double() - o[rows].double()).abs().cpu() <= 2 * tol).all()
