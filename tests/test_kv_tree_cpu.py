"""Host-side checks of kv_cache_append, kv_cache_move and kv_attention_tree
(no GPU)."""
import types

import pytest
import torch

from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv
from test_kv_contract_cpu import host_cache
from test_kv_cpu import A, L, N0, attend, cache, e, msg, needs_device  # noqa: F401 (L is a fixture)


def append(L, c, q=A, k=A, v=A, dt=2, T=3, Hq=4, qs=256, ks=128, vs=128, cos=A, sin=A, max_pos=100, rot=64, inter=0, pos=A,
           slots=A, out=A):
    return L.kv_cache_append(c, q, k, v, dt, T, Hq, qs, ks, vs, cos, sin, max_pos, rot, inter, pos, slots, out, N0)


def move(L, c, src=A, dst=A, M=3, starts=N0, S=3):
    return L.kv_cache_move(c, src, dst, M, starts, S, N0)


def tree(L, c, q=A, dt=2, stride=256, q_start=A, kv_len=A, table=A, mask=A, words=1, B=2, T=9, Hq=4, max_q=4, max_kv=64,
         max_pages=4, scale=0.1, window=0, out=A, lse=N0, ws=N0, ws_bytes=0):
    return L.kv_attention_tree(c, q, dt, stride, q_start, kv_len, table, mask, words, B, T, Hq, max_q, max_kv, max_pages, scale,
                               window, out, lse, ws, ws_bytes, N0)


@pytest.mark.parametrize("call", [append, move, tree])
def test_the_cache_handle_is_checked(L, call):
    assert needs_device(call(L, cache())) and needs_device(call(L, cache(g_k=A, g_v=A)))
    assert call(L, N0) == 1 and "null cache" in msg(L)
    assert call(L, cache(mode=3)) == 1 and call(L, cache(mode=1, g_k=A, g_v=A)) == 1
    assert call(L, cache(page_size=0)) == 1 and call(L, cache(pages=1 << 62, page_size=4)) == 1
    assert call(L, cache(heads=0)) == 1 and call(L, cache(D=48)) == 1 and call(L, cache(D=288)) == 2
    assert call(L, cache(k=N0)) == 1 and call(L, cache(v=A + 8)) == 1


def test_append_arguments(L):
    c = cache()
    assert append(L, c, dt=7) == 2
    for T in (-1, 1 << 40, 1 << 62):
        assert append(L, c, T=T) == 1
    assert append(L, c, Hq=0) == 1 and append(L, c, Hq=65536) == 1
    assert append(L, c, T=1 << 24, Hq=65535, qs=65535 * 64) == 1  # T*Hq*D
    for rot in (0, -16, 8, 24, 80, 128):
        assert append(L, c, rot=rot) == 1 and "rot" in msg(L)
    assert needs_device(append(L, c, rot=16)) and needs_device(append(L, c, rot=48, inter=1))
    assert append(L, c, max_pos=-1) == 1 and append(L, c, max_pos=1 << 31) == 1
    assert needs_device(append(L, c, max_pos=0, cos=N0, sin=N0))
    assert append(L, c, qs=255) == 1 and append(L, c, qs=260) == 1 and append(L, c, ks=127) == 1 and append(L, c, vs=130) == 1
    assert append(L, c, qs=1 << 31) == 1
    assert needs_device(append(L, c, T=1, qs=0, ks=5, vs=1 << 40)) and needs_device(append(L, c, dt=0, qs=260, ks=132, vs=132))
    for bad in ("q", "k", "v", "cos", "sin", "pos", "slots", "out"):
        assert append(L, c, **{bad: N0}) == 1 and "null" in msg(L)
    for bad in ("q", "k", "v", "cos", "sin", "out"):
        assert append(L, c, **{bad: A + 8}) == 1 and "aligned" in msg(L)
    assert append(L, c, pos=A + 2) == 1 and append(L, c, slots=A + 1) == 1 and needs_device(append(L, c, pos=A + 4, slots=A + 4))
    assert append(L, c, T=0, q=N0, k=N0, v=N0, cos=N0, sin=N0, pos=N0, slots=N0, out=N0) == 0


def test_move_arguments(L):
    c = cache()
    assert move(L, c, M=-1, S=-1) == 1 and move(L, c, M=1 << 31, S=1 << 31) == 1 and move(L, c, starts=A, S=-1) == 1
    assert move(L, c, M=3, S=2) == 1 and "without starts" in msg(L)
    assert needs_device(move(L, c, starts=A, S=2)) and needs_device(move(L, c, starts=A + 4, S=1))
    for bad in ("src", "dst"):
        assert move(L, c, **{bad: N0}) == 1 and move(L, c, **{bad: A + 2}) == 1
    assert move(L, c, starts=A + 2, S=2) == 1
    # 64 elements NVFP4: two code pieces and one scale piece a side
    assert move(L, c, M=357913941, S=357913941) == 2 and "2^31" in msg(L)
    assert needs_device(move(L, cache(heads=1), M=357913941, S=357913941))
    assert move(L, c, M=0, S=0, src=N0, dst=N0) == 0 and move(L, c, starts=A, S=0) == 0
    assert move(L, c, M=0, src=N0, dst=N0, starts=A, S=5) == 0


def test_tree_arguments(L):
    c = cache()
    assert tree(L, c, mask=N0) == 1 and "tree_mask" in msg(L)
    assert tree(L, c, q_start=N0) == 1 and "q_start" in msg(L)
    assert tree(L, c, mask=A + 2) == 1 and needs_device(tree(L, c, mask=A + 4))
    for words, max_q, T, ok in ((0, 1, 9, False), (1, 32, 99, True), (1, 33, 99, False), (2, 64, 99, True), (2, 65, 99, False),
                                (1, 1 << 30, 32, True), (1, 1 << 30, 33, False), (-1, 4, 9, False), ((1 << 20) + 1, 4, 9, False)):
        st = tree(L, c, words=words, max_q=max_q, T=T)
        assert (needs_device(st) if ok else st == 1 and "words" in msg(L)), (words, max_q, T)
    # what kv_attention refuses
    assert tree(L, c, dt=0) == 2 and tree(L, c, Hq=3) == 1 and tree(L, c, T=-1) == 1 and tree(L, c, max_kv=65) == 1
    assert tree(L, c, window=-1) == 1 and tree(L, c, scale=float("nan")) == 1 and tree(L, c, stride=260) == 1
    for bad in ("q", "out", "kv_len", "table"):
        assert tree(L, c, **{bad: N0}) == 1 and "null" in msg(L)
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(lse=A + 2), dict(ws=A + 8, ws_bytes=64)):
        assert tree(L, c, **bad) == 1 and "aligned" in msg(L)
    assert tree(L, c, B=0, T=0, q=N0, out=N0, kv_len=N0, table=N0, mask=N0, words=0) == 0
    assert tree(L, c, max_q=0, words=0, mask=N0) == 0
    assert needs_device(tree(L, c, window=1 << 40)) and needs_device(tree(L, c, max_kv=0, max_pages=0, table=N0))
    assert "[kv_attention_tree]" in msg(L)
    assert needs_device(attend(L, c)) and "[kv_attention]" in msg(L)


def test_the_binding_checks_its_tensors(monkeypatch):
    c = host_cache(monkeypatch)  # 4 pages of 16 rows, 2 heads of 64
    monkeypatch.setattr(nv, "_need_cache", lambda cache: 0)
    monkeypatch.setattr(nv, "_need_rows", lambda t, shape, what, dev: t.stride()[0])
    b, f, i = torch.bfloat16, torch.float32, torch.int32
    q, k, v, cos, at = e(3, 4, 64, dtype=b), e(3, 2, 64, dtype=b), e(3, 2, 64, dtype=b), e(9, 32, dtype=f), e(3, dtype=i)

    def call(**kw):
        a = dict(q=q, k=k, v=v, cos=cos, sin=cos, positions=at, slots=at)
        a.update(kw)
        return nv.kv_cache_append(c, **a)

    for bad, what in ((dict(q=e(3, 4, 64, dtype=f)), "share a dtype"), (dict(v=e(3, 2, 64, dtype=torch.float16)), "share a dtype"),
                      (dict(q=e(3, 256, dtype=b)), r"q must be \[T"), (dict(cos=e(9, 32, dtype=b)), "cos"), (dict(sin=e(9, 16, dtype=f)), "cos and sin"),
                      (dict(positions=e(2, dtype=i)), "positions"), (dict(positions=e(3, dtype=torch.int64)), "positions"),
                      (dict(slots=e(3, dtype=torch.int64)), "slots"), (dict(q_out=e(3, 4, 64, dtype=f)), "q_out"),
                      (dict(q_out=e(2, 4, 64, dtype=b)), "q_out")):
        with pytest.raises(ValueError, match=what):
            call(**bad)
    for bad, what in ((dict(src=e(3, dtype=torch.int64), dst=at), "src"), (dict(src=at, dst=e(2, dtype=i)), "src and dst"),
                      (dict(src=at, dst=at, starts=e(0, dtype=i)), "starts"), (dict(src=at, dst=at, starts=e(2, dtype=f)), "starts")):
        with pytest.raises(ValueError, match=what):
            nv.kv_cache_move(c, **bad)
    table, n = e(1, 4, dtype=i), e(1, dtype=i)
    for bad, what in ((e(3, 1, dtype=torch.int64), "tree_mask must be torch.int32"), (e(2, 1, dtype=i), "tree_mask must be"),
                      (e(3, dtype=i), "tree_mask must be")):
        with pytest.raises(ValueError, match=what):
            nv.kv_attention_tree(c, q, table, n, bad, e(2, dtype=i))


def test_the_binding_passes_masks_on(monkeypatch):
    """kv_attention and kv_attention_tree share their argument handling."""
    c = host_cache(monkeypatch)
    monkeypatch.setattr(nv, "_need_cache", lambda cache: 0)
    monkeypatch.setattr(nv, "_need_rows", lambda t, shape, what, dev: t.stride()[0])
    monkeypatch.setattr(nv, "_stream", lambda: None)
    seen = []
    real = nv.lib()
    fake = types.SimpleNamespace(kv_attention=lambda *a: seen.append(("plain", a)) or 0, kv_attention_tree=lambda *a: seen.append(("tree", a)) or 0,
                                 kv_attention_workspace_size=real.kv_attention_workspace_size,
                                 kv_attention_tree_workspace_size=real.kv_attention_tree_workspace_size)
    monkeypatch.setattr(nv, "lib", lambda: fake)
    i = torch.int32
    q, table, n, starts, mask = e(5, 4, 64, dtype=torch.bfloat16), e(1, 4, dtype=i), e(1, dtype=i), e(2, dtype=i), e(5, 3, dtype=i)
    nv.kv_attention(c, q, table, n, starts, 5, 60, causal=False, window=7)
    out, lse = nv.kv_attention_tree(c, q, table, n, mask, starts, 5, 60, window=7, return_lse=True)
    (k0, a), (k1, t) = seen
    assert (k0, k1) == ("plain", "tree")
    assert a[:7] == t[:7] and t[7:9] == (mask.data_ptr(), 3) and a[7:14] == t[9:16]
    assert a[7:14] == (1, 5, 4, 5, 60, 4, 64 ** -0.5) and a[14:16] == (False, 7) and t[16] == 7
    assert t[17] == out.data_ptr() and t[18] == lse.data_ptr()


@pytest.mark.parametrize("args,want", [
    # B, T, Hq, heads, D, max_q, max_kv, window; up to 32 rows k_kv_decode's tiles of 16: 592 workers, two partial results each
    ((1, 8, 32, 8, 128, 8, 1000), 592 * (2 * 16 * (4 * 128 + 8) + 32)),
    ((1, 1, 32, 8, 128, 1, 1000), 592 * (2 * 16 * (4 * 128 + 8) + 32)),
    ((1, 8, 32, 8, 128, 8, 64), 0),                      # one unit of tokens: nothing to split
    # 8 row tiles of 256: 16 chunks of 512 tokens, 128 CTAs of 5 + 4 tiles' time and the join's 3
    ((1, 64, 32, 8, 128, 64, 8192), 16 * 64 * 32 * (4 * 128 + 8)),
    # 144 row tiles fill the GPU: no chunks (what is left is k_kv_decode's, for types that k_kv_prefill does not take)
    ((18, 18 * 64, 32, 8, 128, 64, 4160), 592 * (2 * 16 * (4 * 128 + 8) + 32)),
])
def test_tree_workspace_sizes(L, args, want):
    assert nv.kv_attention_tree_workspace_size(*args) == want


def test_tree_workspace_of_bad_sizes(L):
    for bad in ((-1, 1, 4, 1, 64, 1, 100), (1, 1, 4, 3, 64, 1, 100), (1, 1, 4, 1, 48, 1, 100), (1, 1, 4, 1, 64, 1, -1), (1, 1, 4, 0, 64, 1, 100)):
        assert nv.kv_attention_tree_workspace_size(*bad) == 0
    for kv in (0, 1, 127, 128, 129, 1 << 20, 1 << 30):
        for B, n in ((1, 64), (40, 64), (1, 5000)):
            assert nv.kv_attention_tree_workspace_size(B, B * n, 32, 8, 128, n, kv) <= max(64 * B * n * 32 * 520, 592 * (32 * 520 + 32))
