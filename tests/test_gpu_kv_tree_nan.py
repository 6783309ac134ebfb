"""kv_attention_tree over an NVFP4 cache with block scales of NaN (bytes 0x7F
and 0xFF): among the keys they make the queries that see the token NaN, and no
others; among the values they count as 0.  Alike for few query rows and for
many, which two kernels take."""
import pytest
import torch

from kv_reference import cache_sides, check, seeded
from test_gpu_kv_attention import i32, make
from test_gpu_kv_tree import starts_of
from tree_reference import ancestors, attention_tree, pack

pytestmark = pytest.mark.gpu

# rows of a key/value head and D: k_kv_decode (12 of 64 and 96, 4 of 256), then k_kv_prefill (18 of 256; 120: one query
# tile, whose tokens two slots take in turn; 240 and 260: two)
SHAPES = [(6, 2, 64), (6, 2, 96), (2, 2, 256), (9, 2, 256), (30, 4, 128), (60, 4, 64), (65, 4, 96)]


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def trees(nv, n, G, D):
    lens = [n + 70, 300]
    c, t = make(nv, "nvfp4", lens, 2, D, 16, 3)
    masks = [m for b in range(2) for m in ancestors(n, b)]
    return c, t, lens, masks, seeded((2 * n, 2 * G, D), 5)


def run(nv, c, t, lens, masks, q, n):
    words = -(-n // 32)
    out, lse = nv.kv_attention_tree(c, q, t, i32(lens), pack(masks, words).cuda(), i32(starts_of([n, n])), n, return_lse=True)
    nv.check_device_errors()
    return out, lse


def place(t, j, b):
    return int(t[b, j // 16]), j % 16


@pytest.mark.parametrize("n,G,D", SHAPES)
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_keys(nv, n, G, D, byte):
    # a draft in the middle (its own branch sees it), the root (all drafts do), a token of the context
    for b, j in ((0, 70 + n // 2), (1, 300 - n), (1, 5)):
        c, t, lens, masks, q = trees(nv, n, G, D)
        page, row = place(t, j, b)
        c.k_scales[page, 1, row, (D // 16) // 2] = byte
        out, lse = run(nv, c, t, lens, masks, q, n)
        o, l, tol, ltol = attention_tree(cache_sides(c), q, t, lens, [0, n, 2 * n], masks, D ** -0.5)
        hit = torch.isnan(l)
        d = j - (lens[b] - n)
        sees = [b * n + i for i in range(n) if d < 0 or masks[b * n + i] >> d & 1]
        want = torch.zeros(2 * n, 2 * G, dtype=torch.bool)
        want[sees, G:] = True
        assert torch.equal(hit, want) and sees
        assert torch.isnan(lse.cpu()[hit]).all() and torch.isnan(out.cpu()[hit]).all()
        check(out, o, tol, "out")
        check(lse, l, ltol, "lse")


@pytest.mark.parametrize("n,G,D", SHAPES)
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_values(nv, n, G, D, byte):
    c, t, lens, masks, q = trees(nv, n, G, D)
    for b, j in ((0, 70 + n // 2), (1, 300 - n), (1, 5)):
        page, row = place(t, j, b)
        c.v_scales[page, 1, row, (D // 16) // 2] = byte
    out, lse = run(nv, c, t, lens, masks, q, n)
    K, V = cache_sides(c)
    o, l, tol, ltol = attention_tree((K, torch.nan_to_num(V)), q, t, lens, [0, n, 2 * n], masks, D ** -0.5)
    assert not torch.isnan(l).any()
    check(out, o, tol, "out")
    check(lse, l, ltol, "lse")
