"""Calls that overlap on several streams, each with outputs and workspaces of
its own, give the bits that the same calls give alone, time after time."""
import pytest
import torch

from kv_reference import seeded
from test_gpu_kv_append import i32
from test_gpu_kv_attention import make
from test_gpu_kv_tree import starts_of
from tree_reference import ancestors, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def jobs(nv):
    g = torch.tensor([7.0], device="cuda")
    for rows, K in ((1500, 4096), (2500, 1008), (300, 8208)):
        x, res, dy, w = (seeded(s, 3 + i) for i, s in enumerate(((rows, K), (rows, K), (rows, K), (K,))))

        def norm(x=x, res=res, dy=dy, w=w):
            c, s, h, r = nv.rms_norm_quantize(x, w, "nvfp4", g, 1e-5, res, "swizzled", return_rstd=True)
            return c, s, h, r, *nv.rms_norm_vjp(dy, h, w, r, res)

        yield norm
    # split over workers and joined (6 and 30 drafts), whole (60, of 16 sequences)
    for B, n, L in ((1, 6, 3000), (1, 30, 3000), (16, 60, 500)):
        lens = [L - 7 * b for b in range(B)]
        c, t = make(nv, "nvfp4", lens, 2, 128, 16, 3)
        q, mask = seeded((B * n, 8, 128), 5), pack([m for b in range(B) for m in ancestors(n, b)], 2).cuda()
        kv_len, starts = i32(lens), i32(starts_of([n] * B))

        def tree(c=c, t=t, q=q, mask=mask, kv_len=kv_len, starts=starts, n=n, L=L):
            return nv.kv_attention_tree(c, q, t, kv_len, mask, starts, n, L, return_lse=True)

        yield tree


def test_on_three_streams(nv):
    calls = list(jobs(nv))
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for k in range(len(calls) * 4):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                at = (k + i * (1 + k // len(calls))) % len(calls)
                got += [(at, calls[at]()) for _ in range(2)]
        torch.cuda.synchronize()
        for at, out in got:
            for a, b in zip(out, want[at]):
                assert torch.equal(a, b)
    nv.check_device_errors()
