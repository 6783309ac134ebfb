"""The norm's kernels where a CTA has several rows to do one after the other:
more rows than the grid takes at once, with one and with several warps a row,
of both layouts of a row over its threads, and ragged last steps.

Rows that are enough for that, 148 SMs: k_rms_norm has as many CTAs as fit the
GPU, at most 148 * (2048 / threads of a CTA), of (warps of a CTA) / (warps of a
row) rows each; k_rms_norm_vjp at most 296 (148 above K 4096) CTAs, of two such
rows a step (one of fp32)."""
import numpy as np
import pytest
import torch

from helpers import raw
from norm_reference import forward64, vjp64, vjp_tolerance
from test_gpu_norm import G, oracle

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def seeded(shape, seed, dtype=bf16, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def inputs(rows, K, dtype, seed, sixteen=False):
    """x, residual, weight, of rows 16-byte aligned only if asked."""
    offset = 16 // torch.empty(0, dtype=dtype).element_size() if sixteen else 0

    def at(t):
        s = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        s[offset:] = t.reshape(-1)
        return s[offset:].view(t.shape)

    x, res = seeded((rows, K), seed, dtype), seeded((rows, K), seed + 1, dtype, 3.0)
    x[1], res[1] = 0, 0             # nothing but eps
    x[2, 0] = 200.0                 # one channel far above the rest
    x[rows - 1] *= 2.0 ** -10
    return at(x), at(res), at(seeded((K,), seed + 2, dtype, 0.3) + 1)


# The definition's fp32 steps, as in test_gpu_norm.py but on the GPU (elementary operations, each rounded).
def steps(h, r, w):
    return (h.float() * r[:, None]) * w.float()


def summed(x, res):
    return (x.float() + res.float()).to(x.dtype)


def check_r(h, r, eps):
    r64 = forward64(h.double(), torch.ones(1, dtype=torch.float64, device="cuda"), eps)[1]
    assert ((r.double() / r64 - 1).abs() <= 2.0 ** -24 + (h.shape[1] + 8) * 2.0 ** -53).all()


# rows, K, whether rows are 16-byte aligned only.  Warps a row and rows a CTA: 2 and 4; 8 and 1; 16 and 1; four blocks a
# thread: 5 and 1 (at most 12 CTAs of 160 threads an SM), 1 and 8, 2 and 4
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows,K,sixteen", [(5003, 1008, False), (2500, 4096, False), (1301, 8192, False), (2000, 8208, False),
                                            (10007, 1024, True), (5003, 2064, True)])
def test_plain(nv, dtype, rows, K, sixteen):
    x, res, w = inputs(rows, K, dtype, rows + K, sixteen)
    y, h, r = nv.rms_norm(x, w, 1e-5, res, return_rstd=True)
    want = summed(x, res)
    assert torch.equal(h, want)
    check_r(h, r, 1e-5)
    assert torch.equal(y, steps(h, r, w).to(dtype))
    # in place: the next row's loads are in flight beside these stores
    for in_place_of in ("x", "residual"):
        a, b, _ = inputs(rows, K, dtype, rows + K, sixteen)
        got = nv.rms_norm(a, w, 1e-5, b, h=a if in_place_of == "x" else b, return_rstd=True)
        assert torch.equal(got[0], y) and torch.equal(got[1], h) and torch.equal(got[2], r)
    # without a residual
    y, h2, r = nv.rms_norm(x, w, 1e-5, return_rstd=True)
    check_r(x, r, 1e-5)
    assert h2 is x and torch.equal(y, steps(x, r, w).to(dtype))
    nv.check_device_errors()


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,K,sixteen,layout", [(5003, 992, False, "swizzled"), (2500, 4096, False, "linear"), (1301, 8192, False, "swizzled"),
                                                   (2000, 8224, False, "linear"), (10007, 1024, True, "linear"), (5003, 2080, True, "swizzled")])
def test_codes(nv, orc, mode, rows, K, sixteen, layout):
    x, res, w = inputs(rows, K, bf16, rows + K, sixteen)
    g = torch.tensor([G], device="cuda") if mode == "nvfp4" else None
    c, s, h, r = nv.rms_norm_quantize(x, w, mode, g, 1e-6, res, layout, h=x, return_rstd=True)
    assert h is x
    check_r(h, r, 1e-6)
    y = steps(h, r, w)
    # every row against the quantizer of y (which its own tests hold to the oracle's), some against the oracle
    want = nv.nvfp4_quantize(y, g, layout) if mode == "nvfp4" else (nv.mxfp8_quantize if mode == "mxfp8" else nv.mxfp4_quantize)(y, layout)
    assert torch.equal(c, want[0]) and torch.equal(s, want[1])
    some = [0, 1, 2, rows // 2, rows - 130, rows - 2, rows - 1]
    oc, os_ = oracle(orc, mode, y[some].cpu(), None if g is None else G, "linear")
    assert np.array_equal(raw(c[some]), oc)
    if layout == "linear":
        assert np.array_equal(raw(s[some]), os_)
    nv.check_device_errors()


# Steps a CTA: two and three of eight rows side by side, of four, of one (K 4096, 8192), and three rows of the kernel that
# reads them twice (K 8208); the last one ragged, with and without a step's second row
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows,K", [(5003, 512), (12007, 512), (2500, 1008), (6007, 1008), (1500, 4096), (700, 8192), (700, 8208)])
@pytest.mark.parametrize("past", [True, False])
def test_gradient(nv, dtype, rows, K, past):
    x, dh, w = inputs(rows, K, dtype, rows + K)
    dy = seeded((rows, K), 9, dtype)
    r = nv.rms_norm(x, w, 1e-5, return_rstd=True)[2]
    d64 = [t.double() for t in (dy, x, w, r)] + [dh.double() if past else None]
    want, tol = vjp64(*d64), vjp_tolerance(*d64, dtype)
    n = nv.rms_norm_vjp_workspace_size(rows, K)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    dx, dw = nv.rms_norm_vjp(dy, x, w, r, dh if past else None, workspace=ws[:n])
    assert (ws[n:] == 0x5A).all()
    for got, v, t in zip((dx, dw), want, tol):
        bad = ~((got.double() - v).abs() <= t)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
    # the same bits every time, in place as well (the next step's copies are in flight beside these stores)
    for _ in range(2):
        a, b = dy.clone(), dh.clone()
        got = nv.rms_norm_vjp(a, x, w, r, b if past else None, dx=a)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
        if past:
            got = nv.rms_norm_vjp(dy, x, w, r, b, dx=b)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    # without dw
    dx2 = torch.empty_like(dx)
    st = nv.lib().rms_norm_vjp(dy.data_ptr(), x.data_ptr(), w.data_ptr(), r.data_ptr(), dh.data_ptr() if past else None, nv.DT[dtype],
                               rows, K, dx2.data_ptr(), None, None, 0, nv._stream())
    assert st == 0 and torch.equal(dx2, dx)
    nv.check_device_errors()


def test_rows_do_not_mix(nv):
    """Rows of one value each, many to a CTA: a sum or a factor taken from a
    neighbour, or from the row before, would show in every element."""
    for rows, K in ((5003, 1008), (2500, 4096), (12007, 512), (700, 8208)):
        v = torch.arange(1, rows + 1, device="cuda", dtype=f32)[:, None]
        x = v.expand(rows, K).contiguous()
        w = torch.ones(K, device="cuda")
        y, _, r = nv.rms_norm(x, w, 2.0 ** -126, return_rstd=True)
        # with u = 2^-24: r is 1 / v within half a step, u, and the error of the 64-bit root
        assert ((r.double() * v[:, 0].double() - 1).abs() <= 2.0 ** -24 * (1 + 2.0 ** -20)).all()
        assert torch.equal(y, (v * r[:, None]).expand(rows, K))
        # dy = 1: s = K v without an error (integers below 2^24), f = s (1 / K) r r with four roundings, (v r)^2 within
        # 2 u of 1: dx = r (1 - v f) is r times at most 6 u, and a product's rounding
        dx, dw = nv.rms_norm_vjp(torch.ones_like(x), x, w, r)
        assert (dx.abs() <= r[:, None] * 7 * 2.0 ** -24).all()
        # dw sums rows numbers within 2 u of 1 (r, and its product with v), at most 64 additions one after the other: up
        # to 9 rows of a CTA, 7 rows side by side, 3 parts of a group, 2 shuffles, 32 warps
        assert ((dw.double() - rows).abs() <= rows * (64 + 3) * 2.0 ** -24).all()
