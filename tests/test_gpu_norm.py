"""GPU parity of the root-mean-square norm: with the kernel's own factor r
(itself held to its 64-bit value) h, y, codes and scales are the same bits as
the definition's fp32 steps and the oracle's quantizers; its gradient lies
within norm_reference's tolerance."""
import numpy as np
import pytest
import torch

from helpers import raw
from kv_reference import seeded
from norm_reference import forward64, vjp64, vjp_tolerance

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
G = 7.0


@pytest.fixture(scope="module")
def nv():
    from mxfp8_block_scaled_nvfp4_b200 import build, nvfp4
    build.build()
    return nvfp4


def inputs(rows, K, dtype, seed, residual=True, offset=0):
    """x, residual, weight; offset: elements that each tensor's storage begins before it."""
    def at(t):
        s = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        s[offset:] = t.reshape(-1)
        return s[offset:].view(t.shape)

    x, res = seeded((rows, K), seed, dtype), seeded((rows, K), seed + 1, dtype, 3.0)
    if rows > 2:
        x[1], res[1] = 0, 0             # nothing but eps
        x[2, 0] = 200.0                 # one channel far above the rest
        x[rows - 1] *= 2.0 ** -10
    w = seeded((K,), seed + 2, dtype, 0.3) + 1
    return at(x), at(res) if residual else None, at(w)


def steps(h, r, w):
    """fp32 y on the CPU: each product rounded."""
    return (h.float().cpu() * r.cpu()[:, None]) * w.float().cpu()


def check_r(h, r, eps):
    r64 = forward64(h.double().cpu(), torch.ones(1, dtype=torch.float64), eps)[1]
    tol = 2.0 ** -24 + (h.shape[1] + 8) * 2.0 ** -53
    assert ((r.double().cpu() / r64 - 1).abs() <= tol).all()


def summed(x, res):
    return x if res is None else (x.float().cpu() + res.float().cpu()).to(x.dtype)


SHAPES = [(1, 16), (5, 48), (3, 512), (37, 1008), (9, 4096), (4, 5120), (2, 8192), (3, 8208), (2, 32768)]


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_plain(nv, dtype, rows, K, residual):
    for offset in (0, 16 // torch.empty(0, dtype=dtype).element_size()):  # 32- and 16-byte aligned
        x, res, w = inputs(rows, K, dtype, rows + K, residual, offset)
        y, h, r = nv.rms_norm(x, w, 1e-5, res, return_rstd=True)
        assert torch.equal(h.cpu(), summed(x, res).cpu())
        check_r(h, r, 1e-5)
        assert torch.equal(y.cpu(), steps(h, r, w).to(dtype))
        y2, h2 = nv.rms_norm(x, w, 1e-5, res)
        assert torch.equal(y2, y) and torch.equal(h2, h)
    nv.check_device_errors()


def oracle(orc, mode, y, g, layout):
    y = np.ascontiguousarray(y.numpy())
    if mode == "nvfp4":
        c, s = orc.nvfp4_quantize(y, "f32", g)
    else:
        c, s = (orc.mxfp8_quantize if mode == "mxfp8" else orc.mxfp4_quantize)(y, "f32")
    return c, orc.swizzle_scales(s) if layout == "swizzled" else s


@pytest.mark.parametrize("mode", ["nvfp4", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("layout", ["linear", "swizzled"])
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (130, 288), (33, 1024), (9, 4096), (2, 8224)])
def test_codes(nv, orc, mode, dtype, layout, rows, K):
    for offset in (0, 16 // torch.empty(0, dtype=dtype).element_size()):
        x, res, w = inputs(rows, K, dtype, rows + K, rows != 33, offset)
        g = torch.tensor([G], device="cuda") if mode == "nvfp4" and rows != 5 else None
        c, s, h, r = nv.rms_norm_quantize(x, w, mode, g, 1e-6, res, layout, return_rstd=True)
        assert torch.equal(h.cpu(), summed(x, res).cpu())
        check_r(h, r, 1e-6)
        oc, os_ = oracle(orc, mode, steps(h, r, w), None if g is None else G, layout)
        assert np.array_equal(raw(c), oc) and np.array_equal(raw(s), os_)
    nv.check_device_errors()


def test_nvfp4_blocks_of_an_odd_row(nv, orc):
    """K = 16 j for odd j: scale bytes that four blocks do not share a word for."""
    for rows, K in ((7, 16), (129, 48), (20, 1008)):
        x, res, w = inputs(rows, K, bf16, K)
        for layout in ("linear", "swizzled"):
            c, s, h, r = nv.rms_norm_quantize(x, w, "nvfp4", None, 1e-6, res, layout, return_rstd=True)
            oc, os_ = oracle(orc, "nvfp4", steps(h, r, w), None, layout)
            assert np.array_equal(raw(c), oc) and np.array_equal(raw(s), os_)


def test_many_rows(nv, orc):
    """More rows than the grid takes at once."""
    rows, K = 4100, 512
    x, res, w = inputs(rows, K, bf16, 1)
    c, s, h, r = nv.rms_norm_quantize(x, w, "mxfp8", None, 1e-6, res, "swizzled", return_rstd=True)
    check_r(h, r, 1e-6)
    oc, os_ = oracle(orc, "mxfp8", steps(h, r, w), None, "swizzled")
    assert np.array_equal(raw(c), oc) and np.array_equal(raw(s), os_)
    y, _ = nv.rms_norm(x, w, 1e-6, res)
    assert torch.equal(y.cpu(), steps(h, r, w).to(bf16))


def test_extreme_rows(nv):
    """Squares beyond fp32's range, both ends, and a NaN that stays in its row."""
    x = seeded((6, 256), 1, f32)
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -100
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(256, device="cuda")
    y, _, r = nv.rms_norm(x, w, 2.0 ** -126, return_rstd=True)
    good = [0, 1, 4, 5]
    check_r(x[good], r[good], 2.0 ** -126)
    assert torch.equal(y[good].cpu(), steps(x[good], r[good], w))
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 9]) and (y[3, :9] == 0).all()


def test_in_place_and_outputs_given(nv):
    x, res, w = inputs(11, 640, bf16, 3)
    y, h = nv.rms_norm(x, w, 1e-5, res)
    for target in ("x", "residual"):
        a, b = x.clone(), res.clone()
        out, r = torch.empty_like(x), torch.empty(11, device="cuda")
        got = nv.rms_norm(a, w, 1e-5, b, out=out, h=a if target == "x" else b, rstd=r)
        assert got[0] is out and got[1] is (a if target == "x" else b) and got[2] is r
        assert torch.equal(out, y) and torch.equal(got[1], h)
        assert torch.equal(b if target == "x" else a, res if target == "x" else x)
    y3, h3 = nv.rms_norm(x.view(1, 11, 640), w, 1e-5, res.view(1, 11, 640))
    assert y3.shape == h3.shape == (1, 11, 640) and torch.equal(y3[0], y)
    assert nv.rms_norm(x[:0], w, 1e-5)[0].shape == (0, 640)
    c, s, _ = nv.rms_norm_quantize(x[:0], w, "nvfp4", layout="swizzled")
    assert c.shape[0] == 0


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("rows,K", [(1, 16), (5, 48), (700, 512), (37, 1008), (9, 4096), (3, 8192), (3, 8208), (2, 32768)])
@pytest.mark.parametrize("past", [True, False])
def test_gradient(nv, dtype, rows, K, past):
    for offset in (0, 16 // torch.empty(0, dtype=dtype).element_size()):
        x, dh, w = inputs(rows, K, dtype, rows + K, True, offset)
        dy = torch.empty(x.numel() + offset, dtype=dtype, device="cuda")[offset:].view(x.shape)
        dy.copy_(seeded((rows, K), 9, dtype))
        r = nv.rms_norm(x, w, 1e-5, return_rstd=True)[2]
        d64 = [t.double().cpu() for t in (dy, x, w, r)] + [dh.double().cpu() if past else None]
        want, tol = vjp64(*d64), vjp_tolerance(*d64, dtype)
        dx, dw = nv.rms_norm_vjp(dy, x, w, r, dh if past else None)
        assert dw.dtype == f32
        for got, v, t in zip((dx, dw), want, tol):
            bad = ~((got.double().cpu() - v).abs() <= t)
            assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
        again = nv.rms_norm_vjp(dy, x, w, r, dh if past else None)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # the same bits every time
    nv.check_device_errors()


def test_gradient_in_place_and_of_no_rows(nv):
    x, dh, w = inputs(13, 640, bf16, 3)
    dy = seeded((13, 640), 4, bf16)
    r = nv.rms_norm(x, w, 1e-5, return_rstd=True)[2]
    dx, dw = nv.rms_norm_vjp(dy, x, w, r, dh)
    a, b = dy.clone(), dh.clone()
    assert torch.equal(nv.rms_norm_vjp(a, x, w, r, b, dx=a)[0], dx)
    assert torch.equal(nv.rms_norm_vjp(dy, x, w, r, b, dx=b)[0], dx)
    dw0 = nv.rms_norm_vjp(dy[:0], x[:0], w, r[:0])[1]
    assert (dw0 == 0).all()
    # a workspace of just the size, with a guard behind it
    n = nv.rms_norm_vjp_workspace_size(13, 640)
    ws = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    got = nv.rms_norm_vjp(dy, x, w, r, dh, workspace=ws[:n])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and (ws[n:] == 0x5A).all()
    # without dw no workspace is needed
    dx2 = torch.empty_like(dx)
    st = nv.lib().rms_norm_vjp(dy.data_ptr(), x.data_ptr(), w.data_ptr(), r.data_ptr(), dh.data_ptr(), 2, 13, 640,
                               dx2.data_ptr(), None, None, 0, nv._stream())
    assert st == 0 and torch.equal(dx2, dx)


def test_training_step_of_a_quantized_product(nv):
    """Norm, product and back: the gradients that rms_norm_vjp makes of
    qqmm_vjp's are the formula's on the tensors in between."""
    rows, K, N = 128, 256, 128
    x, res, w = inputs(rows, K, bf16, 5)
    W = seeded((N, K), 8, bf16, 0.1)
    g = torch.tensor([G], device="cuda")
    c, s, h, r = nv.rms_norm_quantize(x, w, "nvfp4", g, 1e-5, res, "swizzled", return_rstd=True)
    g_w = nv.amax(W)
    wc, ws = nv.nvfp4_quantize(W, g_w, "swizzled")
    z = nv.qqmm(c, s, wc, ws, K, "nvfp4", g, g_w)
    y = nv.nvfp4_dequantize(c, s, g, "swizzled")
    dz = seeded((rows, N), 9, bf16)
    dy, _ = nv.qqmm_vjp(y, W, dz, g, g_w)
    dh = seeded((rows, K), 10, bf16)
    dx, dw = nv.rms_norm_vjp(dy, h, w, r, dh)
    d64 = [t.double().cpu() for t in (dy, h, w, r, dh)]
    for got, v, t in zip((dx, dw), vjp64(*d64), vjp_tolerance(*d64, bf16)):
        assert ((got.double().cpu() - v).abs() <= t).all()
    assert z.shape == (rows, N)


def test_in_a_graph_on_another_stream(nv):
    x, res, w = inputs(64, 512, bf16, 5)
    dy = seeded((64, 512), 6, bf16)
    g = torch.tensor([G], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nv.rms_norm_quantize(x, w, "nvfp4", g, 1e-5, res, "swizzled")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c, sc, h, r = nv.rms_norm_quantize(x, w, "nvfp4", g, 1e-5, res, "swizzled", return_rstd=True)
            dx, dw = nv.rms_norm_vjp(dy, h, w, r, res)
        for seed in (11, 12):
            x.copy_(seeded((64, 512), seed, bf16))
            graph.replay()
            s.synchronize()
            c2, sc2, h2, r2 = nv.rms_norm_quantize(x, w, "nvfp4", g, 1e-5, res, "swizzled", return_rstd=True)
            dx2, dw2 = nv.rms_norm_vjp(dy, h2, w, r2, res)
            s.synchronize()
            for a, b in ((c, c2), (sc, sc2), (h, h2), (r, r2), (dx, dx2), (dw, dw2)):
                assert torch.equal(a, b)
