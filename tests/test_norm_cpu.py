"""Host-side checks of the norm calls (no GPU), and the gradient formula the
GPU tests use against differences."""
import pytest
import torch

from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv
from norm_reference import forward64, vjp64
from test_kv_cpu import A, L, N0, e, msg, needs_device  # noqa: F401 (L is a fixture)

INF, NAN = float("inf"), float("nan")


def norm(L, x=A, res=A, w=A, dt=2, rows=3, K=64, eps=1e-5, h=A, y=A, rstd=N0):
    return L.rms_norm(x, res, w, dt, rows, K, eps, h, y, rstd, N0)


def quant(L, mode=0, x=A, res=A, w=A, dt=2, rows=3, K=64, eps=1e-5, g=N0, h=A, codes=A, scales=A, layout=0, rstd=N0):
    return L.rms_norm_quantize(mode, x, res, w, dt, rows, K, eps, g, h, codes, scales, layout, rstd, N0)


def vjp(L, dy=A, h=A, w=A, rstd=A, dh=A, dt=2, rows=3, K=64, dx=A, dw=A, ws=A, ws_bytes=1 << 30):
    return L.rms_norm_vjp(dy, h, w, rstd, dh, dt, rows, K, dx, dw, ws, ws_bytes, N0)


@pytest.mark.parametrize("call", [norm, quant, vjp])
def test_shapes_and_pointers(L, call):
    assert needs_device(call(L)) and needs_device(call(L, dt=0)) and needs_device(call(L, K=32768, rows=1))
    assert call(L, dt=5) == 2 and "dtype" in msg(L)
    assert call(L, rows=-1) == 1 and call(L, rows=1 << 40) == 1 and call(L, rows=1 << 62) == 1
    assert call(L, K=0) == 1 and call(L, K=-16) == 1 and call(L, K=24) == 1 and "multiple of 16" in msg(L)
    assert call(L, K=32768 + 64) == 2 and "at most 32768" in msg(L)
    assert call(L, w=N0) == 1 and "null" in msg(L)
    assert call(L, w=A + 8) == 1 and "aligned" in msg(L)
    assert call(L, rstd=A + 2) == 1
    assert call(L, h=A + 8) == 1


def test_the_forward_calls(L):
    for call in (norm, quant):
        assert call(L, res=N0) == 1 and call(L, h=N0) == 1 and "only then" in msg(L)  # h and the residual go together
        assert needs_device(call(L, res=N0, h=N0)) and needs_device(call(L, rstd=A + 4))
        for eps in (0.0, -1e-5, INF, NAN, 2.0 ** -127, 2.0 ** 127):
            assert call(L, eps=eps) == 1 and "eps" in msg(L)
        assert needs_device(call(L, eps=2.0 ** -126))
        assert call(L, x=N0) == 1 and call(L, x=A + 4) == 1 and call(L, res=A + 8) == 1
        assert call(L, rows=0, x=N0, res=N0, w=N0, h=N0) == 0
    assert norm(L, y=N0) == 1 and norm(L, y=A + 8) == 1
    assert quant(L, codes=N0) == 1 and quant(L, scales=N0) == 1 and quant(L, codes=A + 8) == 1 and quant(L, scales=A + 4) == 1
    assert quant(L, mode=3) == 1 and "mode" in msg(L)
    assert quant(L, layout=2) == 1 and "layout" in msg(L)
    assert quant(L, mode=1, g=A) == 1 and quant(L, mode=2, g=A) == 1 and "only supported for 'nvfp4'" in msg(L)
    assert needs_device(quant(L, g=A)) and quant(L, g=A + 2) == 1
    assert quant(L, mode=1, K=48) == 1 and "multiple of 32" in msg(L) and quant(L, mode=2, K=16) == 1
    assert needs_device(quant(L, mode=0, K=48)) and needs_device(quant(L, mode=1, K=32, layout=1))


def test_the_gradient_call(L):
    size = nv.rms_norm_vjp_workspace_size
    for K in (16, 48, 4096, 8192, 8208, 32768):
        for rows in (1, 3, 100, 5000):
            n = size(rows, K)
            # at least one part of dw, and no more than one a row and 8 rows of 2 * 148 CTAs
            assert 4 * K <= n <= 4 * K * min(rows + 7, 8 * 296)
            assert vjp(L, rows=rows, K=K, ws_bytes=n - 1) == 1 and "workspace" in msg(L)
            assert needs_device(vjp(L, rows=rows, K=K, ws_bytes=n))
            assert vjp(L, rows=rows, K=K, ws=N0, ws_bytes=n) == 1
            assert needs_device(vjp(L, rows=rows, K=K, dw=N0, ws=N0, ws_bytes=0))
    for bad in ((0, 64), (-1, 64), (3, 0), (3, 24), (3, 32784), (1 << 62, 64)):
        assert size(*bad) == 0
    for bad in ("dy", "h", "rstd", "dx"):
        assert vjp(L, **{bad: N0}) == 1 and "null" in msg(L)
    for bad in ("dy", "dh", "dx", "dw", "ws"):
        assert vjp(L, **{bad: A + 8}) == 1 and "aligned" in msg(L)
    assert needs_device(vjp(L, dh=N0))
    assert vjp(L, rows=0, dy=N0, h=N0, w=N0, rstd=N0, dh=N0, dx=N0, dw=N0, ws=N0, ws_bytes=0) == 0


def test_the_binding_checks_its_tensors(monkeypatch):
    monkeypatch.setattr(nv, "_need_cuda", lambda *ts: None)
    f, b = torch.float32, torch.bfloat16
    x, w = e(4, 64, dtype=b), e(64, dtype=b)
    for call in (lambda **k: nv.rms_norm(**{"x": x, "weight": w, **k}),
                 lambda **k: nv.rms_norm_quantize(**{"x": x, "weight": w, "mode": "mxfp8", **k})):
        with pytest.raises(ValueError, match="weight"):
            call(weight=e(64, dtype=f))
        with pytest.raises(ValueError, match="weight"):
            call(weight=e(32, dtype=b))
        with pytest.raises(ValueError, match="residual"):
            call(residual=e(4, 32, dtype=b))
        with pytest.raises(ValueError, match="residual"):
            call(residual=e(4, 64, dtype=f))
        with pytest.raises(ValueError, match="h is given with"):
            call(h=e(4, 64, dtype=b))
        with pytest.raises(ValueError, match="rstd"):
            call(rstd=e(3, dtype=f))
        with pytest.raises(ValueError, match="float32, float16"):
            call(x=e(4, 64))
    with pytest.raises(ValueError, match="out"):
        nv.rms_norm(x, w, out=e(3, 64, dtype=b))
    with pytest.raises(ValueError, match="mode"):
        nv.rms_norm_quantize(x, w, "fp8")
    with pytest.raises(ValueError, match="codes"):
        nv.rms_norm_quantize(x, w, "mxfp8", codes=e(4, 15, dtype=torch.int32))
    with pytest.raises(ValueError, match="scales"):
        nv.rms_norm_quantize(x, w, "mxfp8", layout="swizzled", scales=e(4, 2))
    with pytest.raises(ValueError, match="global scale|g must"):
        nv.rms_norm_quantize(x, w, "nvfp4", g=e(1, dtype=b))
    r = e(4, dtype=f)
    with pytest.raises(ValueError, match="h must"):
        nv.rms_norm_vjp(x, e(4, 32, dtype=b), w, r)
    with pytest.raises(ValueError, match="dx"):
        nv.rms_norm_vjp(x, x, w, r, dx=e(4, 64, dtype=f))
    with pytest.raises(ValueError, match="dw"):
        nv.rms_norm_vjp(x, x, w, r, dw=e(64, dtype=b))
    with pytest.raises(ValueError, match="rstd"):
        nv.rms_norm_vjp(x, x, w, e(4, dtype=b))


def test_the_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(5, 32, generator=g, dtype=torch.float64) for _ in range(2))
    w, eps = torch.rand(32, generator=g, dtype=torch.float64) + 0.5, 1e-3
    x[2] = 0
    y, r = forward64(x, w, eps)
    dx, dw = vjp64(dy, x, w, r)
    d = 1e-6

    def loss(x, w):
        return float((forward64(x, w, eps)[0] * dy).sum())

    for i, k in ((0, 0), (1, 31), (2, 5), (4, 16)):
        up, down = x.clone(), x.clone()
        up[i, k] += d
        down[i, k] -= d
        # a central difference is off by its third derivative times d^2 / 6 (below 1e5 here) and 2^-52 |loss| / d
        assert abs((loss(up, w) - loss(down, w)) / (2 * d) - float(dx[i, k])) < 1e-6
    for k in (0, 9, 31):
        up, down = w.clone(), w.clone()
        up[k] += d
        down[k] -= d
        assert abs((loss(x, up) - loss(x, down)) / (2 * d) - float(dw[k])) < 1e-6
