"""Plain 64-bit reference of the key/value cache and its attention, and the
tolerance its outputs are held to.

Tolerance of an attention output (derived, not fitted).  With z_j the exact
logits, w_j the exact softmax weights, A = sum_j w_j |v_j| per element and
u(T) = finfo(T).eps / 2 the half step of a rounding to T:
- the result is rounded once to T: u(T) |out|;
- the weights may be rounded to 16 bits before the product with v (fp16: a
  half step of 2^-11 relative, or 2^-25 absolute below its normal range
  relative to the largest weight): 2^-11 A + 2^-25 * sum_j |v_j| w_max;
- a logit is a sum of D products in fp32 (an accumulator may truncate: one
  step of 2^-23 each) times a factor: dz <= (D + 4) 2^-23 * S with
  S = max_j scale * sum_d |q_d k_jd|; exp2's argument z log2(e) and the
  running maximum add 2^-22 * max |z|, exp2 itself 2^-22; an error dz of the
  logits moves the weighted mean by at most 2 dz A;
- the sums over n tokens in fp32 run in at least four chains (one a warp) that
  are joined with their partial results: (n / 4 + 160) 2^-23 A covers the
  chains, the join and the cache's factor g / 2688 rounded to fp32.
lse: dz + 2^-22 |lse| + (n / 4 + 160) 2^-23.
"""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_table():
    t = torch.arange(256, dtype=torch.float64)
    e, m, s = (t // 8) % 16, t % 8, t >= 128
    v = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(torch.tensor(-6.0, dtype=torch.float64)) * m / 8)
    v = torch.where(s, -v, v)
    v[0x7F] = v[0xFF] = float("nan")
    return v


E4M3 = _e4m3_table()


def values(codes, scales, mode, g):
    """float64 values of code words [..., words] and scale bytes [..., blocks]."""
    b = codes.contiguous().view(torch.uint8).long().cpu()
    if mode == "mxfp8":
        v = E4M3[b]
    else:
        t = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64)
        v = torch.stack([t[b & 15], t[b >> 4]], -1).flatten(-2)
    s = scales.long().cpu()
    if mode == "nvfp4":
        f = E4M3[s] * (1.0 if g is None else float(g) / 2688.0)
    else:
        f = torch.exp2(s.double() - 127)
    return v * f.repeat_interleave(16 if mode == "nvfp4" else 32, -1)


def cache_sides(cache):
    return (values(cache.k_codes, cache.k_scales, cache.mode, cache.g_k),
            values(cache.v_codes, cache.v_scales, cache.mode, cache.g_v))


def attention(sides, q, page_table, kv_len, q_start, scale, causal=True, window=0):
    """(out, lse, tol, lse_tol) in float64 for the rows the sequences name;
    rows that no sequence names are NaN.  sides: cache_sides(cache)."""
    K, V = sides
    P, H, R, D = K.shape
    T, Hq, _ = q.shape
    G = Hq // H
    q64 = q.double().cpu()
    u = torch.finfo(q.dtype).eps / 2
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    lse, tol, ltol = torch.full((T, Hq), float("nan"), dtype=torch.float64), out.clone(), None
    ltol = lse.clone()
    page_table, kv_len = page_table.cpu().long(), kv_len.cpu().tolist()
    starts = list(range(len(kv_len) + 1)) if q_start is None else q_start.cpu().tolist()
    for b, L in enumerate(kv_len):
        t0, n = starts[b], starts[b + 1] - starts[b]
        j = torch.arange(L)
        page = page_table[b][j // R] if L else torch.zeros(0, dtype=torch.long)
        k, v = K[page, :, j % R].transpose(0, 1), V[page, :, j % R].transpose(0, 1)  # [H, L, D]
        for i in range(n):
            p = L - n + i
            see = torch.ones(L, dtype=torch.bool)
            if causal:
                see &= j <= p
            if window:
                see &= j > p - window
            kk, vv = k[:, see], v[:, see]
            m = int(see.sum())
            x = q64[t0 + i].view(H, G, D)
            if m == 0:
                out[t0 + i], lse[t0 + i], tol[t0 + i], ltol[t0 + i] = 0.0, -float("inf"), 0.0, 0.0
                continue
            z = torch.einsum("hgd,hjd->hgj", x, kk) * scale
            S = (torch.einsum("hgd,hjd->hgj", x.abs(), kk.abs()) * abs(scale)).amax(-1)
            dz = (D + 4) * 2.0 ** -23 * S + 2.0 ** -22 * z.abs().amax(-1) + 2.0 ** -22
            l = torch.logsumexp(z, -1)
            w = torch.exp(z - l[..., None])
            o = torch.einsum("hgj,hjd->hgd", w, vv)
            A = torch.einsum("hgj,hjd->hgd", w, vv.abs())
            sums = (m / 4 + 160) * 2.0 ** -23
            t = u * o.abs() + (2.0 ** -11 + 2 * dz[..., None] + sums) * A
            t += 2.0 ** -25 * w.amax(-1)[..., None] * vv.abs().sum(1)[:, None]
            t += torch.finfo(q.dtype).smallest_normal * u * 2  # outputs below the normal range
            out[t0 + i], lse[t0 + i] = o.reshape(Hq, D), l.reshape(Hq)
            tol[t0 + i] = t.reshape(Hq, D)
            ltol[t0 + i] = (dz + 2.0 ** -22 * l.abs() + sums).reshape(Hq)
    return out, lse, tol, ltol


def check(got, want, tol, what):
    """Rows the reference leaves NaN are not compared."""
    got = got.double().cpu()
    named = ~torch.isnan(want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    cmp = named & ~inf
    bad = ~((got - want).abs() <= tol) & cmp
    if bad.any():
        at = [tuple(int(c) for c in x) for x in bad.nonzero()[:4]]
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(cmp.sum())} off, e.g. " + ", ".join(
            f"{x}: got {got[x]:.6g} want {want[x]:.6g} tol {tol[x]:.3g}" for x in at))


def seeded(shape, seed, dtype=torch.bfloat16, std=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(device)


def distinct_slots(T, total, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(total, generator=g)[:T].to(torch.int32)

