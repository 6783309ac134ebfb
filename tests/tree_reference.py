"""64-bit reference of kv_attention_tree; rows, tolerances and cache values as
in kv_reference (its derivation holds for any set of tokens that a query
sees)."""
import random

import torch


def ancestors(n, seed, near=6, blank=0.0):
    """Masks (Python ints) of a random tree: node 0 is the root, each other one
    hangs on one of the `near` before it.  blank: the share of rows with no bit."""
    rng = random.Random(seed)
    rows = []
    for i in range(n):
        rows.append((1 << i) | (rows[rng.randint(max(0, i - near), i - 1)] if i else 0))
    return [0 if rng.random() < blank else r for r in rows]


def pack(masks, words, junk=0):
    """int32 [T, words] of Python ints; junk: bits to set from bit 32 * words - 1 down (beyond a sequence's drafts)."""
    t = torch.tensor([[(m | junk) >> (32 * w) & 0xFFFFFFFF for w in range(words)] for m in masks], dtype=torch.int64)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32).reshape(len(masks), words)


def attention_tree(sides, q, page_table, kv_len, q_start, masks, scale, window=0):
    """(out, lse, tol, lse_tol) in float64; rows that no sequence names are NaN."""
    K, V = sides
    P, H, R, D = K.shape
    T, Hq, _ = q.shape
    G = Hq // H
    q64 = q.double().cpu()
    u = torch.finfo(q.dtype).eps / 2
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64)
    tol, ltol = out.clone(), lse.clone()
    for b, L in enumerate(kv_len):
        t0, n = q_start[b], q_start[b + 1] - q_start[b]
        j = torch.arange(L)
        page = page_table[b].cpu().long()[j // R] if L else torch.zeros(0, dtype=torch.long)
        k, v = K[page, :, j % R].transpose(0, 1), V[page, :, j % R].transpose(0, 1)
        for i in range(n):
            bits = [d for d in range(n) if masks[t0 + i] >> d & 1]
            see = j < L - n
            if window:
                see &= j > L - n + max(len(bits) - 1, 0) - window
            for d in bits:
                if L - n + d >= 0:
                    see[L - n + d] = True
            kk, vv, m = k[:, see], v[:, see], int(see.sum())
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
            a = torch.einsum("hgj,hjd->hgd", w, vv.abs())
            sums = (m / 4 + 160) * 2.0 ** -23
            t = u * o.abs() + (2.0 ** -11 + 2 * dz[..., None] + sums) * a
            t += 2.0 ** -25 * w.amax(-1)[..., None] * vv.abs().sum(1)[:, None]
            t += torch.finfo(q.dtype).smallest_normal * u * 2
            out[t0 + i], lse[t0 + i] = o.reshape(Hq, D), l.reshape(Hq)
            tol[t0 + i] = t.reshape(Hq, D)
            ltol[t0 + i] = (dz + 2.0 ** -22 * l.abs() + sums).reshape(Hq)
    return out, lse, tol, ltol
