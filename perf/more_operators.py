"""The steps between the block-scaled products and the cache of one decoder layer, as measured cases.

Five operators over NVFP4, MXFP4 and MXFP8 (formats as in perf/operators.py):

- norm: h = x + residual, root-mean-square norm of h, its output plain or quantised for the block-scaled products (and
  dequantised again, which returns the stored codes as the values they stand for);
- norm_grad: that norm's gradient, the quantiser passed straight through;
- append: rotate the queries and keys of new tokens by their positions, quantise keys and values into their slots of the
  paged cache (and read the same slots back);
- tree: attention of drafted tokens that form a tree, over the cached context and each token's own ancestors;
- move: rows of the cache to other slots, as accepted drafts and forked prefixes need it (and read the new slots back).

Cache tensors: codes int32 [pages, kv heads, page size, D / 8] (D / 4 for MXFP8), scales uint8
[pages, kv heads, page size, D / 16] (e4m3, NVFP4) or D / 32 (e8m0); slot = page * page size + row.
"""
import math

import numpy as np
import torch

own = False

F4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def group_of(mode):
    return 16 if mode == "nvfp4" else 32


def row_bytes(case):
    """Code and scale bytes of one row of D (or K) elements."""
    d = case["D"] if "D" in case else case["K"]
    return (d if case["mode"] == "mxfp8" else d // 2) + d // group_of(case["mode"])


def listed():
    def norm(name, mode, dtype, rows, K, residual=True):
        return {"name": name, "op": "norm", "mode": mode, "dtype": dtype, "rows": rows, "K": K, "residual": residual}

    def grad(name, dtype, rows, K, residual=True):
        return {"name": name, "op": "norm_grad", "dtype": dtype, "rows": rows, "K": K, "residual": residual}

    def append(name, mode, dtype, T, Hq, Hkv, D, page, rot, interleaved=False):
        return {"name": name, "op": "append", "mode": mode, "dtype": dtype, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
                "rot": rot, "interleaved": interleaved}

    def tree(name, mode, dtype, B, Hq, Hkv, D, page, kv, n, window=0, lse=False):
        return {"name": name, "op": "tree", "mode": mode, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
                "kv": kv, "n": n, "window": window, "lse": lse}

    def move(name, mode, S, each, Hkv, D, page):
        return {"name": name, "op": "move", "mode": mode, "dtype": "bf16", "S": S, "each": each, "Hkv": Hkv, "D": D, "page": page}

    return [
        # one decoding step's token, for the small-M product that quantises by itself: latency
        norm("norm 1 x 4096 plain", "plain", "bf16", 1, 4096),
        # a prompt in front of the dense product
        norm("norm 4096 x 4096 nvfp4", "nvfp4", "bf16", 4096, 4096),
        # a training batch in front of the eight-bit product
        norm("norm 16384 x 8192 mxfp8", "mxfp8", "bf16", 16384, 8192),
        # training, a micro-batch; the last norm of a model has no stream beside it
        grad("norm gradient 2048 x 4096", "bf16", 2048, 4096, residual=False),
        grad("norm gradient 16384 x 8192", "bf16", 16384, 8192),
        # one decoding step's tokens
        append("append 64 nvfp4", "nvfp4", "bf16", 64, 32, 8, 128, 16, 128),
        # a prompt's tokens; a part of each head turns, in neighbouring pairs
        append("append 16384 mxfp4", "mxfp4", "bf16", 16384, 32, 8, 128, 64, 64, interleaved=True),
        # one chat turn with a few drafts: latency
        tree("tree 1 x 8 over 1000 nvfp4", "nvfp4", "bf16", 1, 32, 8, 128, 64, 1000, 8),
        # a serving batch with wide trees
        tree("tree 16 x 64 over 8192 nvfp4", "nvfp4", "bf16", 16, 32, 8, 128, 16, 8192, 64),
        # small heads, a sliding window, statistics for a later merge; odd pages
        tree("tree 24 x 21 over 5000 mxfp4", "mxfp4", "bf16", 24, 64, 8, 64, 24, 5000, 21, window=1000, lse=True),
        # the accepted drafts of a batch
        move("move 16 x 5 nvfp4", "nvfp4", 16, 5, 8, 128, 64),
        # prefixes that get pages of their own
        move("move 32 x 1000 mxfp8", "mxfp8", 32, 1000, 8, 128, 16),
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm", "norm_grad", "append", "tree", "tree", "move"])
    mode = rng.choice(["nvfp4", "nvfp4", "mxfp4", "mxfp8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_grad"):
        K = 32 * logint(1, 512)
        case = {"op": op, "dtype": dtype, "rows": min(logint(1, 16384), (1 << 27) * 2 // (K * (4 if dtype == "f32" else 2))), "K": K,
                "residual": rng.random() < 0.7}
        return {**case, "mode": rng.choice([mode, "plain"])} if op == "norm" else case
    D = rng.choice([32, 64, 96, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    page = rng.choice([16, 24, 32, 64, 100, 128, 256])
    G = rng.choice([1, 2, 3, 4, 4, 7, 8])
    case = {"op": op, "mode": mode, "Hkv": Hkv, "D": D, "page": page}
    if op == "append":
        top = (1 << 26) * 2 // (4 if dtype == "f32" else 2) // (Hkv * G * D)
        return {**case, "dtype": dtype, "T": min(logint(1, 16384), top), "Hq": Hkv * G, "rot": 16 * rng.randint(1, D // 16),
                "interleaved": rng.random() < 0.5}
    if op == "move":
        S = logint(1, 64)
        return {**case, "dtype": rng.choice(["bf16", "f16"]), "S": S, "each": min(logint(1, 1000), 32000 * 1024 // (S * Hkv * D))}
    n, B = logint(1, 130), logint(1, 32)
    kv = n + logint(1, 65536)
    # no more than the largest listed: its cached elements, its products
    kv = max(n, min(kv, 100_000_000 // (B * Hkv * D), 34_000_000_000 // (B * Hkv * G * n * D)))
    return {**case, "dtype": rng.choice(["bf16", "bf16", "f16"]), "B": B, "Hq": Hkv * G, "kv": kv, "n": n,
            "window": rng.choice([0, 0, 0, logint(1, 4096)]), "lse": rng.random() < 0.4}


def lengths(case):
    """(cached tokens, drafted ones among them) of each sequence: from the longest down to about half, in no order."""
    B = case["B"]
    at = [(b * 7) % B if B % 7 else b for b in range(B)]
    n = [max(1, case["n"] - (a * case["n"]) // (2 * B)) for a in at]
    return [max(m, case["kv"] - (a * case["kv"]) // (2 * B)) for a, m in zip(at, n)], n


# --- the formats, in elementary operations ---------------------------------------------------------------------------


def f32(v, like):
    """A 0-dim tensor: division by a Python number would become a product with its reciprocal."""
    return torch.full((), v, dtype=torch.float32, device=like.device)


def quantise(x, mode, g):
    """(codes as int32 words, scale bytes) of x [..., D] fp32, blocks along D."""
    n = group_of(mode)
    b = x.float().unflatten(-1, (-1, n))
    a = b.abs().amax(-1)
    if mode == "nvfp4":
        e = f32(2688.0, x) / g
        s = ((a / f32(6.0, x)) * e).clamp(max=448.0).to(torch.float8_e4m3fn)
        fs = s.float()
        k = torch.where(fs > 0, e / torch.where(fs > 0, fs, 1.0), 0.0)
        scales = s.view(torch.uint8)
    else:
        m, e = torch.frexp(a / f32(448.0 if mode == "mxfp8" else 6.0, x))
        e = torch.where(m == 0.5, e - 1, e)
        scales = torch.where(a > 0, (e + 127).clamp(0, 254), 0)
        k = torch.exp2((127 - scales).double()).float()
        scales = scales.to(torch.uint8)
    t = b * k.unsqueeze(-1)
    if mode == "mxfp8":
        byte = t.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
        return byte.contiguous().view(torch.int32), scales
    m = t.abs()
    c = (m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    c = (c + torch.signbit(t).byte() * 8).flatten(-2)
    return (c[..., 0::2] + c[..., 1::2] * 16).contiguous().view(torch.int32), scales


def values(codes, scales, mode, g):
    """fp32 values of code words [..., words] with scale bytes [..., blocks]."""
    byte = codes.contiguous().view(torch.uint8)
    if mode == "mxfp8":
        v = byte.view(torch.float8_e4m3fn).float()
    else:
        f = torch.tensor(F4 + [-w for w in F4], device=codes.device)
        pair = torch.stack([f.repeat(16), f.repeat_interleave(16)], -1)  # of each byte: its low and its high code
        v = pair[byte.int()].flatten(-2)
    if mode == "nvfp4":
        s = scales.contiguous().view(torch.float8_e4m3fn).float() * (g / f32(2688.0, codes))
    else:
        s = torch.exp2(scales.float() - 127.0)
    return v.unflatten(-1, (scales.shape[-1], -1)).mul_(s.unsqueeze(-1)).flatten(-2)


# --- inputs ----------------------------------------------------------------------------------------------------------


def normals(shape, seed, spread=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x if spread is None else x.mul_(spread)


def channels(D, seed):
    """Scale of each channel: a few channels are much larger than the rest."""
    s = torch.ones(D, device="cuda")
    s[torch.randperm(D, generator=torch.Generator().manual_seed(seed))[: max(1, D // 32)].cuda()] = 5.0
    return s


def empty_cache(case, pages):
    H, D, P, mode = case["Hkv"], case["D"], case["page"], case["mode"]
    words, blocks = D // (4 if mode == "mxfp8" else 8), D // group_of(mode)
    st = {}
    for side in "kv":
        st[side + "_codes"] = torch.zeros(pages, H, P, words, dtype=torch.int32, device="cuda")
        st[side + "_scales"] = torch.zeros(pages, H, P, blocks, dtype=torch.uint8, device="cuda")
        # the calibrated amax that a program keeps for each side
        st["g_" + side] = torch.full((1,), 24.0 if side == "k" else 5.0, device="cuda") if mode == "nvfp4" else None
    return st


def fill(st, case, seed):
    """Quantised normal keys and values in every slot, a share of the pages at a time."""
    pages, H, P, _ = st["k_codes"].shape
    D = case["D"]
    at = max(1, (1 << 26) // (H * P * D))
    for side in "kv":
        spread = channels(D, seed) if side == "k" else None
        for i, p in enumerate(range(0, pages, at)):
            n = min(at, pages - p)
            x = normals((n, H, P, D), seed * 1000 + 2 * i + (side == "v"), spread).bfloat16()
            c, s = quantise(x, case["mode"], st["g_" + side])
            st[side + "_codes"][p:p + n], st[side + "_scales"][p:p + n] = c, s


def drafts(n, rng):
    """Bits of a tree's ancestors, the node itself included: node 0 is the root, the others hang on one of the last few."""
    rows = []
    for i in range(n):
        rows.append((1 << i) | (rows[rng.randint(max(0, i - 6), i)] if i else 0))
    return rows


def prepare(case, seed):
    order = torch.Generator().manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, K, dtype = case["rows"], case["K"], DT[case["dtype"]]
        spread = channels(K, seed)
        st = {"case": case, "w": (1.0 + 0.1 * normals((K,), seed + 1)).to(dtype)}
        if op == "norm":
            st.update(x=normals((rows, K), seed + 2).to(dtype), residual=normals((rows, K), seed + 3, spread).to(dtype) if case["residual"] else None,
                      # the calibrated amax of the norm's output
                      g=torch.full((1,), 12.0, device="cuda") if case["mode"] == "nvfp4" else None)
        else:
            h = normals((rows, K), seed + 2, spread).to(dtype)
            st.update(h=h, dy=normals((rows, K), seed + 3, 0.01).to(dtype), dh=normals((rows, K), seed + 4, 0.01).to(dtype) if case["residual"] else None,
                      rstd=(h.double().square().mean(-1) + EPS).rsqrt().float())
        return st
    P, H, D = case["page"], case["Hkv"], case["D"]
    if op == "append":
        T, Hq = case["T"], case["Hq"]
        pages = -(-T * 5 // (4 * P)) + 1
        st = empty_cache(case, pages)
        # the tokens of sequences whose pages lie anywhere: whole pages in a shuffled order
        perm = torch.randperm(pages, generator=order)
        slots = (perm[:, None] * P + torch.arange(P)).flatten()[:T]
        # queries, keys and values are parts of one projection's rows
        qkv = normals((T, Hq + 2 * H, D), seed).to(DT[case["dtype"]])
        qkv[:, Hq:Hq + H] *= channels(D, seed).to(qkv.dtype)
        # the table that a program keeps for all positions
        most = max(4096, T)
        angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * torch.exp2(
            torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") * (-2.0 * math.log2(10000.0) / case["rot"]))
        positions = torch.randint(0, most, (T,), generator=order) if T <= 256 else torch.arange(T)
        st.update(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:], cos=angle.cos().float(), sin=angle.sin().float(),
                  positions=positions.to(torch.int32).cuda(), slots=slots.to(torch.int32).cuda())
        return st
    if op == "move":
        S, each = case["S"], case["each"]
        rows = S * each
        pages = -(-2 * rows // P) + 1
        st = empty_cache(case, pages)
        fill(st, case, seed)
        perm = torch.randperm(2 * rows, generator=order) if each < 64 else torch.arange(2 * rows)
        st.update(case=case, src=perm[:rows].to(torch.int32).cuda(), dst=perm[rows:].to(torch.int32).cuda(),
                  # a few drafts of each sequence, one after the other; of a copied prefix every row for itself
                  starts=(torch.arange(S + 1) * each).to(torch.int32).cuda() if each < 64 else None)
        return st
    kv, n = lengths(case)
    need = [-(-m // P) for m in kv]
    st = empty_cache(case, sum(need) + 1)
    fill(st, case, seed)
    perm = torch.randperm(sum(need) + 1, generator=order).to(torch.int32)
    table = torch.zeros(case["B"], max(need), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    rng = np.random.RandomState(seed % (1 << 31))
    words = -(-max(n) // 32)
    bits = [row for m in n for row in drafts(m, rng)]
    mask = np.array([[(row >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for row in bits], dtype=np.uint32)
    starts = np.concatenate([[0], np.cumsum(n)])
    st.update(case=case, page_table=table.cuda(), kv_len=torch.tensor(kv, dtype=torch.int32).cuda(),
              q_start=torch.tensor(starts, dtype=torch.int32).cuda(), max_q=max(n), max_kv=max(kv),
              tree_mask=torch.from_numpy(mask.view(np.int32)).cuda(),
              q=normals((int(starts[-1]), case["Hq"], D), seed + 7).to(DT[case["dtype"]]))
    return st


# --- the operators ---------------------------------------------------------------------------------------------------


def norm_plain(st):
    c = st["case"]
    h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(st["x"].dtype)
    # in 64 bits: a step of the factor moves values across the borders of the codes
    r = (h.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float()
    y = h.float() * r * st["w"].float()
    if c["mode"] != "plain":
        y = values(*quantise(y, c["mode"], st["g"]), c["mode"], st["g"])
    out = (y.to(h.dtype), r[:, 0])
    return out if st["residual"] is None else out + (h,)


def norm_grad_plain(st):
    h, r = st["h"].float(), st["rstd"][:, None]
    dy = st["dy"].float()
    wdy = dy * st["w"].float()
    dx = r * (wdy - h * ((wdy * h).mean(-1, keepdim=True) * (r * r)))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return dx.to(st["h"].dtype), (dy * (h * r)).sum(0)


def rotate_plain(x, cos, sin, rot, interleaved):
    """x [T, heads, D] fp32 by the angles of its tokens, cos and sin [T, rot / 2]."""
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def rows_of(st, slots):
    """The values of slots, both sides."""
    c = st["case"]
    page, row = slots.long() // c["page"], slots.long() % c["page"]
    return tuple(values(st[s + "_codes"][page, :, row], st[s + "_scales"][page, :, row], c["mode"], st["g_" + s]).to(DT[c["dtype"]]) for s in "kv")


def append_plain(st):
    c = st["case"]
    page, row = st["slots"].long() // c["page"], st["slots"].long() % c["page"]
    cos, sin = st["cos"][st["positions"].long()], st["sin"][st["positions"].long()]
    for s, x in (("k", rotate_plain(st["k"].float(), cos, sin, c["rot"], c["interleaved"])), ("v", st["v"])):
        st[s + "_codes"][page, :, row], st[s + "_scales"][page, :, row] = quantise(x, c["mode"], st["g_" + s])
    return (rotate_plain(st["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(st["q"].dtype),) + rows_of(st, st["slots"])


def move_plain(st):
    P = st["case"]["page"]
    src, dst = st["src"].long(), st["dst"].long()
    for t in (st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"]):
        t[dst // P, :, dst % P] = t[src // P, :, src % P]
    return rows_of(st, st["dst"])


def tree_plain(st):
    c = st["case"]
    B, Hkv, D, P, mode = c["B"], c["Hkv"], c["D"], c["page"], c["mode"]
    G, Q, N = c["Hq"] // Hkv, st["max_q"], st["page_table"].shape[1] * P

    def side(s):
        at = st["page_table"].flatten().int()
        codes = st[s + "_codes"].index_select(0, at).unflatten(0, (B, -1)).transpose(1, 2).reshape(B, Hkv, N, -1)
        scales = st[s + "_scales"].index_select(0, at).unflatten(0, (B, -1)).transpose(1, 2).reshape(B, Hkv, N, -1)
        return values(codes, scales, mode, st["g_" + s])

    n_q = (st["q_start"][1:] - st["q_start"][:-1])[:, None].long()
    i = torch.arange(Q, device="cuda")[None]
    rows = (st["q_start"][:-1, None].long() + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    logits = (q @ side("k").transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).unflatten(2, (G, Q))
    bits = ((st["tree_mask"].unsqueeze(-1) >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).flatten(1)[rows].bool()  # [B, Q, 32 words]
    j = torch.arange(N, device="cuda")
    n_kv = st["kv_len"][:, None, None].long()
    at = j - (n_kv - n_q[..., None])  # [B, 1, N]: the token's place among the drafts; negative: context
    ancestor = bits.gather(2, at.clamp(0, bits.shape[2] - 1).expand(B, Q, N))
    seen = torch.where(at < 0, torch.ones_like(ancestor), ancestor) & (j < n_kv)
    if c["window"]:  # a draft's position is the context's length plus its depth
        depth = (bits.sum(-1, keepdim=True) - 1).clamp(min=0)
        seen = seen & ((at >= 0) | (at > depth - c["window"]))
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ side("v")).unflatten(2, (G, Q)) / torch.where(total > 0, total, 1.0)
    used = i < n_q
    out = out.permute(0, 3, 1, 2, 4).reshape(B, Q, Hkv * G, D)[used].to(st["q"].dtype)
    if not c["lse"]:
        return out
    return out, (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, Q, Hkv * G)[used]


def run_own(st):
    from mxfp8_block_scaled_nvfp4_b200 import nvfp4 as nv
    c = st["case"]
    dtype = DT[c["dtype"]]
    if c["op"] == "norm":
        if c["mode"] == "plain":
            y, h, r = nv.rms_norm(st["x"], st["w"], EPS, st["residual"], return_rstd=True)
        else:
            codes, scales, h, r = nv.rms_norm_quantize(st["x"], st["w"], c["mode"], st["g"], EPS, st["residual"], "swizzled", return_rstd=True)
            if c["mode"] == "nvfp4":
                y = nv.nvfp4_dequantize(codes, scales, st["g"], "swizzled", dtype)
            else:
                y = (nv.mxfp8_dequantize if c["mode"] == "mxfp8" else nv.mxfp4_dequantize)(codes, scales, "swizzled", dtype)
        return (y, r) if st["residual"] is None else (y, r, h)
    if c["op"] == "norm_grad":
        return nv.rms_norm_vjp(st["dy"], st["h"], st["w"], st["rstd"], st["dh"])
    cache = st.get("cache")
    if cache is None:  # the handle that a program makes once, beside its cache tensors
        cache = st["cache"] = nv.KvCache(c["mode"], st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["g_k"], st["g_v"])
    if c["op"] == "append":
        q = nv.kv_cache_append(cache, st["q"], st["k"], st["v"], st["cos"], st["sin"], st["positions"], st["slots"], interleaved=c["interleaved"])
        return (q,) + tuple(nv.kv_cache_read(cache, st["slots"], dtype))
    if c["op"] == "move":
        nv.kv_cache_move(cache, st["src"], st["dst"], st["starts"])
        return tuple(nv.kv_cache_read(cache, st["dst"], dtype))
    return nv.kv_attention_tree(cache, st["q"], st["page_table"], st["kv_len"], st["tree_mask"], st["q_start"], max_q=st["max_q"],
                                max_kv=st["max_kv"], window=c["window"], return_lse=c["lse"])


def run(state):
    if own:
        return run_own(state)
    return {"norm": norm_plain, "norm_grad": norm_grad_plain, "append": append_plain, "move": move_plain, "tree": tree_plain}[state["case"]["op"]](state)


def pairs(case):
    """Visible (query, token) pairs of one query head, about (a draft sees half of the drafts at most), and cached tokens read."""
    seen = read = 0
    for m, n in zip(*lengths(case)):
        context = min(m - n, case["window"]) if case["window"] else m - n
        seen, read = seen + n * context + n, read + context + n
    return seen, read


def work(case):
    b16 = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n, K = case["rows"], case["K"]
        # written: the sum (where there is a residual), the output, the factor; a quantised output is read back as values
        out = K * b16 if case["mode"] == "plain" else 2 * row_bytes(case) + K * b16
        return {"bytes": n * ((3 if case["residual"] else 1) * K * b16 + out + 4) + K * b16, "flops": 8 * n * K}
    if case["op"] == "norm_grad":
        n, K = case["rows"], case["K"]
        return {"bytes": n * ((4 if case["residual"] else 3) * K * b16 + 4) + K * (b16 + 4), "flops": 12 * n * K}
    H, D = case["Hkv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        # queries turned; keys and values read, written and read back; the angles of each position once
        return {"bytes": T * (2 * case["Hq"] * D * b16 + 2 * H * (2 * row_bytes(case) + 2 * D * b16) + 4 * case["rot"] + 8), "flops": T * (3 * case["Hq"] + 7 * H) * D}
    if case["op"] == "move":
        rows = 2 * case["S"] * case["each"] * H
        return {"bytes": rows * (3 * row_bytes(case) + D * b16), "flops": rows * D}
    seen, read = pairs(case)
    rows = sum(lengths(case)[1])
    return {"bytes": 2 * read * H * row_bytes(case) + rows * (case["Hq"] * (4 * D + (4 if case["lse"] else 0)) + 4 * -(-case["n"] // 32)),
            "flops": 4 * seen * case["Hq"] * D}


# --- the same from the definitions, in 64 bits -----------------------------------------------------------------------


def decode64(codes, scales, mode, g):
    """Values in float64 of numpy code words and scale bytes, element by element from the formats' definitions."""
    def tiny(c, bits, bias):  # sign, exponent, `bits` of mantissa
        e, m = (c >> bits) & (7 if bits == 1 else 15), c & ((1 << bits) - 1)
        if bits == 1:
            e = (c >> 1) & 3
        v = np.where(e > 0, np.ldexp(1.0 + m / (1 << bits), (e - bias).astype(np.int32)), np.ldexp(m / (1 << bits), 1 - bias))
        return np.where((c >> (3 if bits == 1 else 7)) & 1, -v, v)

    b = codes.view(np.uint8)
    if mode == "mxfp8":
        v = tiny(np.arange(256), 3, 7)[b]
    else:
        t = tiny(np.arange(16), 1, 1)
        v = np.empty(b.shape[:-1] + (2 * b.shape[-1],))
        v[..., 0::2], v[..., 1::2] = t[b & 15], t[b >> 4]
    s = tiny(np.arange(256), 3, 7)[scales] * float(g) / 2688.0 if mode == "nvfp4" else np.ldexp(1.0, scales.astype(np.int32) - 127)
    return v * np.repeat(s, group_of(mode), -1)


def encode64(x, mode, g):
    """Values in float64 that the formats hold for x [..., D] (fp32 numbers). The scale and the quotient are defined in 32
    bits, in this order; the rounding to the grid is exact."""
    def at_step(t, low, bits):
        return torch.exp2(((torch.frexp(t)[1] - 1).clamp(min=low) - bits).double())

    b = x.float().reshape(x.shape[:-1] + (-1, group_of(mode)))
    a = b.abs().amax(-1)
    if mode == "nvfp4":
        e = torch.tensor(np.float32(2688.0) / np.float32(g), device=x.device)
        t = ((a / torch.full_like(a, 6.0)) * e).clamp(max=448.0).double()
        step = at_step(t, -6, 3)
        s = torch.round(t / step) * step
        k = torch.where(s > 0, e / torch.where(s > 0, s, 1.0).float(), torch.zeros_like(a))
        unit = s * float(g) / 2688.0
    else:
        t = (a / torch.full_like(a, 448.0 if mode == "mxfp8" else 6.0)).double()
        m, up = torch.frexp(t)
        up = torch.where(t > 0, torch.where(m == 0.5, up - 1, up), -127).clamp(min=-127).double()
        unit, k = torch.exp2(up), torch.exp2(-up).float()
    y = (b * k[..., None]).double()
    low, top, bits = (-6, 448.0, 3) if mode == "mxfp8" else (0, 6.0, 1)
    step = at_step(y.abs(), low, bits)
    return ((torch.round(y / step) * step).clamp(-top, top) * unit[..., None]).reshape(x.shape)


def turn64(x, cos, sin, rot, interleaved):
    """x [T, heads, D] float64; each product and each sum a 32-bit number."""
    first = torch.arange(0, rot, 2, device=x.device) if interleaved else torch.arange(rot // 2, device=x.device)
    second = first + (1 if interleaved else rot // 2)
    c, s = cos.double()[:, None], sin.double()[:, None]
    r = lambda v: v.float().double()  # noqa: E731
    out = x.clone()
    out[..., first] = r(r(x[..., first] * c) - r(x[..., second] * s))
    out[..., second] = r(r(x[..., second] * c) + r(x[..., first] * s))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        if case["rows"] * case["K"] > 1 << 27:
            return None
        h = st["x"] if st["residual"] is None else (st["x"].double() + st["residual"].double()).to(st["x"].dtype)
        r64 = 1.0 / torch.sqrt((h.double() ** 2).sum(-1) / case["K"] + EPS)
        if case["mode"] == "plain":
            y = h.double() * r64[:, None] * st["w"].double()
        else:  # what is quantised is a 32-bit number: the factor, its product with h, and that with w, each rounded
            y = (h.double() * r64.float().double()[:, None]).float().double() * st["w"].double()
            y = encode64(y.float(), case["mode"], 1.0 if st["g"] is None else float(st["g"]))
        full = h.double() if st["residual"] is None else st["x"].double() + st["residual"].double()
        return (y, r64) if st["residual"] is None else (y, r64, full)
    if op == "norm_grad":
        if case["rows"] * case["K"] > 1 << 27:
            return None
        h, dy, w, r = st["h"].double(), st["dy"].double(), st["w"].double(), st["rstd"].double()[:, None]
        dx = r * dy * w - h * r ** 3 * (dy * w * h).sum(-1, keepdim=True) / case["K"]
        return dx if st["dh"] is None else dx + st["dh"].double(), (dy * h * r).sum(0)
    g = {s: 1.0 if st["g_" + s] is None else float(st["g_" + s]) for s in "kv"}
    mode, P = case["mode"], case["page"]
    if op == "append":
        cos, sin = st["cos"][st["positions"].long()], st["sin"][st["positions"].long()]
        q, k = (turn64(st[n].double(), cos, sin, case["rot"], case["interleaved"]) for n in "qk")
        return q, encode64(k, mode, g["k"]), encode64(st["v"].double(), mode, g["v"])
    host = {n: v.cpu().numpy() for n, v in st.items() if isinstance(v, torch.Tensor) and v.dtype != torch.bfloat16}
    if op == "move":
        at = host["src"] // P, host["src"] % P
        return tuple(decode64(np.ascontiguousarray(host[s + "_codes"][at[0], :, at[1]]), host[s + "_scales"][at[0], :, at[1]], mode, g[s]) for s in "kv")
    kv, n = lengths(case)
    Hkv, G, D = case["Hkv"], case["Hq"] // case["Hkv"], case["D"]
    out = torch.zeros(sum(n), case["Hq"], D, dtype=torch.float64)
    lse = torch.full((sum(n), case["Hq"]), -math.inf, dtype=torch.float64)
    at = 0
    for b, (L, m) in enumerate(zip(kv, n)):
        pages = host["page_table"][b, : -(-L // P)]
        words = host["tree_mask"][at:at + m].view(np.uint32)
        drafted = np.array([[(int(row[d // 32]) >> (d % 32)) & 1 for d in range(m)] for row in words], dtype=bool)
        ok = torch.ones(m, L, dtype=torch.bool)
        ok[:, L - m:] = torch.from_numpy(drafted)
        if case["window"]:
            position = torch.from_numpy(L - m + np.maximum(drafted.sum(1) - 1, 0))
            ok[:, :L - m] &= torch.arange(L - m)[None] > position[:, None] - case["window"]
        ok = ok.cuda()
        for h in range(Hkv):
            K, V = (torch.from_numpy(decode64(host[s + "_codes"][pages, h].reshape(len(pages) * P, -1)[:L],
                                              host[s + "_scales"][pages, h].reshape(len(pages) * P, -1)[:L], mode, g[s])).cuda() for s in "kv")
            for r in range(h * G, h * G + G):
                z = (st["q"][at:at + m, r].double() @ K.T) / math.sqrt(D)
                z = torch.where(ok, z, -math.inf)
                l = torch.logsumexp(z, -1)
                p = torch.where(ok, torch.exp(z - torch.where(l > -math.inf, l, 0.0)[:, None]), 0.0)
                out[at:at + m, r] = (p @ V).cpu()
                lse[at:at + m, r] = l.cpu()
        at += m
    return (out, lse) if case["lse"] else out
