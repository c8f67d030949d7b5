"""Inputs, the plain 64-bit definitions and the error bounds of the tests of norms, rotation and the
4-bit cache (include/dsa_rope.h, include/dsa_kv4.h).  Everything here runs on the CPU."""


import numpy as np



def dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def ints(a, device="cpu"):
    import torch
    return torch.tensor(list(a), dtype=torch.int32, device=device)


def prefix(a):
    return ints(np.concatenate([[0], np.cumsum(a)]).astype(int))


# ------------------------------------------------------------ norm and rotation

def inv_freq(rot, base=1e4):
    import torch
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))


def turned(x, weight, positions, freq, first=0, adjacent=False, eps=1e-6):
    """(y, magnitude): x [T, H, D] normed and rotated in 64 bits, and for each value the sum of its own and its
    partner's magnitudes before the rotation."""
    import torch
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + float(np.float32(eps))) * weight.double()
    y, size = x.clone(), x.abs()
    half = 0 if freq is None else freq.shape[0]
    for i in range(half):
        a, b = (first + 2 * i, first + 2 * i + 1) if adjacent else (first + i, first + i + half)
        t = positions.double()[:, None] * freq[i]
        y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
        y[..., b] = x[..., b] * t.cos() + x[..., a] * t.sin()
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def turned_bound(y, size, dt):
    """One rounding to the type, u |y| (fp16: at least half a subnormal step, 2^-25), and in fp32 20 * 2^-24 of the pair's
    magnitudes: 13 + 2 roundings of the sum of squares and its mean, halved by the root, 4 of the root, 2 of the
    products, 4 of sine and cosine (their argument's and their own), 2 of the rotation."""
    import torch
    return torch.finfo(dt).eps / 2 * y.abs() * 1.01 + 21 * 2.0 ** -24 * size + (2.0 ** -25 if dt == torch.float16 else 1e-38)


# ------------------------------------------------------------------- quantising

def quantised(x):
    """(codes 1..15, scales) of x [..., D] in 64 bits, exactly."""
    import torch
    g = x.double().unflatten(-1, (-1, 64))
    top = g.abs().amax(dim=-1)
    t = top / torch.full_like(top, 7.0)          # (by a tensor: a number would become a product with 1 / 7)
    m, e = torch.frexp(t)
    scale = torch.ldexp(torch.round(m * 16) / 16, e)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    codes = torch.where(scale[..., None] > 0, torch.round(g / scale[..., None]), torch.zeros_like(g))
    return (codes + 8).flatten(-2).to(torch.uint8), scale


def held(x):
    """The values that 4 bits keep of x."""
    codes, scale = quantised(x)
    return (codes.double() - 8) * scale.repeat_interleave(64, dim=-1)


def block_bytes(dk, dv, ps):
    return ps * (dk + dv) * 17 // 32


def put(pages, page, place, k, v, dk, dv, ps, head=None):
    """Writes one position's k [H, dk] and v [H, dv] (64-bit values) into the pool, byte by byte."""
    import torch
    gk, gv = dk // 64, dv // 64
    for x, code0, scale0, G in ((k, 0, (gk + gv) * ps * 32, gk), (v, gk * ps * 32, (gk + gv) * ps * 32 + gk * ps * 2, gv)):
        codes, scale = quantised(x)
        packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).unflatten(1, (G, 32))
        raw = scale.to(torch.bfloat16).view(torch.uint8).unflatten(1, (G, 2))
        for g in range(G):
            pages[page, :, code0 + (g * ps + place) * 32:code0 + (g * ps + place) * 32 + 32] = packed[:, g]
            pages[page, :, scale0 + (g * ps + place) * 2:scale0 + (g * ps + place) * 2 + 2] = raw[:, g]


def parts(pages, dk, dv, ps):
    """Views of the blocks: codes [n, H, G, ps, 32] of K and V, scales [n, H, G, ps] of K and V."""
    import torch
    gk, gv = dk // 64, dv // 64
    a, b, c = gk * ps * 32, (gk + gv) * ps * 32, (gk + gv) * ps * 32 + gk * ps * 2
    return (pages[..., :a].unflatten(2, (gk, ps, 32)), pages[..., a:b].unflatten(2, (gv, ps, 32)),
            pages[..., b:c].view(torch.bfloat16).unflatten(2, (gk, ps)), pages[..., c:].view(torch.bfloat16).unflatten(2, (gv, ps)))


def values(pages, dk, dv, ps):
    """(K, V) of whole pages in 64 bits: [n, ps, H, D]."""
    import torch
    kc, vc, ks, vs = parts(pages, dk, dv, ps)
    out = []
    for codes, scales in ((kc, ks), (vc, vs)):
        x = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double() - 8
        out.append((x * scales.double()[..., None]).permute(0, 3, 1, 2, 4).flatten(-2))
    return out


# ------------------------------------------------------------------- attention

def make(rows, lens, hq, hkv, dk, dv, ps, dt="bf16", seed=0, row_len=None, extra_rows=0, spare=2, fused=False, amp=1.0):
    """CPU tensors of one problem; the pool's pages hold normals, in an order of their own."""
    import torch
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    n = sum(need) + spare
    pages = torch.empty(n, hkv, block_bytes(dk, dv, ps), dtype=torch.uint8)
    kc, vc, ks, vs = parts(pages, dk, dv, ps)
    for codes, scales in ((kc, ks), (vc, vs)):
        c, s = quantised(torch.randn(*codes.shape[:4], 64, generator=g))
        codes[:] = c[..., 0::2] | (c[..., 1::2] << 4)
        scales[:] = s[..., 0].to(torch.bfloat16)
    order = torch.randperm(n, generator=g).int()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    R = sum(rows) + extra_rows
    if fused:
        q = (amp * torch.randn(R, hq * dk + 64, generator=g)).to(dtype(dt))[:, 32:32 + hq * dk].unflatten(1, (hq, dk))
    else:
        q = (amp * torch.randn(R, hq, dk, generator=g)).to(dtype(dt))
    if row_len is None:
        row_len = [max(0, min(b, b - m + i + 1)) for m, b in zip(rows, lens) for i in range(m)]
    return dict(pages=pages, table=table, q=q, row_offsets=prefix(rows), row_len=ints(list(row_len) + [0] * extra_rows),
                dk=dk, dv=dv, ps=ps)


def reference(t, scale, seen=None):
    """(out, lse, bound of out, bound of lse) in 64 bits.

    A = sum_t w_t |v_t| (w the softmax weights), u = eps / 2 of the operands' type.  A weight (or a weight times a scale) is
    rounded once to the operands' type or to fp16: u A; the output once: u |out|.
    Logits: codes are 1..15 with 8 to be taken off, so the running sums' magnitude is at most 23 / 7 of what
    X = scale sum_g s_g sum_d 7 |q_d| is; 8 roundings of 2^-23 of it (four products of 16 to a group, and the groups'
    sums), and a few 2^-22 of the maximum's subtraction and the exponential: each weight is off by
    e = 2^-20 (1 + 23/7 max_t X) of itself, numerator and denominator both: 2 e A.
    Sums over positions: (n / 16 + 8) roundings of 2^-23 of sum_t w_t 23 s_t.
    Small weights: what is below fp16's range is off by 2^-32 of the row's largest weight, times twice the
    request's largest scale, times 15: 15 * 2^-31 n s / Z (the operands' own fp16, unlifted: as the first kernel's).
    """
    import torch
    dk, dv, ps = t["dk"], t["dv"], t["ps"]
    q = t["q"].double()
    u = torch.finfo(t["q"].dtype).eps / 2
    R, hq, _ = q.shape
    hkv = t["pages"].shape[1]
    G = hq // hkv
    out = torch.zeros(R, hq, dv, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse = torch.full((R, hq), -np.inf, dtype=torch.float64)
    lbound = torch.zeros_like(lse)
    ro, rl = t["row_offsets"].tolist(), t["row_len"].tolist()
    for b in range(len(ro) - 1):
        far = max([rl[r] for r in range(ro[b], ro[b + 1])], default=0)
        if far <= 0:
            continue
        ids = t["table"][b, :-(-far // ps)].long()
        ok = (ids >= 0) & (ids < t["pages"].shape[0])
        pool = t["pages"][ids.clamp(0, t["pages"].shape[0] - 1)]
        k, v = (x.flatten(0, 1)[:far] for x in values(pool, dk, dv, ps))
        _, _, ks, vs = parts(pool, dk, dv, ps)
        ks, vs = (x.double().permute(0, 3, 1, 2).flatten(0, 1)[:far] for x in (ks, vs))       # [far, hkv, G]
        there = ok.repeat_interleave(ps)[:far]
        kk, vv = k.repeat_interleave(G, dim=1), v.repeat_interleave(G, dim=1)
        ksq = ks.repeat_interleave(64, dim=2).repeat_interleave(G, dim=1)
        vsq = vs.repeat_interleave(64, dim=2).repeat_interleave(G, dim=1)
        for r in range(ro[b], ro[b + 1]):
            see = there & (torch.arange(far) < rl[r])
            n = int(see.sum())
            if n == 0:
                continue
            s = (torch.einsum("hd,nhd->hn", q[r], kk) * scale)[:, see]
            X = (torch.einsum("hd,nhd->hn", q[r].abs(), 7 * ksq) * scale)[:, see].amax(dim=1)
            m = s.amax(dim=1, keepdim=True)
            z = torch.exp(s - m).sum(dim=1)
            lse[r] = m[:, 0] + torch.log(z)
            w = torch.exp(s - m) / z[:, None]
            out[r] = torch.einsum("hn,nhd->hd", w, vv[see])
            A = torch.einsum("hn,nhd->hd", w, vv[see].abs())
            S = torch.einsum("hn,nhd->hd", w, vsq[see])
            e = 2.0 ** -20 * (1 + 23 / 7 * X)
            bound[r] = (1.01 * u * (A + out[r].abs()) + 2 * e[:, None] * A + (n / 16 + 8) * 2.0 ** -23 * 23 * S
                        + 15 * 2.0 ** -31 * n * vsq.amax(dim=0) / z[:, None] + 1e-30)
            if u < 2.0 ** -9:
                bound[r] += 2.0 ** -25
            lbound[r] = 2 * e + 2.0 ** -22 * lse[r].abs()
    return out, lse, bound, lbound


def problem(t, scale, device="cuda", **kw):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    q = t["q"]
    if not q.is_contiguous():                       # keep a view's strides
        flat = torch.empty(0, dtype=q.dtype).set_(q.untyped_storage()).to(device)
        q = flat.as_strided(q.shape, q.stride(), q.storage_offset())
    else:
        q = q.to(device)
    cache = dsa.KV4Cache.from_tensors(pages=t["pages"].to(device), table=t["table"].to(device), page_size=t["ps"], D_k=t["dk"],
                                      D_v=t["dv"])
    return dsa.KV4Problem.from_tensors(cache=cache, q=q, row_offsets=t["row_offsets"].to(device),
                                       row_len=t["row_len"].to(device), softmax_scale=scale, **kw)


def run(t, scale, with_lse=True, ws_fill=0x5A, stream=None, **kw):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    prob = problem(t, scale, **kw)
    out = torch.full((prob.R, prob.H_q, t["dv"]), 77.0, dtype=t["q"].dtype, device="cuda")
    lse = torch.full((prob.R, prob.H_q), 77.0, dtype=torch.float32, device="cuda") if with_lse else None
    ws = dsa.alloc_kv4_workspace(prob)
    ws.fill_(ws_fill)
    dsa.dsa_kv4_attn(prob, out, lse, ws, stream=stream)
    bits = dsa.dsa_read_device_status(ws)
    return out.cpu(), None if lse is None else lse.cpu(), bits


def check(t, scale, got, lse, rows=None):
    import torch
    out, l, bound, lb = reference(t, scale)
    rows = slice(0, int(t["row_offsets"][-1])) if rows is None else rows
    err = (got.double() - out).abs()[rows]
    assert torch.isfinite(got.float()[rows]).all()
    worst = (err / bound[rows].clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= bound[rows]).all()), f"output off by {worst:.3g} x its bound"
    if lse is not None:
        a, b = lse.double()[rows], l[rows]
        empty = torch.isinf(b)
        assert torch.equal(torch.isinf(a), empty) and bool((a[empty] < 0).all())
        assert bool(((a - b).abs() <= lb[rows])[~empty].all()), "lse off"
    return worst
