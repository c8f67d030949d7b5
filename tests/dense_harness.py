"""Inputs, the plain 64-bit definition and the error bounds of the dense
attention tests (include/dsa_dense.h)."""
import numpy as np


def make(rows, lens, hq, hkv, dk, dv, dtype="bf16", seed=0, fused=False, row_len=None, extra_rows=0):
    """CPU tensors of one problem.  row_len: None (causal), or a list."""
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    R, L = sum(rows) + extra_rows, sum(lens)

    def rnd(*shape):
        return torch.randn(*shape, generator=g).to(dt)

    if fused:
        x = rnd(R, hq * dk)[:, None].reshape(R, hq * dk)
        pad = rnd(R, 8 * hq * dk // 4 + 64)
        q = torch.cat([pad[:, :64], x, pad[:, 64:128]], dim=1)[:, 64:64 + hq * dk].unflatten(1, (hq, dk))
        y = rnd(L, hkv * (dk + dv) + 40)
        k = y[:, 24:24 + hkv * dk].unflatten(1, (hkv, dk))
        v = y[:, 24 + hkv * dk:24 + hkv * (dk + dv)].unflatten(1, (hkv, dv))
    else:
        q, k, v = rnd(R, hq, dk), rnd(L, hkv, dk), rnd(L, hkv, dv)
    if row_len is None:
        row_len = [max(0, min(b, b - n + i + 1)) for n, b in zip(rows, lens) for i in range(n)]
    pre = lambda a: torch.tensor(np.concatenate([[0], np.cumsum(a)]).astype(np.int32))
    return dict(q=q, k=k, v=v, row_len=torch.tensor(list(row_len) + [0] * extra_rows, dtype=torch.int32),
                offsets=pre(lens), row_offsets=pre(rows))


def reference(t, scale):
    """(out, lse, bound) in float64; bound: how far each value of the kernel's
    output may be from it.

    A = sum_t w_t |v_t| (w the softmax weights).  The weights are rounded to the
    operands' type (at most u = eps / 2 of each: u A), the output once more
    (u |out|).  fp32: a logit is a sum of D_k products in at most D_k / 16 + 4
    roundings of at most 2^-23 of the running magnitude, at most 2^-18 of
    X = scale sum_d |q_d k_d| for the widths here, and the scaling, the
    subtraction of the maximum and the exponential cost a few 2^-22 more; so
    each weight is off by at most e = 2^-18 (1 + max_t X) of itself, numerator
    and denominator both: 2 e A.  fp16 alone: weights below 2^-14 of the largest
    are rounded to multiples of 2^-24, 2^-25 |v_t| / Z each, Z = sum exp(s - max).
    """
    import torch
    q, k, v = (t[x].double() for x in "qkv")
    dt = t["q"].dtype
    u = torch.finfo(dt).eps / 2
    R, hq, dk = q.shape
    G = hq // k.shape[1]
    out = torch.zeros(R, hq, v.shape[2], dtype=torch.float64)
    lse = torch.full((R, hq), -np.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lbound = torch.zeros_like(lse)
    ro, of, rl = t["row_offsets"].tolist(), t["offsets"].tolist(), t["row_len"].tolist()
    for b in range(len(of) - 1):
        for r in range(ro[b], ro[b + 1]):
            n = min(max(rl[r], 0), of[b + 1] - of[b])
            if n == 0:
                continue
            kk = k[of[b]:of[b] + n].repeat_interleave(G, dim=1)       # [n, hq, dk]
            vv = v[of[b]:of[b] + n].repeat_interleave(G, dim=1)
            s = torch.einsum("hd,nhd->hn", q[r], kk) * scale
            X = (torch.einsum("hd,nhd->hn", q[r].abs(), kk.abs()) * scale).amax(dim=1)
            m = s.amax(dim=1, keepdim=True)
            z = torch.exp(s - m).sum(dim=1)
            lse[r] = m[:, 0] + torch.log(z)
            w = torch.exp(s - m) / z[:, None]
            out[r] = torch.einsum("hn,nhd->hd", w, vv)
            A = torch.einsum("hn,nhd->hd", w, vv.abs())
            e = 2.0 ** -18 * (1 + X)
            bound[r] = 1.01 * u * (A + out[r].abs()) + 2 * e[:, None] * A + 1e-30
            if dt == torch.float16:
                bound[r] += 2.0 ** -25 * vv.abs().sum(dim=0) / z[:, None] + 2.0 ** -25
            lbound[r] = 2 * e + 2.0 ** -22 * lse[r].abs()
    return out, lse, bound, lbound


def problem(t, scale, rows_max=None, device="cuda"):
    import dsa_sparse_attention_03_gb300 as dsa
    d = {}
    for name, x in t.items():
        if x.dim() == 3 and not x.is_contiguous():      # keep a view's strides
            wide = x.untyped_storage()
            import torch
            flat = torch.empty(0, dtype=x.dtype).set_(wide).to(device)
            d[name] = flat.as_strided(x.shape, x.stride(), x.storage_offset())
        else:
            d[name] = x.to(device)
    prob = dsa.DenseProblem.from_tensors(softmax_scale=scale, **d)
    if rows_max is not None:
        prob.set(rows_max=rows_max)
    return prob, d


def run(t, scale, rows_max=None, with_lse=True, ws_fill=0x5A, stream=None):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    prob, d = problem(t, scale, rows_max)
    out = torch.full((prob.R, prob.H_q, prob.D_v), 77.0, dtype=t["q"].dtype, device="cuda")
    lse = torch.full((prob.R, prob.H_q), 77.0, dtype=torch.float32, device="cuda") if with_lse else None
    ws = dsa.alloc_dense_workspace(prob)
    ws.fill_(ws_fill)
    dsa.dsa_dense_attn(prob, out, lse, ws, stream=stream)
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
