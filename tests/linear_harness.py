"""Inputs, the plain 64-bit recurrence and the error bounds of the linear
attention tests (include/dsa_linear.h)."""
import numpy as np

C = 128   # tokens of a chunk


def make(rows, H, dk, dv, dtype="bf16", seed=0, state=True, fused=False, amp=1.0, decay=None, extra_rows=0,
         n_states=None):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    R = sum(rows) + extra_rows

    def rnd(*shape):
        return (torch.randn(*shape, generator=g) * amp).to(dt)

    if fused:
        x = rnd(R, H * (2 * dk + dv) + 24)
        q, k = x[:, 8:8 + H * dk].unflatten(1, (H, dk)), x[:, 8 + H * dk:8 + 2 * H * dk].unflatten(1, (H, dk))
        v = x[:, 8 + 2 * H * dk:8 + H * (2 * dk + dv)].unflatten(1, (H, dv))
    else:
        q, k, v = rnd(R, H, dk), rnd(R, H, dk), rnd(R, H, dv)
    if decay is None:
        ld = torch.log1p(-torch.exp2(-torch.linspace(1.0, 11.0, H).double())).float()
    else:
        ld = torch.full((H,), decay, dtype=torch.float32)
    pre = torch.tensor(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
    n = len(rows) if n_states is None else n_states
    s0 = torch.randn(n, H, dk, dv, generator=g) * amp * amp if state else None
    return dict(q=q, k=k, v=v, log_decay=ld, row_offsets=pre), s0


def reference(t, s0, scale, places=None):
    """Per request in float64: [(out, out_bound, state, state_bound)].

    u = eps / 2 of the operands' type.  Each weight P_ij = scale l^(i-j) q_i.k_j
    of a token's own chunk is rounded once (u of it), and so is each value of the
    state H at the chunk's start where the queries read it; the output once more.
    fp32: S is a sum of D_k products (at most 2^-18 of the sum of their
    magnitudes, as in dense_harness), the decays cost a few 2^-22 relative.
    fp16 rounds values below 2^-14 of their row's (column's) largest to multiples
    of 2^-24 of it at worst: 2^-24 of the row's largest P for each |v_j|, 2^-24 of
    the column's largest H for each |q|.

    State, fp32: the decayed values enter with at least 22 bits, the products
    of a chunk are added in at most 24 roundings, then one multiply-add per
    chunk; every power of the decay costs 2^-22 and the rounding of its exponent
    (x 2^-x <= 0.54, in 2^-23): at most (48 + 4 chunks) 2^-23 of the sum of
    magnitudes A.
    """
    import torch
    dt = t["q"].dtype
    u = torch.finfo(dt).eps / 2
    half = dt == torch.float16
    lam = torch.exp(t["log_decay"].double().clamp(max=0.0))
    H = lam.shape[0]
    ro = t["row_offsets"].tolist()
    res = []
    for b in range(len(ro) - 1):
        q, k, v = (t[x][ro[b]:ro[b + 1]].double() for x in "qkv")
        n, dk, dv = q.shape[0], q.shape[2], v.shape[2]
        at = b if places is None else places[b]
        S = s0[at].double().clone() if s0 is not None and at >= 0 else torch.zeros(H, dk, dv, dtype=torch.float64)
        A = S.abs()
        out, bound = torch.zeros(n, H, dv, dtype=torch.float64), torch.zeros(n, H, dv, dtype=torch.float64)
        for i in range(n):
            if i % C == 0:
                S0, A0 = S.clone(), A.clone()
            S = lam[:, None, None] * S + k[i][:, :, None] * v[i][:, None, :]
            A = lam[:, None, None] * A + (k[i].abs()[:, :, None] * v[i].abs()[:, None, :])
            out[i] = scale * torch.einsum("hd,hde->he", q[i], S)
        for c in range(0, n, C):
            m = min(C, n - c)
            w = torch.arange(m)[:, None] - torch.arange(m)[None]
            D = torch.where(w >= 0, lam[:, None, None] ** w.clamp(min=0), torch.zeros((), dtype=torch.float64))
            x = slice(c, c + m)
            s = torch.einsum("ihd,jhd->hij", q[x], k[x])
            sa = torch.einsum("ihd,jhd->hij", q[x].abs(), k[x].abs())
            va = v[x].abs()
            bound[x] += abs(scale) * torch.einsum("hij,jhe->ihe", D * (1.01 * u * s.abs() + 2.0 ** -17 * sa), va)
            if c == 0:
                Hs, Ha = (s0[at].double() if s0 is not None and at >= 0 else torch.zeros(H, dk, dv, dtype=torch.float64)), None
            else:
                Hs = states[c]
            reach = lam[None, :] ** (torch.arange(m)[:, None] + 1)
            bound[x] += abs(scale) * 1.01 * (u + 2.0 ** -15) * reach[..., None] * torch.einsum("ihd,hde->ihe", q[x].abs(), Hs.abs())
            if half:
                low = torch.where(w[None] >= 0, s.abs(), torch.zeros_like(s)).amax(dim=2)          # [h, i]
                bound[x] += abs(scale) * 2.0 ** -24 * torch.einsum("hi,hij,jhe->ihe", low, (D > 0).double(), va)
                bound[x] += abs(scale) * 2.0 ** -24 * reach[..., None] * torch.einsum(
                    "ihd,he->ihe", q[x].abs(), Hs.abs().amax(dim=1))
            # the state at the next chunk's start, exactly
            dec = lam[:, None] ** (m - 1 - torch.arange(m))[None]
            nxt = lam[:, None, None] ** m * Hs + torch.einsum("hj,jhd,jhe->hde", dec, k[x], v[x])
            states = {c + C: nxt}
        bound += 1.01 * u * out.abs() + (2.0 ** -25 if half else 0.0)
        chunks = (n + C - 1) // C
        res.append((out, bound, S, A * 2.0 ** -23 * (48 + 4 * chunks) + 1e-37))
    return res


def to_device(t):
    import torch
    d = {}
    for name, x in t.items():
        if not x.is_contiguous():
            flat = torch.empty(0, dtype=x.dtype).set_(x.untyped_storage()).cuda()
            d[name] = flat.as_strided(x.shape, x.stride(), x.storage_offset())
        else:
            d[name] = x.cuda()
    return d


def run(t, s0, scale, step=False, places=None, in_place=False, want_state=True, rows_max=None, n_states=None,
        ws_fill=0x5A, stream=None):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    d = to_device(t)
    idx = None if places is None else torch.tensor(places, dtype=torch.int32, device="cuda")
    if step:
        d.pop("row_offsets")
    p = dsa.LinearProblem.from_tensors(scale=scale, state_idx=idx, n_states=n_states, **d)
    if rows_max is not None:
        p.set(rows_max=rows_max)
    ws = dsa.alloc_linear_workspace(p)
    ws.fill_(ws_fill)
    out = torch.full((p.R, p.H, p.D_v), 77.0, dtype=t["q"].dtype, device="cuda")
    sin = None if s0 is None else s0.cuda()
    sout = sin if in_place else (torch.full((p.n_states, p.H, p.D_k, p.D_v), 77.0, device="cuda") if want_state else None)
    (dsa.dsa_linear_step if step else dsa.dsa_linear_attn)(p, sin, sout, out, ws, stream=stream)
    bits = dsa.dsa_read_device_status(ws)
    return out.cpu(), None if sout is None else sout.cpu(), bits


def check(t, s0, scale, out, state, places=None, only=None):
    import torch
    ro = t["row_offsets"].tolist()
    for b, (o, bound, S, sb) in enumerate(reference(t, s0, scale, places)):
        if only is not None and b not in only:
            continue
        got = out[ro[b]:ro[b + 1]].double()
        err = (got - o).abs()
        assert torch.isfinite(got).all()
        assert bool((err <= bound).all()), f"request {b}: output off by {(err / bound.clamp(min=1e-300)).max():.3g} x its bound"
        if state is not None:
            e = (state[b if places is None else places[b]].double() - S).abs()
            assert bool((e <= sb).all()), f"request {b}: state off by {(e / sb).max():.3g} x its bound"
