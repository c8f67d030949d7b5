"""Dense attention on the GPU where most of what counts has small weights (fp16), and where one
request is much longer than the others, against the definition in 64 bits."""
import pytest

import dense_harness as H

pytestmark = pytest.mark.gpu

W = [(64, 64), (128, 128), (192, 128)]


def peaks_and_tail(rows, L, hq, hkv, dk, dv, depth, seed):
    """A peak every 300 positions, whose value is 0, and between them logits about `depth`
    below, with values of about 1000: the output is the tail's."""
    import torch
    scale = 0.125
    g = torch.Generator().manual_seed(seed)
    t = H.make([rows], [L], hq, hkv, dk, dv, "fp16", seed=seed, row_len=[L - i for i in range(rows)])
    t["q"].zero_()
    t["q"][:, :, 0] = 1.0
    t["k"].zero_()
    t["k"][:, :, 0] = (-(depth + torch.rand(L, hkv, generator=g)) / scale).half()
    t["k"][::300, :, 0] = 0.0
    t["v"] = (1000 + 100 * torch.randn(L, hkv, dv, generator=g)).half()
    t["v"][::300] = 0.0
    return t, scale


def bound_of_small_weights(t, scale):
    """(out, lse, bound, lse's bound) of one request in float64.  As in the harness, but for the
    last term: a weight is held as 2^7 of it, so that what fp16 rounds to half of its
    smallest step is off by 2^-25 2^-7 = 2^-32 of the largest weight."""
    import torch
    q, k, v = (t[x].double() for x in "qkv")
    G, u = q.shape[1] // k.shape[1], 2.0 ** -11
    out, lse, bound, lbound = [], [], [], []
    for r, n in enumerate(t["row_len"].tolist()):
        kk, vv = (x[:n].repeat_interleave(G, dim=1) for x in (k, v))
        s = torch.einsum("hd,nhd->hn", q[r], kk) * scale
        X = torch.einsum("hd,nhd->hn", q[r].abs(), kk.abs()).amax(dim=1) * scale
        m = s.amax(dim=1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(dim=1)
        o = torch.einsum("hn,nhd->hd", p, vv) / z[:, None]
        A = torch.einsum("hn,nhd->hd", p, vv.abs()) / z[:, None]
        e = (2.0 ** -18 * (1 + X))[:, None]
        out.append(o)
        lse.append(m[:, 0] + torch.log(z))
        bound.append(1.01 * u * (A + o.abs()) + 2 * e * A + 2.0 ** -32 * vv.abs().sum(dim=0) / z[:, None] + 2.0 ** -25)
        lbound.append(2 * e[:, 0] + 2.0 ** -22 * lse[-1].abs())
    return tuple(torch.stack(x) for x in (out, lse, bound, lbound))


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("rows,L,hq,hkv", [(1, 20000, 4, 1), (2, 20000, 6, 2), (150, 3000, 2, 2)])
@pytest.mark.parametrize("depth", [9.5, 16.5])
def test_many_small_weights(dk, dv, rows, L, hq, hkv, depth):
    # 2^-14 and 2^-24 of the largest weight: fp16's last normal number, and its last one.
    t, scale = peaks_and_tail(rows, L, hq, hkv, dk, dv, depth, seed=51)
    got, lse, bits = H.run(t, scale)
    assert bits == 0
    out, l, bound, lb = bound_of_small_weights(t, scale)
    err = (got.double() - out).abs()
    assert bool((err <= bound).all()), f"output off by {(err / bound).max():.3g} x its bound"
    assert bool(((lse.double() - l).abs() <= lb).all())


def test_a_long_context_with_one_peak():
    # 307200 positions, one peak 18 above the rest, which is 0.47% of the weight or less; split
    # over the GPU, and in one part.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    L = 307200
    t, scale = peaks_and_tail(1, L, 2, 1, 64, 64, 18.0, seed=52)
    t["k"][300::300] = t["k"][1]
    t["v"][300::300] = t["v"][1]
    p, d = H.problem(t, scale)
    for split in (True, False):
        if not split:                     # other requests, without rows, that fill the GPU
            of = torch.full((4097,), L, dtype=torch.int32)
            ro = torch.ones(4097, dtype=torch.int32)
            of[0] = ro[0] = 0
            d["offsets"], d["row_offsets"] = of.cuda(), ro.cuda()
            p = dsa.DenseProblem.from_tensors(softmax_scale=scale, **d)
        out = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
        lse = torch.zeros(1, 2, device="cuda")
        ws = dsa.alloc_dense_workspace(p)
        dsa.dsa_dense_attn(p, out, lse, ws)
        assert dsa.dsa_read_device_status(ws) == 0
        o, l, bound, lb = bound_of_small_weights(t, scale)
        err = (out.cpu().double() - o).abs()
        assert bool((err <= bound).all()), f"output off by {(err / bound).max():.3g} x its bound (split {split})"
        assert bool(((lse.cpu().double() - l).abs() <= lb).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_long_request_among_short_ones(dtype):
    # More items than the GPU has slots for, of which the long request's are cut.
    rows, lens = [1] * 40, [100, 6000] + [(13 * i) % 90 for i in range(38)]
    t = H.make(rows, lens, 64, 8, 128, 128, dtype, seed=53)
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)
