"""The attention operators together, as a serving loop of a hybrid stack calls
them: packed prompts, then single tokens, through a linear-attention layer and a
dense one over caches that grow; and dense attention against the sparse step
where the selection takes every position."""
import math

import numpy as np
import pytest

import dense_harness as DH
import linear_harness as LH

pytestmark = pytest.mark.gpu

H, D, HKV = 4, 64, 2


def test_prompts_then_tokens():
    # Layer 1 linear, layer 2 dense: layer 2's q, k and v are layer 1's output (a fixed
    # scaling of it), so a wrong value of the first layer shows in the second too.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    prompts, new, cap = [130, 1, 257], 4, 320
    B, T = len(prompts), [n + 4 for n in prompts]
    g = torch.Generator().manual_seed(1)
    bf = torch.bfloat16
    x = [torch.randn(t, 3, H, D, generator=g).to(bf) for t in T]           # q, k, v of every token, by request
    ld = torch.log1p(-torch.exp2(-torch.linspace(2.0, 8.0, H).double())).float()
    i32 = lambda a: torch.tensor(list(a), dtype=torch.int32, device="cuda")
    state = torch.zeros(B + 2, H, D, D, device="cuda")
    places = i32([2, 0, 4])
    # Caches with room for every request: request b owns positions b * cap ..
    kc = torch.full((B * cap, HKV, D), float("nan"), dtype=bf, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    offsets = i32(b * cap for b in range(B + 1))
    out1 = [[] for _ in range(B)]
    out2 = [[] for _ in range(B)]

    def layers(parts, first):
        """parts[b]: the request's new tokens; first[b]: their position."""
        n = [p.shape[0] for p in parts]
        tok = torch.cat(parts).cuda()
        ro = i32(np.concatenate([[0], np.cumsum(n)]))
        step = all(m == 1 for m in n)
        lp = dsa.LinearProblem.from_tensors(q=tok[:, 0], k=tok[:, 1], v=tok[:, 2], log_decay=ld.cuda(),
                                            row_offsets=None if step else ro, scale=0.125, state_idx=places,
                                            n_states=B + 2)
        o1 = torch.empty(sum(n), H, D, dtype=bf, device="cuda")
        wl = dsa.alloc_linear_workspace(lp)
        (dsa.dsa_linear_step if step else dsa.dsa_linear_attn)(lp, state, state, o1, wl)
        h = torch.tanh(o1.float()).to(bf)
        where = torch.cat([torch.arange(f, f + m) + b * cap for b, (f, m) in enumerate(zip(first, n))]).cuda()
        kc[where] = h[:, :HKV]
        vc[where] = h[:, HKV:]
        seen = i32(f + i + 1 for f, m in zip(first, n) for i in range(m))
        dp = dsa.DenseProblem.from_tensors(q=h, k=kc, v=vc, offsets=offsets, row_offsets=ro, row_len=seen,
                                           softmax_scale=1.0)
        o2 = torch.empty(sum(n), H, D, dtype=bf, device="cuda")
        wd = dsa.alloc_dense_workspace(dp)
        dsa.dsa_dense_attn(dp, o2, None, wd)
        assert dsa.dsa_read_device_status(wl) == 0 and dsa.dsa_read_device_status(wd) == 0
        at = 0
        for b, m in enumerate(n):
            out1[b].append(o1[at:at + m].cpu())
            out2[b].append(o2[at:at + m].cpu())
            at += m

    layers([x[b][:prompts[b]] for b in range(B)], [0] * B)
    for s in range(new):
        layers([x[b][prompts[b] + s:prompts[b] + s + 1] for b in range(B)], [p + s for p in prompts])
    for b in range(B):
        one = {n: x[b][:, i] for i, n in enumerate("qkv")}
        one["log_decay"] = ld
        one["row_offsets"] = torch.tensor([0, T[b]], dtype=torch.int32)
        o, bound, S, sb = LH.reference(one, None, 0.125)[0]
        got = torch.cat(out1[b])
        assert bool(((got.double() - o).abs() <= bound).all())
        assert bool(((state[int(places[b])].cpu().double() - S).abs() <= sb * (1 + new)).all())
        h = torch.tanh(got.cuda().float()).to(bf).cpu()
        t = dict(q=h, k=h[:, :HKV].contiguous(), v=h[:, HKV:].contiguous(),
                 row_len=torch.arange(1, T[b] + 1, dtype=torch.int32), offsets=torch.tensor([0, T[b]], dtype=torch.int32),
                 row_offsets=torch.tensor([0, T[b]], dtype=torch.int32))
        DH.check(t, 1.0, torch.cat(out2[b]), None)
    assert not state[1].any() and not state[3].any()


@pytest.mark.parametrize("R", [1, 3])
def test_dense_equals_sparse_over_every_position(R):
    # A cache no longer than the top-k: the sparse step selects everything, and is
    # dense attention with one K/V head whose values are the row's first columns.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    L, Hq, Dk = 500, 16, 128
    g = torch.Generator().manual_seed(2)
    q = torch.randn(R, Hq, Dk, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(L, Dk, generator=g).to(torch.bfloat16).cuda()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    seen = i32(*range(L - R + 1, L + 1))
    sp = dsa.Problem(R=R, B=1, H_i=4, D_i=32, H_q=Hq, D_k=Dk, D_v=Dk, k=512, L_max=L, L_total=L,
                     softmax_scale=1 / math.sqrt(Dk), q=q.view(torch.int16), kv=kv.view(torch.int16),
                     offsets=i32(0, L), row_offsets=i32(0, R), row_len=seen)
    idx = torch.full((R, 512), -1, dtype=torch.int32, device="cuda")
    for r in range(R):
        idx[r, :L - R + 1 + r] = torch.arange(L - R + 1 + r, dtype=torch.int32)
    a = torch.empty(R, Hq, Dk, dtype=torch.int16, device="cuda")
    la = torch.empty(R, Hq, device="cuda")
    dsa.dsa_sparse_attn(sp, idx, None, a, la, dsa.alloc_workspace(sp))
    dp = dsa.DenseProblem.from_tensors(q=q, k=kv[:, None], v=kv[:, None], offsets=i32(0, L), row_offsets=i32(0, R),
                                       row_len=seen, softmax_scale=1 / math.sqrt(Dk))
    b = torch.empty(R, Hq, Dk, dtype=torch.bfloat16, device="cuda")
    lb = torch.empty(R, Hq, device="cuda")
    dsa.dsa_dense_attn(dp, b, lb, dsa.alloc_dense_workspace(dp))
    t = dict(q=q.cpu(), k=kv.cpu()[:, None], v=kv.cpu()[:, None], row_len=seen.cpu(),
             offsets=torch.tensor([0, L], dtype=torch.int32), row_offsets=torch.tensor([0, R], dtype=torch.int32))
    DH.check(t, 1 / math.sqrt(Dk), b.cpu(), lb.cpu())
    # Both round the weights and the output to bf16 once: 2^-8 of sum w |v| each way.
    out, _, bound, _ = DH.reference(t, 1 / math.sqrt(Dk))
    assert bool(((a.view(torch.bfloat16).cpu().double() - b.cpu().double()).abs() <= 2 * bound).all())
    assert bool(((la - lb).abs() <= 2e-3).all())


@pytest.mark.parametrize("case", ["tokens", "rows", "prompt", "short rows", "short prompts", "split prompt", "step"])
def test_inputs_written_just_before(case):
    # Each call's first kernel may be resident before what precedes it in the stream has
    # ended: a large copy and this library's own kernels right before, their outputs
    # and the offsets among the inputs, and the last call's workspace and output reused.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(4)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    big = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")      # 40 us of writing
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    if case in ("tokens", "rows", "prompt", "short rows"):
        R, L = {"tokens": (1, 3000), "rows": (400, 700), "prompt": (900, 900), "short rows": (130, 200)}[case]
        src = [[rnd(R, 8, 64), rnd(L, 2, 64), rnd(L, 2, 64),
                i32(*[max(0, L - R + i + 1 - 7 * v) for i in range(R)]), i32(0, L - v), i32(0, R)] for v in range(3)]
        use = [x.clone() for x in src[0]]
        q, k, v, rl, off, ro = use
        prob = dsa.DenseProblem.from_tensors(q=q, k=k, v=v, offsets=off, row_offsets=ro, row_len=rl, L_total=L,
                                             L_max=L, softmax_scale=0.125)
        out, ws = torch.empty(R, 8, 64, dtype=torch.bfloat16, device="cuda"), dsa.alloc_dense_workspace(prob)
        call = lambda: dsa.dsa_dense_attn(prob, out, None, ws)
        outs = [out]
    else:
        rows = {"short prompts": [150, 20, 300], "split prompt": [6000], "step": [1] * 5}[case]
        R, H_ = sum(rows), 4
        pre = [0] + list(np.cumsum(rows))
        src = [[rnd(R, H_, 64), rnd(R, H_, 64), rnd(R, H_, 64), -torch.rand(H_, generator=g).cuda() * 0.01,
                i32(*[max(0, x - v) for x in pre]), torch.randn(len(rows), H_, 64, 64, generator=g).cuda()] for v in range(3)]
        use = [x.clone() for x in src[0]]
        q, k, v, ld, ro, s0 = use
        prob = dsa.LinearProblem.from_tensors(q=q, k=k, v=v, log_decay=ld, row_offsets=None if case == "step" else ro,
                                              scale=0.125, rows_max=max(rows))
        out, s1 = torch.empty(R, H_, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s0)
        ws = dsa.alloc_linear_workspace(prob)
        fn = dsa.dsa_linear_step if case == "step" else dsa.dsa_linear_attn
        call = lambda: fn(prob, s0, s1, out, ws)
        outs = [out, s1]
    want = []
    for v in range(3):                                   # one at a time
        for a, b in zip(use, src[v]):
            a.copy_(b)
        for o in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        assert dsa.dsa_read_device_status(ws) == 0
        want.append([o.clone() for o in outs])
    assert not want[0][0].equal(want[1][0])
    got = []
    side = torch.cuda.Stream()
    for rep in range(12):                                # back to back, every other time written on another stream
        here = torch.cuda.current_stream()
        for o in outs:
            o.fill_(0)
        if rep % 2:
            side.wait_stream(here)
        with torch.cuda.stream(side if rep % 2 else here):
            big.fill_(rep)
            for a, b in zip(use, src[rep % 3]):
                a.copy_(b)
        if rep % 2:
            here.wait_stream(side)
        call()
        got.append([o.clone() for o in outs])
        call()                                           # once more into the same output: what a reader finds is whole
        got.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    for n, x in enumerate(got):
        for a, b in zip(x, want[n // 2 % 3]):
            assert a.equal(b), (n, case)
    assert dsa.dsa_read_device_status(ws) == 0
