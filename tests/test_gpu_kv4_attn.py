"""Attention over the 4-bit cache on the GPU (dsa_kv4_attn) against the definition in 64 bits
(tests/kv4_harness.py holds the bounds and where they come from)."""
import math

import pytest

import kv4_harness as H

pytestmark = pytest.mark.gpu

W = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dt,ps", [("bf16", 16), ("fp16", 32), ("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("rows,lens,hq,hkv", [
    ([1], [1], 1, 1),
    ([1], [129], 4, 2),
    ([1, 1, 1, 1, 1], [0, 127, 128, 1, 300], 8, 2),         # single tokens, one place unused
    ([1, 1], [1030, 17], 16, 1),                            # sixteen heads to a K/V head
    ([4, 1, 3], [260, 77, 3], 6, 2),                        # a few rows each, three heads to a K/V head
    ([130], [130], 2, 2),                                   # a prompt a little over one row tile
    ([300, 1, 65, 129], [300, 1, 400, 129], 2, 1),
    ([257], [1000], 3, 1),
])
def test_matches_definition(dk, dv, dt, ps, rows, lens, hq, hkv):
    t = H.make(rows, lens, hq, hkv, dk, dv, ps, dt, seed=dk + len(rows))
    scale = 1 / math.sqrt(dk)
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    H.check(t, scale, out, lse)


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("rows,hq,hkv,L", [(1, 8, 1, 6000), (1, 2, 2, 2500), (3, 4, 4, 3001), (1, 16, 2, 9000), (200, 2, 1, 1700)])
def test_split_cache(dk, dv, rows, hq, hkv, L):
    # One request: its positions are shared out over the grid and joined.
    t = H.make([rows], [L], hq, hkv, dk, dv, 64, seed=L)
    scale = 1 / math.sqrt(dk)
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    H.check(t, scale, out, lse)


@pytest.mark.parametrize("rows_max", [None, 0, 1, 4000])
def test_rows_max_only_changes_the_kernel(rows_max):
    # (one too small is allowed as well: it sizes nothing)
    t = H.make([2, 140, 1], [500, 140, 900], 4, 2, 128, 128, 32, seed=9)
    out, lse, bits = H.run(t, 0.09, rows_max=rows_max)
    assert bits == 0
    H.check(t, 0.09, out, lse)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([200, 150], [700, 150]), ([1, 2], [700, 333]), ([3, 9, 1], [300, 200, 100])])
def test_any_row_len(dt, rows, lens):
    # row_len need not be causal: random lengths, none for some rows, in any order.
    import torch
    g = torch.Generator().manual_seed(3)
    rl = [int(torch.randint(0, L + 1, (1,), generator=g)) * (i % 5 != 1) for n, L in zip(rows, lens) for i in range(n)]
    t = H.make(rows, lens, 4, 2, 128, 128, 64, dt, seed=4, row_len=rl)
    out, lse, bits = H.run(t, 0.1)
    assert bits == 0
    H.check(t, 0.1, out, lse)
    assert not out[t["row_len"] == 0].any()


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("rows", [[1, 1, 1], [40, 1, 170]])
def test_places_no_row_sees(rows, ps):
    # What lies behind the last position that a request's rows see, in its last page or in pages of others,
    # must not reach the output: scales of NaN and infinity, any codes.
    import torch
    lens = [300, 140, 500]
    rl = [x for n, L in zip(rows, lens) for x in range(L - 60 - n, L - 60)]
    t = H.make(rows, lens, 4, 2, 128, 128, ps, seed=5, row_len=rl)
    dirty = dict(t, pages=t["pages"].clone())
    keep = torch.zeros(t["pages"].shape[0], ps, dtype=torch.bool)
    for b, L in enumerate(lens):
        for x in range(L - 61):
            keep[t["table"][b, x // ps], x % ps] = True
    kc, vc, ks, vs = H.parts(dirty["pages"], 128, 128, ps)
    gone = ~keep[:, None, None, :]
    ks.masked_fill_(gone, float("nan"))
    vs.masked_fill_(gone, float("inf"))
    kc.masked_fill_(gone[..., None], 0)
    vc.masked_fill_(gone[..., None], 0xF0)
    dirty["table"] = t["table"].clone()
    for b, L in enumerate(lens):
        dirty["table"][b, -(-(L - 61) // ps):] = 1 << 30
    got, lse, bits = H.run(dirty, 0.09)
    assert bits == 0
    H.check(t, 0.09, got, lse)


def test_masked_keys_of_a_prompt_may_be_anything():
    # K of positions that some rows mask: any scale, for those rows.
    import torch
    t = H.make([100], [100], 2, 1, 128, 128, 64, seed=6)
    dirty = dict(t, pages=t["pages"].clone())
    ks = H.parts(dirty["pages"], 128, 128, 64)[2]
    ks[t["table"][0, 1].long()] = float("inf")         # positions 64 on
    got, lse, _ = H.run(dirty, 0.09)
    H.check(t, 0.09, got, lse, rows=slice(0, 64))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("amp", [0.0, 8.0, 40.0])
def test_peaked_and_flat(amp, dt):
    t = H.make([1, 3], [2000, 900], 8, 2, 128, 128, 32, dt, seed=11, amp=amp)
    out, lse, bits = H.run(t, 1 / math.sqrt(128))
    assert bits == 0
    H.check(t, 1 / math.sqrt(128), out, lse)


@pytest.mark.parametrize("qx,kx,vx", [(-90, 90, 0), (90, -90, 60), (0, 0, -100), (0, 0, 100)])
@pytest.mark.parametrize("rows", [1, 150])
def test_magnitudes(rows, qx, kx, vx):
    # Queries, keys and values far from 1: powers of two that cancel in the logits.
    import torch
    t = H.make([rows], [700], 4, 2, 64, 64, 64, seed=12)
    t["q"] = (t["q"].float() * 2.0 ** qx).bfloat16()
    _, _, ks, vs = H.parts(t["pages"], 64, 64, 64)
    ks.copy_((ks.float() * 2.0 ** kx).bfloat16())
    vs.copy_((vs.float() * 2.0 ** vx).bfloat16())
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse)


def test_scales_of_all_sizes():
    # V's scales grow by 2^40 along the cache and shrink again; groups of zeros.
    import torch
    t = H.make([1, 2], [1500, 800], 8, 2, 128, 128, 16, seed=13)
    vs = H.parts(t["pages"], 128, 128, 16)[3]
    f = torch.exp2(torch.randint(-20, 21, vs.shape, generator=torch.Generator().manual_seed(1)).float())
    vs.copy_((vs.float() * f).bfloat16())
    vs[:, :, 1, ::3] = 0
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)


def test_scale_that_is_not_finite_reaches_its_request_alone():
    import torch
    t = H.make([1, 1, 1], [300, 200, 300], 4, 2, 64, 64, 64, seed=14)
    clean = dict(t, pages=t["pages"].clone())
    vs = H.parts(t["pages"], 64, 64, 64)[3]
    vs[t["table"][1, 0].long(), :, 0, 5] = float("nan")
    out, lse, _ = H.run(t, 0.1)
    assert out[1].isnan().all()
    H.check(clean, 0.1, torch.where(out.isnan(), 0, out), lse, rows=[0, 2])


@pytest.mark.parametrize("rows", [[1, 1], [70, 3]])
def test_bad_pages_are_masked_and_flagged(rows):
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make(rows, [500, 300], 4, 2, 128, 128, 32, seed=15)
    t["table"][0, 3] = -5
    t["table"][0, 7] = t["pages"].shape[0]
    t["table"][1, 0] = (1 << 31) - 1
    out, lse, bits = H.run(t, 0.09)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    H.check(t, 0.09, out, lse)
    t["table"][:] = -1
    out, lse, bits = H.run(t, 0.09)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX and not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("rows", [[1, 2], [150, 2]])
def test_row_len_outside_is_clamped_and_flagged(rows):
    import dsa_sparse_attention_03_gb300 as dsa
    n = sum(rows)
    t = H.make(rows, [320, 320], 4, 2, 64, 64, 64, seed=16, row_len=[-3] + [1000] + [100] * (n - 2))
    out, lse, bits = H.run(t, 0.1, L_max=1000)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    good = dict(t, row_len=t["row_len"].clamp(0, 320))
    H.check(good, 0.1, out, lse)
    out, lse, bits = H.run(t, 0.1, L_max=90)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    H.check(dict(t, row_len=t["row_len"].clamp(0, 90)), 0.1, out, lse)


@pytest.mark.parametrize("rows", [[2, 3], [150, 2]])
def test_rows_outside_are_left_alone(rows):
    import torch
    t = H.make(rows, [400, 400], 4, 2, 64, 64, 64, seed=17, extra_rows=3)
    t["row_offsets"] += 2
    t["row_len"] = torch.cat([t["row_len"][-2:], t["row_len"][:-2]])
    out, lse, bits = H.run(t, 0.1)
    n = sum(rows)
    assert bits == 0 and (out[:2] == 77).all() and (out[2 + n:] == 77).all() and (lse[:2] == 77).all() and (lse[2 + n:] == 77).all()
    H.check(t, 0.1, out, lse, rows=slice(2, 2 + n))


@pytest.mark.parametrize("rows", [1, 100])
def test_shared_pages_and_a_strided_query(rows):
    # Two requests over one prefix; queries out of a fused projection.
    t = H.make([rows, rows], [400, 400], 8, 2, 128, 128, 64, seed=18, fused=True)
    t["table"][1, :5] = t["table"][0, :5]
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)


@pytest.mark.parametrize("B", [33, 300, 1500])
def test_many_requests(B):
    import torch
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[B // 2] = 1500
    rows = [(1 if i % 7 else 0) + (2 if i % 31 == 0 else 0) for i in range(B)]
    rows = [min(r, max(n, 1)) for r, n in zip(rows, lens)]
    t = H.make(rows, lens, 2, 1, 64, 64, 16, seed=B)
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse)


def test_most_requests():
    rows, lens = [1] * 4096, [(7 * i) % 40 for i in range(4096)]
    t = H.make(rows, lens, 1, 1, 64, 64, 16, seed=1)
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse)


@pytest.mark.parametrize("rows", [1, 130])
def test_pages_beyond_32_bits(rows):
    # A pool of more than 2^32 bytes; the request's pages are its first and its last.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([rows], [300], 16, 8, 128, 128, 128, seed=19, spare=0)
    n = (1 << 32) // (8 * H.block_bytes(128, 128, 128)) + 40
    pool = dsa.alloc_kv4_pages(n, 8, 128, 128, 128)
    at = torch.tensor([n - 1, 0, n - 7])
    pool[at.cuda()] = t["pages"][t["table"][0].long()].cuda()
    cache = dsa.KV4Cache.from_tensors(pages=pool, table=at.int()[None].cuda(), page_size=128, D_k=128, D_v=128)
    prob = dsa.KV4Problem.from_tensors(cache=cache, q=t["q"].cuda(), row_offsets=t["row_offsets"].cuda(),
                                       row_len=t["row_len"].cuda(), softmax_scale=0.09)
    out = torch.empty(rows, 16, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    dsa.dsa_kv4_attn(prob, out, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    H.check(t, 0.09, out.cpu(), None)


@pytest.mark.parametrize("rows,lens,hq", [([1], [3000], 8), ([1, 4, 2], [3000, 40, 700], 8), ([150, 1], [700, 2000], 8)])
def test_same_bits_every_time_and_captured(rows, lens, hq):
    # Eager twice with another workspace content, then captured and replayed with new inputs in place.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make(rows, lens, hq, 2, 128, 128, 64, seed=20)
    a, la, _ = H.run(t, 0.09)
    b, lb, _ = H.run(t, 0.09, ws_fill=0xC3)
    assert a.equal(b) and la.equal(lb)
    prob = H.problem(t, 0.09)
    out = torch.zeros_like(a, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dsa.dsa_kv4_attn(prob, out, None, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_kv4_attn(prob, out, None, ws)
    other = H.make(rows, lens, hq, 2, 128, 128, 64, seed=21)
    prob._keep["q"].copy_(other["q"])
    prob._keep_cache._keep["pages"].copy_(other["pages"])
    prob._keep_cache._keep["table"].copy_(other["table"])
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert dsa.dsa_read_device_status(ws) == 0
    want, _, _ = H.run(other, 0.09)
    assert out.cpu().equal(want)


def test_two_streams_at_once():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    ts = [H.make([1, 3], [4000, 900], 8, 2, 128, 128, 64, seed=22 + i) for i in range(2)]
    want = [H.run(t, 0.09)[0] for t in ts]
    probs = [H.problem(t, 0.09) for t in ts]
    outs = [torch.zeros_like(w, device="cuda") for w in want]
    wss = [dsa.alloc_kv4_workspace(p) for p in probs]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, o, w, s in zip(probs, outs, wss, streams):
            dsa.dsa_kv4_attn(p, o, None, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert o.cpu().equal(w)


def test_input_written_just_before():
    # The call's first kernel starts under what precedes it in the stream and waits there.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([1, 2], [900, 900], 8, 2, 128, 128, 64, seed=25)
    want, _, _ = H.run(t, 0.09)
    prob = H.problem(t, 0.09)
    q = prob._keep["q"]
    good = q.clone()
    out = torch.zeros_like(want, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    for _ in range(20):
        q.fill_(3.0)
        torch.cuda._sleep(20000)
        q.copy_(good)
        dsa.dsa_kv4_attn(prob, out, None, ws)
    assert out.cpu().equal(want)


def test_nothing_to_do():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([0, 0], [100, 30], 4, 2, 64, 64, 64, seed=26)
    out, lse, bits = H.run(t, 0.1)
    assert bits == 0 and out.numel() == 0


@pytest.mark.parametrize("rows", [[1], [200]])
def test_missing_stage_is_bounded(rows):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make(rows, [2000], 8, 2, 128, 128, 64, seed=27)
    prob = H.problem(t, 0.09)
    out = torch.zeros(prob.R, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    dsa.dsa_test_kv4_missing_stage(prob, out, None, ws, 20_000_000)
    assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEVICE_TIMEOUT
    dsa.dsa_kv4_attn(prob, out, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    H.check(t, 0.09, out.cpu(), None)


# Many rows of a request: the pages are widened into the workspace first.

def _few(t, keep):
    """The problem's rows `keep` (of one or several requests, ascending) alone."""
    import torch
    ro = t["row_offsets"].tolist()
    n = [sum(1 for r in keep if a <= r < b) for a, b in zip(ro, ro[1:])]
    return dict(t, q=t["q"][keep], row_len=t["row_len"][keep], row_offsets=H.prefix(n))


def _is_copied(t, scale):
    # (told by the workspace, which holds K and V in 16 bits then)
    import dsa_sparse_attention_03_gb300 as dsa
    prob = H.problem(t, scale)
    return dsa.dsa_kv4_workspace_size(prob) >= len(t["table"]) * prob.L_max * t["pages"].shape[1] * (t["dk"] + t["dv"]) * 2


def _sample(rows, step=37):
    out, r = [], 0
    for n in rows:
        out += sorted({r, r + n - 1, r + n // 2} | set(range(r + 2, r + n, step)))
        r += n
    return out


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dt,ps,rows,lens,hq,hkv", [
    ("bf16", 64, [1030], [1030], 8, 1),
    ("fp16", 16, [300, 1, 513, 0, 7], [300, 900, 1500, 40, 7], 16, 2),
    ("bf16", 128, [400], [2500], 7, 1),                      # a group that does not divide a row tile
])
def test_copied(dk, dv, dt, ps, rows, lens, hq, hkv):
    t = H.make(rows, lens, hq, hkv, dk, dv, ps, dt, seed=dk + ps)
    scale = 1 / math.sqrt(dk)
    assert _is_copied(t, scale)
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    keep = _sample(rows)
    H.check(_few(t, keep), scale, out[keep], lse[keep])
    again, _, _ = H.run(t, scale, ws_fill=0xC3)
    assert again.equal(out)


def test_copied_and_not_agree():
    # The three kernels on one problem: few rows at a time, widened by the way, widened first.
    t = H.make([600, 2], [900, 40], 16, 2, 128, 128, 32, seed=40)
    assert _is_copied(t, 0.09)
    outs = [H.run(t, 0.09, rows_max=n)[0].double() for n in (1, 300, 600)]
    ref, _, bound, _ = H.reference(_few(t, _sample([600, 2])), 0.09)
    for out in outs:
        assert bool(((out[_sample([600, 2])] - ref).abs() <= bound).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_copied_any_row_len_and_places_no_row_sees(dt):
    import torch
    g = torch.Generator().manual_seed(41)
    rows, lens, ps = [700, 560], [900, 640], 64
    rl = [int(torch.randint(0, L - 60, (1,), generator=g)) * (i % 5 != 1) for n, L in zip(rows, lens) for i in range(n)]
    t = H.make(rows, lens, 16, 2, 128, 128, ps, dt, seed=41, row_len=rl)
    assert _is_copied(t, 0.1)
    dirty = dict(t, pages=t["pages"].clone(), table=t["table"].clone())
    seen = torch.zeros(t["pages"].shape[0], ps, dtype=torch.bool)
    for b, (n, a) in enumerate(zip(rows, (0, rows[0]))):
        far = max(rl[a:a + n])
        for x in range(far):
            seen[t["table"][b, x // ps], x % ps] = True
        dirty["table"][b, -(-far // ps):] = -9
    _, _, ks, vs = H.parts(dirty["pages"], 128, 128, ps)
    ks.masked_fill_(~seen[:, None, None], float("inf"))
    vs.masked_fill_(~seen[:, None, None], float("nan"))
    out, lse, bits = H.run(dirty, 0.1)
    assert bits == 0 and not out[t["row_len"] == 0].any()
    keep = _sample(rows)
    H.check(_few(t, keep), 0.1, out[keep], lse[keep])


def test_copied_bad_pages_are_masked_and_flagged():
    import dsa_sparse_attention_03_gb300 as dsa
    rows = [600, 520]
    t = H.make(rows, [900, 600], 16, 2, 128, 128, 32, seed=42)
    assert _is_copied(t, 0.09)
    t["table"][0, 3] = -5
    t["table"][0, 20] = t["pages"].shape[0]
    out, lse, bits = H.run(t, 0.09)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    keep = _sample(rows)
    H.check(_few(t, keep), 0.09, out[keep], lse[keep])
    t["table"][1] = -1
    out, lse, bits = H.run(t, 0.09)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX and not out[600:].any() and (lse[600:] == -math.inf).all()
    H.check(_few(t, keep), 0.09, out[keep], lse[keep])


def test_copied_row_len_outside_and_rows_outside():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([560, 540], [640, 640], 16, 2, 64, 64, 64, seed=43, extra_rows=3)
    assert _is_copied(t, 0.1)
    t["row_offsets"] += 2
    t["row_len"] = torch.cat([t["row_len"][-2:], t["row_len"][:-2]])
    t["row_len"][5], t["row_len"][9] = -4, 5000
    out, lse, bits = H.run(t, 0.1, L_max=700)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    assert (out[:2] == 77).all() and (out[1102:] == 77).all() and (lse[1102:] == 77).all()
    good = dict(t, row_len=t["row_len"].clamp(0, 640))
    keep = [2 + x for x in _sample([560, 540])] + [5, 9]
    keep = sorted(set(keep))
    few = dict(good, q=t["q"][keep], row_len=good["row_len"][keep],
               row_offsets=H.prefix([sum(r < 562 for r in keep), sum(r >= 562 for r in keep)]))
    H.check(few, 0.1, out[keep], lse[keep])


def test_copied_captured():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    rows, lens = [600, 1], [700, 2000]
    t, other = (H.make(rows, lens, 16, 2, 128, 128, 64, seed=44 + i) for i in range(2))
    assert _is_copied(t, 0.09)
    prob = H.problem(t, 0.09)
    out = torch.zeros(601, 16, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dsa.dsa_kv4_attn(prob, out, None, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_kv4_attn(prob, out, None, ws)
    prob._keep["q"].copy_(other["q"])
    prob._keep_cache._keep["pages"].copy_(other["pages"])
    prob._keep_cache._keep["table"].copy_(other["table"])
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want, _, _ = H.run(other, 0.09)
    assert dsa.dsa_read_device_status(ws) == 0 and out.cpu().equal(want)


def test_copied_missing_tile_is_bounded():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([600], [2000], 16, 2, 128, 128, 64, seed=46)
    assert _is_copied(t, 0.09)
    prob = H.problem(t, 0.09)
    out = torch.zeros(600, 16, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_kv4_workspace(prob)
    dsa.dsa_test_kv4_missing_stage(prob, out, None, ws, 20_000_000)
    assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEVICE_TIMEOUT
    dsa.dsa_kv4_attn(prob, out, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    keep = _sample([600])
    H.check(_few(t, keep), 0.09, out.cpu()[keep], None)


@pytest.mark.parametrize("rows", [1, 150, 600])
def test_values_near_the_end_of_the_range(rows):
    # K's scales of 2^121: 136 of them are beyond bf16, the values are not.  V's of 2^89: the sums of weights (held as up
    # to 2^15 of them) times values have to stay in fp32, 2^15 * 700 * 7 * 2^89 = 2^116.3; with 2^121 as well they
    # would be 2^148.
    t = H.make([rows], [700], 16, 2, 64, 64, 64, seed=47)
    assert _is_copied(t, 0.125) == (rows == 600)
    _, _, ks, vs = H.parts(t["pages"], 64, 64, 64)
    vs.copy_((vs.float() * 2.0 ** 90).bfloat16())
    ks.copy_((ks.float() * 2.0 ** 122).bfloat16())
    t["q"] = (t["q"].float() * 2.0 ** -122).bfloat16()
    out, lse, bits = H.run(t, 0.125)
    keep = _sample([rows])
    assert bits == 0
    H.check(_few(t, keep), 0.125, out[keep], lse[keep])


@pytest.mark.parametrize("B", [31, 32, 33, 65, 290])
@pytest.mark.parametrize("hq,hkv,most", [(8, 1, 1), (4, 2, 5), (2, 2, 20)])
def test_many_requests_are_found(B, hq, hkv, most):
    # Rows that are not their requests' numbers, requests without rows, contexts of nothing to some thousand positions.
    import random
    r = random.Random(B * 100 + most)
    lens = [r.choice([0, 1, 17, 128, 129, r.randint(1, 3000)]) for _ in range(B)]
    rows = [min(r.randint(0, most), x) if x else r.choice([0, 1]) for x in lens]
    t = H.make(rows, lens, hq, hkv, 64, 64, 16, seed=B)
    scale = 0.125
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    H.check(t, scale, out, lse)
