"""Dense attention on the GPU (dsa_dense_attn) against the definition in 64 bits
(tests/dense_harness.py holds the bounds and where they come from)."""
import math

import pytest

import dense_harness as H

pytestmark = pytest.mark.gpu

W = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,hq,hkv", [
    ([1], [1], 1, 1),
    ([1], [129], 4, 2),
    ([1, 1, 1, 1, 1], [0, 127, 128, 1, 300], 8, 2),         # single tokens, one place unused
    ([4, 1, 3], [260, 77, 3], 6, 2),                        # a few rows each, three heads to a K/V head
    ([130], [130], 2, 2),                                   # a prompt a little over one row tile
    ([300, 1, 65, 129], [300, 1, 400, 129], 2, 1),
    ([257], [1000], 3, 1),
])
def test_matches_definition(dk, dv, dtype, rows, lens, hq, hkv):
    t = H.make(rows, lens, hq, hkv, dk, dv, dtype, seed=dk + len(rows))
    scale = 1 / math.sqrt(dk)
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    H.check(t, scale, out, lse)


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("rows,hq,hkv,L", [(1, 8, 1, 6000), (1, 2, 2, 2500), (3, 4, 4, 3001), (200, 2, 1, 1700)])
def test_split_cache(dk, dv, rows, hq, hkv, L):
    # One request with few row tiles: the positions are split over the grid and joined.
    t = H.make([rows], [L], hq, hkv, dk, dv, seed=L)
    scale = 1 / math.sqrt(dk)
    out, lse, bits = H.run(t, scale)
    assert bits == 0
    H.check(t, scale, out, lse)


@pytest.mark.parametrize("rows,hq,hkv,L", [(2570, 16, 16, 5200), (900, 48, 16, 1900), (2600, 16, 8, 5300)])
def test_last_wave_in_parts(rows, hq, hkv, L):
    # A chunk behind a cache as long: more items than SMs, the last ones split and joined.
    t = H.make([rows], [L], hq, hkv, 64, 64, seed=L)
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    keep = sorted({0, 1, 127, 128, rows // 2, rows - 1} | set(range(3, rows, 61)))
    few = dict(t, q=t["q"][keep], row_len=t["row_len"][keep])
    import torch
    few["row_offsets"] = torch.tensor([0, len(keep)], dtype=torch.int32)
    H.check(few, 0.125, out[keep], lse[keep])
    again, _, _ = H.run(t, 0.125, rows_max=rows, ws_fill=0xC3)
    assert again.equal(out)
    assert torch.isfinite(out.float()).all() and not (out == 77.0).all(dim=2).any()


@pytest.mark.parametrize("rows_max", [None, 0, 4000])
def test_rows_max_only_changes_the_split(rows_max):
    t = H.make([2, 140, 1], [500, 140, 900], 4, 2, 128, 128, seed=9)
    out, lse, bits = H.run(t, 0.09, rows_max)
    assert bits == 0
    H.check(t, 0.09, out, lse)


def test_rows_max_too_small_is_flagged():
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([600, 600], [600, 600], 1, 1, 64, 64, seed=2)
    _, _, bits = H.run(t, 0.125, rows_max=1)
    assert bits & dsa.DSA_DEVICE_CAPACITY


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([200, 150], [700, 150]), ([1, 2], [700, 333])])
def test_any_row_len(dtype, rows, lens):
    # row_len need not be causal: random lengths, none for some rows, in any order.
    import torch
    g = torch.Generator().manual_seed(3)
    rl = [int(torch.randint(0, L + 1, (1,), generator=g)) * (i % 5 != 1) for n, L in zip(rows, lens) for i in range(n)]
    t = H.make(rows, lens, 4, 2, 128, 128, dtype, seed=4, row_len=rl)
    out, lse, bits = H.run(t, 0.1)
    assert bits == 0
    H.check(t, 0.1, out, lse)
    empty = t["row_len"] == 0
    assert not out[empty].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [[1, 1, 1], [40, 1, 170]])
def test_values_no_row_sees(bad, rows):
    # What lies behind the last position that a request's rows see (cache slots
    # not yet written, another request's rows) must not reach the output.
    lens = [300, 140, 500]
    rl = [x for n, L in zip(rows, lens) for x in range(L - 60 - n, L - 60)]
    t = H.make(rows, lens, 4, 2, 128, 128, seed=5, row_len=rl)
    o = t["offsets"].tolist()
    for b, L in enumerate(lens):
        t["k"][o[b] + L - 61:o[b + 1]] = bad
        t["v"][o[b] + L - 61:o[b + 1]] = bad
    got, lse, bits = H.run(t, 0.09)
    assert bits == 0
    clean = {x: y.clone() for x, y in t.items()}
    for x in "kv":
        clean[x][~t[x].isfinite()] = 0.0
    H.check(clean, 0.09, got, lse)


def test_masked_keys_of_a_prompt_may_be_anything():
    # K of positions that some rows mask: any value, for those rows.
    t = H.make([100], [100], 2, 1, 128, 128, seed=6)
    t["k"][60:] = float("inf")
    got, lse, _ = H.run(t, 0.09)
    clean = {x: y.clone() for x, y in t.items()}
    clean["k"][60:] = 0.0
    H.check(clean, 0.09, got, lse, rows=slice(0, 60))


@pytest.mark.parametrize("amp", [8.0, 40.0])
def test_growing_maximum(amp):
    # Logits that grow along the cache by far more than 2^8 from tile to tile:
    # the running maximum is renewed and the sums are rescaled.
    import torch
    for rows in ([1], [300]):
        t = H.make(rows, [900], 2, 1, 64, 64, seed=7)
        ramp = torch.linspace(0.0, 1.0, 900)[:, None, None]
        t["q"][:] = t["q"].abs() + 0.5
        t["k"] = (t["k"].float().abs() * amp * ramp).to(torch.bfloat16)
        out, lse, bits = H.run(t, 0.125)
        assert bits == 0
        H.check(t, 0.125, out, lse)


@pytest.mark.parametrize("rows,lens", [([1, 1, 2], [700, 300, 900]), ([150, 300], [150, 900])])
def test_strides_of_a_fused_projection(rows, lens):
    t = H.make(rows, lens, 4, 2, 64, 64, seed=8, fused=True)
    assert not t["q"].is_contiguous() and not t["k"].is_contiguous()
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse)


@pytest.mark.parametrize("rows", [[1, 1], [130, 2]])
def test_rows_behind_the_last_request_stay(rows):
    t = H.make(rows, [200, 400], 2, 2, 128, 128, seed=10, extra_rows=5)
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)
    assert (out[-5:] == 77.0).all() and (lse[-5:] == 77.0).all()


@pytest.mark.parametrize("rows,L,hq,hkv,front", [
    (1, 700, 4, 1, 0), (3, 5000, 4, 1, 0), (3, 700, 4, 1, 2), (200, 300, 4, 4, 0), (200, 300, 4, 4, 3),
    (300, 700, 80, 80, 3),       # more items than SMs, the last ones in parts
])
def test_rows_around_a_single_request_stay(rows, L, hq, hkv, front):
    # One request takes part of the call's rows, as the padded batch of a captured graph has it.
    t = H.make([rows], [L], hq, hkv, 64, 64, seed=12, extra_rows=8)
    t["row_len"][rows:] = L            # a length that would be computed
    if front:
        for x in ("q", "row_len"):
            t[x] = t[x].roll(front, 0)
        t["row_offsets"] += front
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse, rows=slice(front, front + rows))
    for x in (out, lse):
        assert (x[:front] == 77.0).all() and (x[front + rows:] == 77.0).all()


def test_length_beyond_the_request_is_clamped_and_flagged():
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([1, 2], [100, 200], 2, 1, 128, 128, seed=11)
    t["row_len"][0] = 150
    t["row_len"][1] = -3
    out, lse, bits = H.run(t, 0.09)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    H.check(t, 0.09, out, lse)


def test_no_rows_and_empty_cache():
    import torch
    t = H.make([2, 1], [0, 0], 2, 1, 128, 128)
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0 and not out.any() and torch.isinf(lse).all()
    t = H.make([0, 0], [10, 20], 2, 1, 128, 128)
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0 and out.numel() == 0


@pytest.mark.parametrize("B", [33, 64, 65, 100, 700])
def test_many_requests(B):
    # More requests than one warp looks up at a time, or than the lookup table has
    # blocks, some without rows.
    rows = [i % 3 for i in range(B)]
    lens = [(37 * i) % 211 for i in range(B)]
    t = H.make(rows, lens, 2, 1, 64, 64, seed=12)
    out, lse, bits = H.run(t, 0.125)
    assert bits == 0
    H.check(t, 0.125, out, lse)


def test_without_lse_and_repeatable():
    import torch
    t = H.make([1, 200], [3000, 200], 4, 2, 128, 128, seed=13)
    a, _, _ = H.run(t, 0.09, with_lse=False)
    b, _, _ = H.run(t, 0.09, ws_fill=0xC3)
    assert torch.equal(a, b)


def test_graph_replay_and_another_stream():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    probs = []
    for seed, rows, L in ((1, [1], [4000]), (2, [260], [260])):
        t = H.make(rows, L, 4, 2, 128, 128, seed=seed)
        p, d = H.problem(t, 0.09)
        out = torch.zeros(p.R, 4, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(p.R, 4, device="cuda")
        probs.append((t, p, d, out, lse, dsa.alloc_dense_workspace(p)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for t, p, d, out, lse, ws in probs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            dsa.dsa_dense_attn(p, out, lse, ws)
        graphs.append(g)
    for t, p, d, out, lse, ws in probs:      # new values in the captured buffers
        for x in "qkv":
            t[x] = t[x].flip(0).contiguous()
            d[x].copy_(t[x])
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for t, p, d, out, lse, ws in probs:
        H.check(t, 0.09, out.cpu(), lse.cpu())
        out.zero_()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, (t, p, d, out, lse, ws) in zip(side, probs):   # both at once, each with its workspace
        for _ in range(3):
            dsa.dsa_dense_attn(p, out, lse, ws, stream=st)
    torch.cuda.synchronize()
    for t, p, d, out, lse, ws in probs:
        assert dsa.dsa_read_device_status(ws) == 0
        H.check(t, 0.09, out.cpu(), lse.cpu())


def test_long_offsets_pass_32_bits():
    # Element offsets into k and v past 2^32 (8.6 GB each): the second request
    # lies behind a long first one.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    far, L, hkv, D = (1 << 32) // (8 * 128) + 1000, 700, 8, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(far + L, hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = H.make([2], [L], hkv, hkv, D, D, seed=14)
    k[far:].copy_(small["k"])
    v[far:].copy_(small["v"])
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    p = dsa.DenseProblem.from_tensors(q=small["q"].cuda(), k=k, v=v, offsets=i32(0, far, far + L),
                                      row_offsets=i32(0, 0, 2), row_len=small["row_len"].cuda(), softmax_scale=0.09)
    out = torch.zeros(2, hkv, D, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_dense_workspace(p)
    dsa.dsa_dense_attn(p, out, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    H.check(small, 0.09, out.cpu(), None)


@pytest.mark.parametrize("rows,lens", [([1], [3000]), ([400, 1], [400, 900])])
def test_a_wait_that_runs_out(rows, lens):
    # The first K tile never lands: the call returns with the status bit, and the
    # workspace and the context go on working.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make(rows, lens, 4, 2, 128, 128, seed=20)
    p, d = H.problem(t, 0.09)
    out = torch.zeros(p.R, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_dense_workspace(p)
    dsa.dsa_test_dense_missing_tile(p, out, None, ws, 1_000_000)
    assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEVICE_TIMEOUT
    dsa.dsa_dense_attn(p, out, None, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    H.check(t, 0.09, out.cpu(), None)
