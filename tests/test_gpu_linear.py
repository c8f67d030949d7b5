"""Linear attention on the GPU (dsa_linear_attn, dsa_linear_step) against the
recurrence in 64 bits (tests/linear_harness.py holds the bounds)."""
import math

import pytest

import linear_harness as H

pytestmark = pytest.mark.gpu

W = [(64, 64), (128, 128), (64, 128), (128, 64)]


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [[1], [128], [129], [127, 1, 300], [5, 0, 256, 64], [600]])
def test_prompts_match_the_recurrence(dk, dv, dtype, rows):
    t, s0 = H.make(rows, 3, dk, dv, dtype, seed=len(rows) + dk)
    out, state, bits = H.run(t, s0, 1 / math.sqrt(dk))
    assert bits == 0
    H.check(t, s0, 1 / math.sqrt(dk), out, state)


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_from_an_empty_state(dk, dv, dtype):
    t, _ = H.make([200, 33], 2, dk, dv, dtype, seed=1)
    out, state, bits = H.run(t, None, 0.1)
    assert bits == 0
    H.check(t, None, 0.1, out, state)
    out2, none, _ = H.run(t, None, 0.1, want_state=False)
    assert none is None and out2.equal(out)


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("rows", [[3000], [1700, 40, 1100]])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_requests_in_segments(dk, dv, rows, in_place):
    # Few heads and long requests: segments of at least 512 tokens on several SMs.
    t, s0 = H.make(rows, 2, dk, dv, seed=3)
    out, state, bits = H.run(t, s0, 0.1, in_place=in_place)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)


def test_segments_from_an_empty_state():
    t, _ = H.make([2000], 2, 128, 128, "fp16", seed=4)
    out, state, bits = H.run(t, None, 0.1)
    assert bits == 0
    H.check(t, None, 0.1, out, state)


@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.7, -30.0, -1000.0, -float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decays(decay, dtype):
    # From nothing forgotten to nothing kept.
    t, s0 = H.make([300, 1], 2, 128, 128, dtype, seed=5, decay=decay)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)
    t, s0 = H.make([1, 1, 1], 2, 64, 64, dtype, seed=6, decay=decay)
    out, state, bits = H.run(t, s0, 0.1, step=True)
    assert bits == 0
    check_step(t, s0, 0.1, out, state)


def test_positive_decay_counts_as_zero():
    a, s0 = H.make([150], 2, 64, 64, seed=7, decay=0.5)
    b = dict(a, log_decay=a["log_decay"] * 0)
    x, y = H.run(a, s0, 0.1), H.run(b, s0, 0.1)
    assert x[0].equal(y[0]) and x[1].equal(y[1])


@pytest.mark.parametrize("amp", [1e-3, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_small_and_large_values(amp, dtype):
    # fp16 holds 6e-5 .. 65504 in full precision: products and states outside it
    # have to be scaled into range.
    scale = 0.1 / amp ** 2
    t, s0 = H.make([300], 2, 128, 64, dtype, seed=8, amp=amp)
    out, state, bits = H.run(t, s0, scale)
    assert bits == 0
    H.check(t, s0, scale, out, state)


def check_step(t, s0, scale, out, state, places=None):
    """fp32 throughout: a decay with |ld2| 2^-23 + 2^-22 of itself, two roundings
    per state value, at most 40 per output (16 rows of a thread, 16 partial sums
    and the products), one rounding of the output."""
    import torch
    u = torch.finfo(t["q"].dtype).eps / 2
    lam = torch.exp(t["log_decay"].double().clamp(max=0.0))
    q, k, v = (t[x].double() for x in "qkv")
    B = q.shape[0]
    for b in range(B):
        at = b if places is None else places[b]
        S0 = s0[at].double() if s0 is not None else torch.zeros(state.shape[1:], dtype=torch.float64)
        S = lam[:, None, None] * S0 + k[b][:, :, None] * v[b][:, None, :]
        A = lam[:, None, None] * S0.abs() + (k[b][:, :, None] * v[b][:, None, :]).abs()
        x = (t["log_decay"].double() * 1.4427).clamp(-300, 0).abs()[:, None, None]
        assert bool(((state[at].double() - S).abs() <= A * 2.0 ** -22 * (2 + x) + 1e-37).all())
        o = scale * torch.einsum("hd,hde->he", q[b], S)
        oa = abs(scale) * torch.einsum("hd,hde->he", q[b].abs(), A)
        lim = 1.01 * u * o.abs() + oa * 2.0 ** -23 * (40 + 4 * x[:, 0]) + 2.0 ** -25
        assert bool(((out[b].double() - o).abs() <= lim).all())


@pytest.mark.parametrize("dk,dv", W)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H_", [(1, 1), (5, 3), (40, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(dk, dv, dtype, B, H_, in_place):
    t, s0 = H.make([1] * B, H_, dk, dv, dtype, seed=B)
    out, state, bits = H.run(t, s0, 0.1, step=True, in_place=in_place)
    assert bits == 0
    check_step(t, s0, 0.1, out, state)


def test_step_from_an_empty_state_and_fused_strides():
    t, _ = H.make([1] * 4, 3, 128, 64, seed=9, fused=True)
    assert not t["q"].is_contiguous()
    out, state, bits = H.run(t, None, 0.1, step=True)
    assert bits == 0
    check_step(t, None, 0.1, out, state)


def test_fused_strides():
    t, s0 = H.make([140, 300], 3, 64, 128, seed=10, fused=True)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_places(step, in_place):
    # Requests name their states' places; one entry of the batch is unused.
    import torch
    rows = [1] * 4 if step else [130, 70, 1, 1500]
    places = [5, -1, 0, 3]
    t, s0 = H.make(rows, 2, 128, 128, seed=11, n_states=7)
    out, state, bits = H.run(t, s0, 0.1, step=step, places=places, in_place=in_place, n_states=7)
    assert bits == 0
    ro = t["row_offsets"].tolist()
    assert (out[ro[1]:ro[2]] == 77.0).all()
    untouched = s0 if in_place else torch.full_like(s0, 77.0)
    for i in (1, 2, 4, 6):
        assert state[i].equal(untouched[i])
    for b in (0, 2, 3):
        one = {x: t[x][ro[b]:ro[b + 1]] if x in "qkv" else t[x] for x in t}
        one["row_offsets"] = torch.tensor([0, rows[b]], dtype=torch.int32)
        H.check(one, s0[places[b]][None], 0.1, out[ro[b]:ro[b + 1]], state[places[b]][None])


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("places", [[1, 2, 1], [0, 9, 1], [2, 2, 2]])
def test_bad_places_are_skipped_and_flagged(step, places):
    import dsa_sparse_attention_03_gb300 as dsa
    rows = [1] * 3 if step else [700, 20, 600]
    t, s0 = H.make(rows, 2, 64, 64, seed=12, n_states=3)
    out, state, bits = H.run(t, s0, 0.1, step=step, places=places, in_place=True, n_states=3)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    ro = t["row_offsets"].tolist()
    seen = set()
    for b, at in enumerate(places):
        good = at < 3 and at not in seen
        seen.add(at)
        if good:
            one = {x: t[x][ro[b]:ro[b + 1]] if x in "qkv" else t[x] for x in t}
            import torch
            one["row_offsets"] = torch.tensor([0, rows[b]], dtype=torch.int32)
            H.check(one, s0[at][None], 0.1, out[ro[b]:ro[b + 1]], state[at][None])
        else:
            assert (out[ro[b]:ro[b + 1]] == 77.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_what_lies_behind_a_request_does_not_reach_it(bad, dtype):
    # Requests share chunk tiles with the rows behind them: another request's, or nobody's.
    t, s0 = H.make([40, 100, 200], 2, 128, 128, dtype, seed=13, extra_rows=60)
    for x in "qkv":
        t[x][40:140] = bad
        t[x][340:] = bad
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    H.check(t, s0, 0.1, out, state, only=(0, 2))
    assert (out[340:] == 77.0).all()


def test_no_tokens():
    t, s0 = H.make([0, 0], 2, 64, 64, seed=14)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0 and state.equal(s0)
    out, state, bits = H.run(t, None, 0.1)
    assert bits == 0 and not state.any()


@pytest.mark.parametrize("rows_max", [1, 500, 0, 100000])
def test_rows_max_only_changes_the_split(rows_max):
    t, s0 = H.make([1400, 90], 1, 64, 64, seed=15)
    out, state, bits = H.run(t, s0, 0.1, rows_max=rows_max)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)


@pytest.mark.parametrize("rows", [[(7 * i) % 40 for i in range(70)], [i % 4 for i in range(900)],
                                  [2, 2000, 0, 1] * 9, [3] * 700 + [1900] + [1] * 20])
def test_many_requests(rows):
    # More than 32, without and with a long one that is split; more than threads.
    t, s0 = H.make(rows, 1, 64, 64, seed=16)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)


def test_repeatable_graph_replay_and_streams():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t, s0 = H.make([1500, 300], 2, 128, 128, seed=17)
    a = H.run(t, s0, 0.1)
    b = H.run(t, s0, 0.1, ws_fill=0xC3)
    assert a[0].equal(b[0]) and a[1].equal(b[1])
    d = H.to_device(t)
    p = dsa.LinearProblem.from_tensors(scale=0.1, **d)
    state = s0.cuda()
    out = torch.zeros(1800, 2, 128, dtype=torch.bfloat16, device="cuda")
    ws = dsa.alloc_linear_workspace(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dsa.dsa_linear_attn(p, state, state, out, ws)      # in place: every replay goes on
    g.replay()
    torch.cuda.synchronize()
    assert out.cpu().equal(a[0]) and state.cpu().equal(a[1])
    g.replay()
    torch.cuda.synchronize()
    H.check(t, a[1], 0.1, out.cpu(), state.cpu())
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:                                     # two calls at once
        o, so, w = torch.zeros_like(out), torch.zeros_like(state), dsa.alloc_linear_workspace(p)
        st.wait_stream(torch.cuda.current_stream())
        outs.append((o, so, w))
    s_in = s0.cuda()
    torch.cuda.synchronize()
    for st, (o, so, w) in zip(streams, outs):
        dsa.dsa_linear_attn(p, s_in, so, o, w, stream=st)
    torch.cuda.synchronize()
    for o, so, w in outs:
        assert o.cpu().equal(a[0]) and so.cpu().equal(a[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prompt_then_steps(dtype):
    """A prompt and then single tokens, as a serving loop calls them, against one
    recurrence over all of them."""
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    n, extra = 137, 5
    t, s0 = H.make([n + extra] * 2, 2, 128, 128, dtype, seed=18)
    ref = H.reference(t, s0, 0.1)
    d = H.to_device(t)
    q, k, v = (d[x].view(2, n + extra, 2, 128) for x in "qkv")
    part = lambda x: x[:, :n].reshape(2 * n, 2, 128)
    ro = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    p = dsa.LinearProblem.from_tensors(q=part(q), k=part(k), v=part(v), log_decay=d["log_decay"], row_offsets=ro, scale=0.1)
    state = s0.cuda()
    out = torch.zeros(2 * n, 2, 128, dtype=d["q"].dtype, device="cuda")
    dsa.dsa_linear_attn(p, state, state, out, dsa.alloc_linear_workspace(p))
    outs = [out.view(2, n, 2, 128)]
    for i in range(n, n + extra):
        tok = lambda x: x[:, i].contiguous()
        sp = dsa.LinearProblem.from_tensors(q=tok(q), k=tok(k), v=tok(v), log_decay=d["log_decay"], scale=0.1)
        o = torch.zeros(2, 2, 128, dtype=d["q"].dtype, device="cuda")
        dsa.dsa_linear_step(sp, state, state, o, dsa.alloc_linear_workspace(sp))
        outs.append(o[:, None])
    got = torch.cat(outs, dim=1).cpu().double()
    for b in range(2):
        o, bound, S, sb = ref[b]
        assert bool(((got[b] - o).abs() <= bound).all())
        assert bool(((state[b].cpu().double() - S).abs() <= sb + sb * extra).all())


@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.7, -30.0, -float("inf")])
def test_segments_with_every_decay(decay):
    # The state launch ends where the decay reaches 0 in fp32: never, or at once.
    t, s0 = H.make([2500], 1, 128, 64, seed=21, decay=decay)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == 0
    H.check(t, s0, 0.1, out, state)


@pytest.mark.parametrize("rows", [[300], [3000]])
def test_a_wait_that_runs_out(rows):
    # The first K and V tile never lands: the call returns with the status bit, and
    # the workspace and the context go on working.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t, s0 = H.make(rows, 2, 128, 128, seed=22)
    d = H.to_device(t)
    p = dsa.LinearProblem.from_tensors(scale=0.1, **d)
    out = torch.zeros(rows[0], 2, 128, dtype=torch.bfloat16, device="cuda")
    sin, sout, ws = s0.cuda(), torch.zeros(1, 2, 128, 128, device="cuda"), dsa.alloc_linear_workspace(p)
    dsa.dsa_test_linear_missing_tile(p, sin, sout, out, ws, 1_000_000)
    assert dsa.dsa_read_device_status(ws) & dsa.DSA_DEVICE_TIMEOUT
    dsa.dsa_linear_attn(p, sin, sout, out, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    H.check(t, s0, 0.1, out.cpu(), sout.cpu())


@pytest.mark.parametrize("step", [False, True])
def test_fewer_places_than_requests_is_flagged(step):
    import dsa_sparse_attention_03_gb300 as dsa
    rows = [1] * 3 if step else [20, 30, 40]
    t, s0 = H.make(rows, 2, 64, 64, seed=23, n_states=2)
    out, state, bits = H.run(t, s0, 0.1, step=step, n_states=2)
    assert bits & dsa.DSA_DEVICE_BAD_INDEX
    ro = t["row_offsets"].tolist()
    assert (out[ro[2]:] == 77.0).all() and not (out[:ro[2]] == 77.0).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_segments_of_many_requests(in_place, dtype):
    # Long and short requests in turn, more than a warp looks up; the long ones are split,
    # one of them and a short one are unused, and the states' places are in another order.
    import torch
    rows = [0, 900, 5, 2000, 1, 1300] + [3] * 30 + [1100, 0, 700]
    B = len(rows)
    places = [(7 * b + 3) % 41 for b in range(B)]
    places[5] = places[8] = -1
    t, s0 = H.make(rows, 2, 64, 128, dtype=dtype, seed=31, n_states=41)
    out, state, bits = H.run(t, s0, 0.1, places=places, in_place=in_place, n_states=41)
    assert bits == 0
    ro = t["row_offsets"].tolist()
    for b, at in enumerate(places):
        if at < 0:
            assert (out[ro[b]:ro[b + 1]] == 77.0).all()
            continue
        one = {x: t[x][ro[b]:ro[b + 1]] if x in "qkv" else t[x] for x in t}
        one["row_offsets"] = torch.tensor([0, rows[b]], dtype=torch.int32)
        H.check(one, s0[at][None], 0.1, out[ro[b]:ro[b + 1]], state[at][None])
    untouched = s0 if in_place else torch.full_like(s0, 77.0)
    for i in set(range(41)) - set(places):
        assert state[i].equal(untouched[i])


@pytest.mark.parametrize("state", [False, True])
def test_many_segments_of_one_head(state):
    # One head on the whole GPU: more segments than the scan loads at a time.
    t, s0 = H.make([20000], 1, 64, 64, seed=32, state=state, decay=-3e-4)
    out, s1, bits = H.run(t, s0, 0.1, in_place=state)
    assert bits == 0
    H.check(t, s0, 0.1, out, s1)


def test_offsets_that_overlap_are_flagged():
    # Three requests over the same rows: more segments than the workspace has end states
    # for.  Those that do not fit are skipped.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t, s0 = H.make([3000], 1, 64, 64, seed=33, n_states=5)
    one = dict(t)
    t["row_offsets"] = torch.tensor([0, 3000, 0, 3000, 0, 3000], dtype=torch.int32)
    out, state, bits = H.run(t, s0, 0.1)
    assert bits == dsa.DSA_DEVICE_CAPACITY
    H.check(one, s0[:1], 0.1, out, state[:1])
    assert (state[2] == 77.0).all() and (state[4] == 77.0).all()
