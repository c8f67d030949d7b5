"""Attention over the 4-bit cache with values far apart, against the definition in 64 bits: cleared places
before others, groups of columns and positions of very different sizes, the ends of the types' ranges."""
import math

import pytest

import kv4_harness as H

pytestmark = pytest.mark.gpu


def _scale_places(t, factors):
    """Multiplies V's scales at position x of request b by factors[b][x] (powers of two or 0)."""
    import torch
    vs = H.parts(t["pages"], t["dk"], t["dv"], t["ps"])[3]
    f = torch.ones(vs.shape[0], t["ps"], dtype=torch.float64)
    for b, fb in enumerate(factors):
        x = torch.arange(len(fb))
        f[t["table"][b, x // t["ps"]].long(), x % t["ps"]] = torch.as_tensor(fb, dtype=torch.float64)
    vs.copy_((vs.double() * f[:, None, None, :]).bfloat16())


def _cleared(L, where, before, after):
    """Factors of L positions: `before` at the first ones or in blocks of two stages out of three, else `after`."""
    import torch
    x = torch.arange(L)
    first = (x // 128) % 3 != 2 if where == "blocks" else x < where
    return torch.where(first, torch.tensor(before, dtype=torch.float64), torch.tensor(after, dtype=torch.float64))


def _rows(t, keep):
    """The problem's rows `keep` (ascending) alone."""
    ro = t["row_offsets"].tolist()
    n = [sum(1 for r in keep if a <= r < b) for a, b in zip(ro, ro[1:])]
    return dict(t, q=t["q"][keep], row_len=t["row_len"][keep], row_offsets=H.prefix(n))


@pytest.mark.parametrize("after", [1.0, 2.0 ** 4, 2.0 ** 10, 2.0 ** 80])
@pytest.mark.parametrize("where", [32, 128, 300, "blocks"])
@pytest.mark.parametrize("rows,lens,heads,ps", [
    ([1] * 24, [900] * 24, (32, 16), 64),                   # items of several stages, each taken whole
    ([1], [40000], (16, 8), 16),                            # one request cut into the CTAs' shares
    ([2, 1] * 14, [700, 1100] * 14, (64, 16), 128),         # a few rows each
    ([4, 1, 3] * 8, [1200, 400, 600] * 8, (32, 16), 32),
])
def test_cleared_places_come_first(rows, lens, heads, ps, where, after):
    # V of the first positions is zero (padded tokens, cleared places): what follows may have any scale.
    t = H.make(rows, lens, *heads, 64, 64, ps, seed=60)
    _scale_places(t, [_cleared(L, where, 0.0, after) for L in lens])
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)


@pytest.mark.parametrize("before,after", [(2.0 ** -122, 1.0), (2.0 ** -100, 2.0 ** 22), (2.0 ** -100, 2.0 ** 80), (2.0 ** -60, 2.0 ** 66)])
@pytest.mark.parametrize("rows,lens,dk,dv", [([1] * 24, [900] * 24, 64, 64), ([3, 1] * 10, [900, 1000] * 10, 192, 128)])
def test_tiny_places_come_first(rows, lens, dk, dv, before, after):
    t = H.make(rows, lens, 32, 16, dk, dv, 64, seed=61)
    _scale_places(t, [_cleared(L, 200, before, after) for L in lens])
    out, lse, bits = H.run(t, 0.1)
    assert bits == 0
    H.check(t, 0.1, out, lse)


@pytest.mark.parametrize("rows_max", [1, 100, 600])
@pytest.mark.parametrize("after", [2.0 ** 4, 2.0 ** 80])
def test_cleared_places_whatever_the_kernel(rows_max, after):
    # Few rows at a time, widened by the way, widened first.
    t = H.make([600], [900], 16, 2, 128, 128, 32, seed=62)
    _scale_places(t, [_cleared(900, 300, 0.0, after)])
    out, lse, bits = H.run(t, 0.09, rows_max=rows_max)
    assert bits == 0
    keep = [0, 1, 130, 255, 256, 400, 599]
    H.check(_rows(t, keep), 0.09, out[keep], lse[keep])


def test_nothing_but_cleared_places():
    t = H.make([1, 3], [700, 200], 8, 2, 128, 128, 64, seed=63)
    _scale_places(t, [[0.0] * 700, [0.0] * 200])
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0 and not out.any()
    H.check(t, 0.09, out, lse)


@pytest.mark.parametrize("small", [0, 1])
@pytest.mark.parametrize("e", [10, 20, 24, 32, 60])
@pytest.mark.parametrize("rows,lens", [([1], [700]), ([1], [5000]), ([4, 2], [300, 900]), ([100], [300])])
def test_one_group_of_columns_far_below_the_other(rows, lens, e, small):
    # (columns of V often differ in size for good; the bound takes each group's own largest scale)
    t = H.make(rows, lens, 8, 2, 128, 128, 64, seed=64 + e)
    vs = H.parts(t["pages"], 128, 128, 64)[3]
    vs[:, :, small] = (vs[:, :, small].float() * 2.0 ** -e).bfloat16()
    out, lse, bits = H.run(t, 0.09)
    assert bits == 0
    H.check(t, 0.09, out, lse)
    ref, _, bound, _ = H.reference(t, 0.09)
    assert (ref.abs() > bound)[..., 64 * small:64 * small + 64].float().mean() > 0.5   # (the bound tells a lost group)


@pytest.mark.parametrize("at", [0, 200])
@pytest.mark.parametrize("e", [8, 20])
def test_one_position_far_above_the_others(e, at):
    import torch
    # What the header states: sums over 16 positions are cut 2^-14 of the largest weight times scale in them below, each of
    # their 17 addends.
    t = H.make([1, 3], [900, 300], 8, 2, 128, 128, 32, seed=65)
    _scale_places(t, [[2.0 ** e if x == at else 1.0 for x in range(L)] for L in (900, 300)])
    out, lse, bits = H.run(t, 0.09)
    ref, _, bound, _ = H.reference(t, 0.09)
    most = torch.zeros_like(ref)
    _, _, ks, vs = H.parts(t["pages"], 128, 128, 32)
    K, _ = H.values(t["pages"], 128, 128, 32)
    for r, (b, n) in enumerate(zip([0, 1, 1, 1], t["row_len"].tolist())):
        x = torch.arange(n)
        page = t["table"][b, x // 32].long()
        k = K[page, x % 32].repeat_interleave(4, dim=1)
        s = vs.double()[page, :, :, x % 32].repeat_interleave(4, dim=1)                     # [n, heads, groups]
        w = torch.softmax(torch.einsum("hd,nhd->nh", t["q"][r].double(), k) * 0.09, dim=0)
        most[r] = (w[..., None] * s).amax(dim=0).repeat_interleave(64, dim=1)
    assert bits == 0 and bool(((out.double() - ref).abs() <= bound + 17 * 2.0 ** -14 * most).all())


@pytest.mark.parametrize("rows", [1, 150, 600])
def test_fp16_keys_and_values_of_tiny_scales(rows, monkeypatch):
    # The kernels in tiles take K and V as dsa_kv4_read gives them in fp16, rounded once; the other one takes them as they are.
    import torch
    t = H.make([rows], [700], 16, 2, 64, 64, 64, "fp16", seed=67)
    _, _, ks, _ = H.parts(t["pages"], 64, 64, 64)
    ks.copy_((ks.float() * 2.0 ** -21).bfloat16())             # scales of about 2^-22.5
    t["q"] = (t["q"].float() * 2.0 ** 11).half()
    if rows > 1:
        plain = H.values
        monkeypatch.setattr(H, "values", lambda *a: [x.half().double() for x in plain(*a)])
    out, lse, bits = H.run(t, 2.0 ** 7)
    keep = [r for r in (0, 1, 70, 149, 300, 599) if r < rows]
    assert bits == 0
    H.check(_rows(t, keep), 2.0 ** 7, out[keep], lse[keep])


@pytest.mark.parametrize("rows", [1, 150, 600])
def test_fp16_output_of_tiny_values(rows):
    # All codes 15 and one scale, 1.125 * 2^-22: 31.5 steps of fp16's subnormals, 32 as the values are rounded once.
    import torch
    t = H.make([rows], [700], 16, 2, 64, 64, 64, "fp16", seed=68)
    _, vc, _, vs = H.parts(t["pages"], 64, 64, 64)
    vc.fill_(0xFF)
    vs.fill_(1.125 * 2.0 ** -22)
    out, _, bits = H.run(t, 0.125)
    assert bits == 0 and bool(((out.double() / 2.0 ** -24 - 31.5).abs() <= 1.0).all())


def test_one_batch_in_two_calls():
    # Single tokens and a long chunk, as the header advises: the tokens' call ends behind their rows, the chunk's leaves them alone.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    rows, lens, T = [1, 1, 0, 1, 400], [700, 30, 5, 1500, 900], 3
    t = H.make(rows, lens, 16, 2, 128, 128, 64, seed=77)
    prob = H.problem(t, 0.09)
    q, ro, rl = (prob._keep[x] for x in ("q", "row_offsets", "row_len"))
    out = torch.full((403, 16, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    calls = (dict(q=q[:T], row_offsets=ro.clamp(max=T), row_len=rl[:T]),
             dict(q=q, row_offsets=ro.clamp(min=T), row_len=rl, L_max=900))
    for part, kw in zip((out[:T], out), calls):
        p = dsa.KV4Problem.from_tensors(cache=prob._keep_cache, softmax_scale=0.09, **kw)
        ws = dsa.alloc_kv4_workspace(p)
        before = out.clone()
        dsa.dsa_kv4_attn(p, part, None, ws)
        # (the chunk's L_max is below a token's length: rows outside row_offsets are not looked at)
        assert dsa.dsa_read_device_status(ws) == 0
    assert out[:T].equal(before[:T])
    keep = [0, 1, 2, 3, 130, 258, 402]
    H.check(_rows(t, keep), 0.09, out.cpu()[keep], None)


def test_no_copy_where_few_rows_are_declared():
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([600], [900], 16, 2, 128, 128, 32, seed=78)
    sizes = [dsa.dsa_kv4_workspace_size(H.problem(t, 0.09, rows_max=n)) for n in (600, 2304 // 8 - 1)]
    assert sizes[0] >= 900 * 2 * 256 * 2 and sizes[1] < sizes[0] - 900 * 2 * 256 * 2 // 2


@pytest.mark.parametrize("rows", [1, 200, 600])
@pytest.mark.parametrize("L_max", [0, 300])
def test_rows_that_see_nothing_at_all(rows, L_max):
    t = H.make([rows, 1], [300, 40], 16, 2, 64, 64, 16, seed=79, row_len=[0] * (rows + 1))
    t["table"][:] = -1
    out, lse, bits = H.run(t, 0.1, L_max=L_max)
    assert bits == 0 and not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("e", [-100, -60])
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_small_values_are_kept(rows, e):
    # The harness allows 1e-30 beside what its bound is made of, more than all of these outputs; here it is taken off again.
    # bf16's subnormals end at 2^-133: half a step of them, and of fp32's sums, is 2^-133 together.
    t = H.make([rows], [700], 4, 2, 64, 64, 64, seed=66)
    vs = H.parts(t["pages"], 64, 64, 64)[3]
    vs.copy_((vs.float() * 2.0 ** e).bfloat16())
    out, _, bits = H.run(t, 0.125)
    ref, _, bound, _ = H.reference(t, 0.125)
    bound = bound - 1e-30 + 2.0 ** -133
    assert bits == 0 and bool(((out.double() - ref).abs() <= bound).all())
    assert bool((ref.abs() > bound).any(dim=-1).all())     # (zeros would not do)
