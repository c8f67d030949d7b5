"""Norms and rotation, the 4-bit cache written and read back on the GPU (dsa_qk_norm_rope,
dsa_kv4_append, dsa_kv4_read), against the definitions in 64 bits: what goes into the cache has to
be the same bytes."""
import math

import pytest

import kv4_harness as H

pytestmark = pytest.mark.gpu


def _fused(T, sizes, dt, g, pad=8):
    """Views [T, heads, width] of one projection with a few columns around them."""
    import torch
    x = torch.randn(T, sum(h * d for h, d in sizes) + 2 * pad, generator=g).to(dt).cuda()
    out, at = [], pad
    for h, d in sizes:
        out.append(x[:, at:at + h * d].unflatten(1, (h, d)))
        at += h * d
    return out


TURNS = [
    dict(D=64, rot=64, first=0, adjacent=False, norm="qk"),
    dict(D=128, rot=128, first=0, adjacent=False, norm="qk"),
    dict(D=128, rot=64, first=0, adjacent=True, norm="k"),
    dict(D=128, rot=32, first=20, adjacent=False, norm="q"),
    dict(D=192, rot=64, first=128, adjacent=True, norm=""),
    dict(D=192, rot=8, first=4, adjacent=False, norm="qk"),
    dict(D=256, rot=256, first=0, adjacent=False, norm="qk"),
    dict(D=256, rot=0, first=0, adjacent=False, norm="qk"),
    dict(D=64, rot=0, first=0, adjacent=False, norm=""),
]


@pytest.mark.parametrize("c", TURNS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,hq,hkv,strided", [(1, 1, 1, False), (5, 64, 8, True), (77, 3, 3, False), (3, 128, 128, False), (700, 4, 1, True)])
def test_norm_and_rotation(c, dt, T, hq, hkv, strided):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(T + c["D"])
    D, ty = c["D"], H.dtype(dt)
    if strided:
        q, k = _fused(T, [(hq, D), (hkv, D)], ty, g)
    else:
        q, k = (torch.randn(T, h, D, generator=g).to(ty).cuda() for h in (hq, hkv))
    pos = torch.randint(0, 1 << 20, (T,), generator=g).int()
    pos[0] = 0
    weight = {x: (1 + 0.3 * torch.randn(D, generator=g)).to(ty) if x in c["norm"] else None for x in "qk"}
    freq = H.inv_freq(c["rot"]) if c["rot"] else None
    prob = dsa.QKProblem.from_tensors(
        q=q, k=k, positions=pos.cuda(), inv_freq=None if freq is None else freq.cuda(), rot_first=c["first"],
        interleaved=c["adjacent"], eps=1e-6, **{x + "_weight": None if w is None else w.cuda() for x, w in weight.items()})
    qo, ko = (torch.full(x.shape, 77.0, dtype=ty, device="cuda") for x in (q, k))
    dsa.dsa_qk_norm_rope(prob, qo, ko)
    for name, x, got in (("q", q, qo), ("k", k, ko)):
        y, size = H.turned(x.cpu(), weight[name], pos, freq, c["first"], c["adjacent"])
        err = (got.cpu().double() - y).abs()
        assert bool((err <= H.turned_bound(y, size, ty)).all()), (err / H.turned_bound(y, size, ty)).max()
    # in place, with the inputs' strides, it gives the same
    dsa.dsa_qk_norm_rope(prob, q, k)
    assert q.equal(qo) and k.equal(ko)


def test_one_of_the_two_and_skipped_rows():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 4, 128, generator=g).bfloat16()
    pos = H.ints([3, -1, 0, -2147483648, 2147483647, 9])
    freq = H.inv_freq(128)
    for name in "qk":
        prob = dsa.QKProblem.from_tensors(positions=pos.cuda(), inv_freq=freq.cuda(), **{name: x.cuda()})
        out = torch.full_like(x, 77.0, device="cuda")
        dsa.dsa_qk_norm_rope(prob, *((out, None) if name == "q" else (None, out)))
        y, size = H.turned(x, None, pos, freq)
        live = pos >= 0
        assert (out.cpu()[~live] == 77).all()
        assert bool(((out.cpu().double() - y).abs() <= H.turned_bound(y, size, torch.bfloat16))[live].all())


def test_heads_that_are_not_finite_stay_alone():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    x = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    x[1, 3, 7] = float("nan")
    x[2, 0, 60] = float("inf")
    w = torch.ones(64).bfloat16()
    prob = dsa.QKProblem.from_tensors(q=x.cuda(), positions=H.ints([1, 2, 3]).cuda(), inv_freq=H.inv_freq(64).cuda(), q_weight=w.cuda())
    out = torch.empty_like(x, device="cuda")
    dsa.dsa_qk_norm_rope(prob, out, None)
    bad = ~out.cpu().isfinite().all(dim=2)
    assert bad[1, 3] and bad[2, 0] and bad.sum() == 2


# ------------------------------------------------------------------------------- the cache

def _append(rows, starts, hq, hkv, dk, dv, ps, dt="bf16", rot=None, first=0, adjacent=False, norm=True, seed=0, fused=True,
            x=None, skip=()):
    """Appends rows and returns (pool before, pool after, what the pool has to be, q, q_out, bits)."""
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(seed)
    ty, T = H.dtype(dt), sum(rows)
    rot = dk if rot is None else rot
    sizes = [(hkv, dk), (hkv, dv)]
    k, v = _fused(T, sizes, ty, g) if fused else [torch.randn(T, h, d, generator=g).to(ty).cuda() for h, d in sizes]
    if x is not None:
        k, v = (y.to(ty).cuda() for y in x)
    q = torch.randn(T, hq, dk, generator=g).to(ty).cuda() if hq else None
    kw, qw = ((1 + 0.3 * torch.randn(dk, generator=g)).to(ty) if norm else None for _ in range(2))
    freq = H.inv_freq(rot) if rot else None
    pos = torch.tensor([s + i for n, s in zip(rows, starts) for i in range(n)], dtype=torch.int32)
    for r in skip:
        pos[r] = -1
    need = [-(-(n + s) // ps) for n, s in zip(rows, starts)]
    n = sum(need) + 2
    pool = torch.randint(0, 256, (n, hkv, H.block_bytes(dk, dv, ps)), dtype=torch.uint8, generator=g)
    order = torch.randperm(n, generator=g).int()
    table = torch.full((len(rows), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    cache = dsa.KV4Cache.from_tensors(pages=pool.cuda(), table=table.cuda(), page_size=ps, D_k=dk, D_v=dv)
    ro = H.prefix(rows)
    prob = dsa.QKProblem.from_tensors(
        q=q, k=k, v=v, positions=pos.cuda(), inv_freq=None if freq is None else freq.cuda(), rot_first=first,
        interleaved=adjacent, q_weight=None if qw is None or q is None else qw.cuda(), k_weight=None if kw is None else kw.cuda(),
        eps=1e-5, row_offsets=ro.cuda())
    q_out = torch.full_like(q, 77.0) if hq else None
    ws = dsa.alloc_kv4_workspace()
    dsa.dsa_kv4_append(cache, prob, q_out, ws)
    bits = dsa.dsa_read_device_status(ws)
    want = pool.clone()
    yk, _ = H.turned(k.cpu(), kw, pos, freq, first, adjacent, 1e-5)
    r = 0
    for b, m in enumerate(rows):
        for _ in range(m):
            p = int(pos[r])
            if p >= 0 and 0 <= int(table[b, p // ps]) < n:
                H.put(want, int(table[b, p // ps]), p % ps, yk[r], v[r].cpu().double(), dk, dv, ps)
            r += 1
    return dict(cache=cache, before=pool, want=want, q=q, q_out=q_out, qw=qw, pos=pos, freq=freq, bits=bits, ro=ro, prob=prob,
                k=k, v=v, ws=ws, table=table)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,starts,hq,hkv,ps", [
    ([1], [0], 0, 1, 16),
    ([1, 1, 0, 1], [130, 63, 0, 4095], 8, 2, 64),           # a decode step
    ([40, 3, 129], [0, 17, 31], 3, 3, 32),                  # prompts and chunks over page borders
    ([65], [100], 64, 8, 128),
])
def test_append_writes_the_definitions_bytes(dk, dv, dt, rows, starts, hq, hkv, ps):
    import torch
    a = _append(rows, starts, hq, hkv, dk, dv, ps, dt, seed=dk + ps)
    assert a["bits"] == 0
    assert a["cache"]._keep["pages"].cpu().equal(a["want"])
    if hq:
        y, size = H.turned(a["q"].cpu(), a["qw"], a["pos"], a["freq"], eps=1e-5)
        assert bool(((a["q_out"].cpu().double() - y).abs() <= H.turned_bound(y, size, H.dtype(dt))).all())


@pytest.mark.parametrize("c", [dict(rot=64, first=128, adjacent=True, norm=False), dict(rot=0, norm=True), dict(rot=0, norm=False),
                               dict(rot=32, first=12, adjacent=False, norm=True)])
def test_append_of_other_turns(c):
    a = _append([33, 5], [7, 2000], 2, 2, 192, 128, 16, seed=3, **c)
    assert a["bits"] == 0 and a["cache"]._keep["pages"].cpu().equal(a["want"])


def test_borders_fall_where_exact_arithmetic_puts_them():
    # 130000 heads' groups: some hundred values lie nearer to a border than fp32 can tell.
    a = _append([8200], [0], 0, 8, 128, 128, 64, seed=5)
    got = a["cache"]._keep["pages"].cpu()
    assert a["bits"] == 0 and got.equal(a["want"])


@pytest.mark.parametrize("c", [dict(), dict(rot=64), dict(rot=0), dict(adjacent=True), dict(norm=False)])
def test_keys_with_columns_far_above_the_others(c):
    # (a few columns 30 to 3000 times the others, a group of zeros, heads of zeros)
    import torch
    g = torch.Generator().manual_seed(21)
    k, v = torch.randn(1500, 4, 128, generator=g), torch.randn(1500, 4, 128, generator=g)
    k[:, 0, 5] *= 30
    k[:, 1, 70] *= 300
    k[:, 2, 100] *= 3000
    k[:, 3, 64:] = 0
    k[::3, 3] = 0
    a = _append([1500], [0], 0, 4, 128, 128, 64, seed=22, x=(k, v), **c)
    assert a["bits"] == 0 and a["cache"]._keep["pages"].cpu().equal(a["want"])


def test_values_that_need_no_turn_are_exact_ties_included():
    # Halves of a scale: ties go to the even code.  Zeros, one value alone, tiny and huge groups.
    import torch
    base = torch.tensor([7.0, -7.0, 0.5, 1.5, 2.5, -0.5, -3.5, 6.5] + [0.25 * i for i in range(-28, 28)])
    x = torch.stack([base * 2.0 ** e for e in (0, -20, 40, 100, -100, -125)] + [torch.zeros(64)] +
                    [torch.eye(64)[i] * 3.7 for i in (0, 1, 63)] + [base * f for f in (1.0625, 1.09375, 1.03125, 1.15625)])
    x = x.bfloat16()[:, None].repeat(1, 2, 1)
    a = _append([x.shape[0]], [5], 0, 2, 64, 64, 16, rot=0, norm=False, x=(x, x.flip(2)))
    assert a["bits"] == 0 and a["cache"]._keep["pages"].cpu().equal(a["want"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_group_that_is_not_finite(bad):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(4, 2, 128, generator=g).bfloat16() for _ in range(2))
    k[1, 0, 70], v[2, 1, 3] = bad, bad
    a = _append([4], [0], 0, 2, 128, 128, 16, rot=0, norm=False, x=(k, v))
    ko, vo = (torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dsa.dsa_kv4_read(a["cache"], a["ro"].cuda(), a["pos"].cuda(), ko, vo, a["ws"])
    lost_k, lost_v = ~ko.cpu().isfinite(), ~vo.cpu().isfinite()
    assert lost_k[1, 0, 64:].all() and lost_k.sum() == 64 and lost_v[2, 1, :64].all() and lost_v.sum() == 64


def test_skipped_rows_and_bad_places():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    a = _append([5, 3], [10, 60], 4, 2, 64, 64, 16, seed=9, skip=(1, 6))
    assert a["bits"] == 0 and a["cache"]._keep["pages"].cpu().equal(a["want"])
    assert (a["q_out"][[1, 6]] == 77).all() and not (a["q_out"][[0, 2, 3, 4, 5, 7]] == 77).any()
    # positions past the table, pages outside the pool
    a["cache"]._keep["pages"].copy_(a["before"])
    pos, table = a["pos"].clone(), a["table"].clone()
    pos[0] = 16 * table.shape[1]
    pos[2] = 2147483647
    table[1, 3] = a["before"].shape[0]
    table[1, 4 if table.shape[1] > 4 else 3] = -7
    prob = a["prob"].set(positions=pos.cuda())
    cache = dsa.KV4Cache.from_tensors(pages=a["cache"]._keep["pages"], table=table.cuda(), page_size=16, D_k=64, D_v=64)
    dsa.dsa_kv4_append(cache, prob, a["q_out"], a["ws"])
    assert dsa.dsa_read_device_status(a["ws"]) & dsa.DSA_DEVICE_BAD_INDEX
    got = cache._keep["pages"].cpu()
    changed = (got != a["before"]).flatten(1).any(dim=1).nonzero().flatten().tolist()
    assert set(changed) <= {int(table[0, 0])}                # rows 3 and 4 of the first request alone
    ko = torch.full((8, 2, 64), 55.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_kv4_read(cache, a["ro"].cuda(), pos.cuda(), ko, None, a["ws"])
    assert dsa.dsa_read_device_status(a["ws"]) & dsa.DSA_DEVICE_BAD_INDEX
    assert (ko[[0, 1, 2, 6]] == 55).all() and not (ko[[3, 4]] == 55).any()


@pytest.mark.parametrize("rows", [[1], [200, 0, 56], [1] * 300, [257, 255], [300, 213], [1] * 600])
def test_status_is_each_calls_own(rows):
    # (up to 512 rows the call's kernel sets the status, above a launch before clears it)
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    T = sum(rows)
    a = _append(rows, [3] * len(rows), 1, 1, 64, 64, 16, seed=11)
    assert a["bits"] == 0
    ko = torch.empty(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    for at in sorted({0, T // 2, T - 1}):
        pos = a["pos"].clone()
        for value, bits in ((16 * a["table"].shape[1], dsa.DSA_DEVICE_BAD_INDEX), (-1, 0)):
            pos[at] = value
            for call in ("append", "read"):
                a["ws"].fill_(-1 if a["ws"].dtype != torch.uint8 else 255)
                if call == "append":
                    dsa.dsa_kv4_append(a["cache"], a["prob"].set(positions=pos.cuda()), a["q_out"], a["ws"])
                else:
                    dsa.dsa_kv4_read(a["cache"], a["ro"].cuda(), pos.cuda(), ko, None, a["ws"])
                assert dsa.dsa_read_device_status(a["ws"]) == bits, (call, at, value)


def test_rows_outside_the_requests():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    a = _append([6, 4], [0, 3], 2, 1, 64, 64, 16, seed=10)
    a["cache"]._keep["pages"].copy_(a["before"])
    ro = H.ints([2, 5, 8]).cuda()
    prob = a["prob"].set(row_offsets=ro)
    a["q_out"].fill_(77)
    dsa.dsa_kv4_append(a["cache"], prob, a["q_out"], a["ws"])
    assert dsa.dsa_read_device_status(a["ws"]) == 0
    assert (a["q_out"][[0, 1, 8, 9]] == 77).all() and not (a["q_out"][2:8] == 77).all(dim=2).any()
    ko = torch.full((10, 1, 64), 55.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_kv4_read(a["cache"], ro, a["pos"].cuda(), ko, None, a["ws"])
    assert (ko[[0, 1, 8, 9]] == 55).all() and not (ko[2:8] == 55).all(dim=2).any()


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("dt,ps", [("bf16", 16), ("fp16", 64), ("bf16", 128)])
def test_read_is_exact(dk, dv, dt, ps):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    lens, ty = [3 * ps + 5, 1, 0, 2 * ps, 40], H.dtype(dt)
    t = H.make([0] * 5, lens, 3, 3, dk, dv, ps, dt, seed=ps)
    cache = dsa.KV4Cache.from_tensors(pages=t["pages"].cuda(), table=t["table"].cuda(), page_size=ps, D_k=dk, D_v=dv)
    rows = [lens[0], 1, 0, 7, 40]
    pos = torch.cat([torch.arange(lens[0]), torch.tensor([0]), torch.randint(0, lens[3], (7,)), torch.arange(40).flip(0)]).int()
    ko = torch.full((sum(rows), 3, dk), 55.0, dtype=ty, device="cuda")
    vo = torch.full((sum(rows), 3, dv), 55.0, dtype=ty, device="cuda")
    ws = dsa.alloc_kv4_workspace()
    dsa.dsa_kv4_read(cache, H.prefix(rows).cuda(), pos.cuda(), ko, vo, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    K, V = H.values(t["pages"], dk, dv, ps)
    b = torch.repeat_interleave(torch.arange(5), torch.tensor(rows))
    page = t["table"][b, pos.long() // ps].long()
    assert ko.cpu().equal(K[page, pos.long() % ps].to(ty)) and vo.cpu().equal(V[page, pos.long() % ps].to(ty))


def test_read_into_a_view_and_one_of_the_two():
    # Outputs that begin 16 bytes off a multiple of 32.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    t = H.make([0], [70], 2, 2, 128, 128, 32, seed=6)
    cache = dsa.KV4Cache.from_tensors(pages=t["pages"].cuda(), table=t["table"].cuda(), page_size=32, D_k=128, D_v=128)
    flat = torch.full((8 + 70 * 256 + 8,), 55.0, dtype=torch.bfloat16, device="cuda")
    vo = flat[8:-8].view(70, 2, 128)
    pos, ro, ws = torch.arange(70, dtype=torch.int32), H.prefix([70]).cuda(), dsa.alloc_kv4_workspace()
    dsa.dsa_kv4_read(cache, ro, pos.cuda(), None, vo, ws)
    _, V = H.values(t["pages"], 128, 128, 32)
    assert vo.cpu().double().equal(V[t["table"][0, pos.long() // 32].long(), pos.long() % 32])
    assert (flat[:8] == 55).all() and (flat[-8:] == 55).all()


@pytest.mark.parametrize("e", [-124, -60, 0, 60, 119, 123])
def test_read_of_all_magnitudes(e):
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(7)
    x = (torch.rand(9, 2, 128, generator=g, dtype=torch.float64) * 2 - 1).mul(2.0 ** e * 14).bfloat16()
    a = _append([9], [0], 0, 2, 128, 128, 16, rot=0, norm=False, x=(x, x.flip(2)))
    ko, vo = (torch.zeros(9, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dsa.dsa_kv4_read(a["cache"], a["ro"].cuda(), a["pos"].cuda(), ko, vo, a["ws"])
    assert ko.cpu().double().equal(H.held(x)) and vo.cpu().double().equal(H.held(x.flip(2)))


def test_pool_beyond_32_bits():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    n = (1 << 32) // (8 * H.block_bytes(128, 128, 128)) + 3
    pool = dsa.alloc_kv4_pages(n, 8, 128, 128, 128)
    table = torch.tensor([[n - 1, 1]], dtype=torch.int32, device="cuda")
    cache = dsa.KV4Cache.from_tensors(pages=pool, table=table, page_size=128, D_k=128, D_v=128)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(130, 8, 128, generator=g).bfloat16().cuda() for _ in range(2))
    pos, ro = torch.arange(130, dtype=torch.int32, device="cuda"), H.ints([0, 130], "cuda")
    prob = dsa.QKProblem.from_tensors(k=k, v=v, positions=pos, row_offsets=ro)
    ws = dsa.alloc_kv4_workspace()
    dsa.dsa_kv4_append(cache, prob, None, ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    dsa.dsa_kv4_read(cache, ro, pos, ko, vo, ws)
    assert ko.cpu().double().equal(H.held(k.cpu())) and vo.cpu().double().equal(H.held(v.cpu()))


def test_captured_and_on_another_stream():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    a = _append([2, 1, 30], [5, 100, 0], 4, 2, 128, 128, 64, seed=12)
    want = a["cache"]._keep["pages"].clone()
    q_want = a["q_out"].clone()
    s = torch.cuda.Stream()
    ko, vo = (torch.zeros(33, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ro, pos = a["ro"].cuda(), a["pos"].cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_kv4_append(a["cache"], a["prob"], a["q_out"], a["ws"])
        dsa.dsa_kv4_read(a["cache"], ro, pos, ko, vo, a["ws"])
    a["cache"]._keep["pages"].copy_(a["before"])
    a["q_out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert a["cache"]._keep["pages"].equal(want) and a["q_out"].equal(q_want)
    K, V = H.values(want.cpu(), 128, 128, 64)
    b = torch.repeat_interleave(torch.arange(3), torch.tensor([2, 1, 30]))
    page, at = a["table"][b, a["pos"].long() // 64].long(), a["pos"].long() % 64
    assert ko.cpu().double().equal(K[page, at]) and vo.cpu().double().equal(V[page, at])


# ------------------------------------------------------------------------------ together

def test_prompts_then_tokens():
    """A layer as a server runs it: prompts attended densely and appended, then tokens normed, rotated, appended and
    attended over the 4-bit cache; a prompt's second chunk over its first, taken back into 16 bits."""
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(30)
    hq, hkv, D, ps, scale = 8, 2, 128, 32, 1 / math.sqrt(128)
    lens, steps = [70, 33, 1], 3
    freq = H.inv_freq(D).cuda()
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2))
    table = torch.randperm(12, generator=g).int()[:12].reshape(3, 4).cuda()
    cache = dsa.KV4Cache.from_tensors(pages=dsa.alloc_kv4_pages(12, hkv, D, D, ps), table=table, page_size=ps, D_k=D, D_v=D)
    ws = dsa.alloc_kv4_workspace()
    T = sum(lens)
    q, k, v = _fused(T, [(hq, D), (hkv, D), (hkv, D)], torch.bfloat16, g)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    ro = H.prefix(lens).cuda()
    qk = dsa.QKProblem.from_tensors(q=q, k=k, v=v, positions=pos, inv_freq=freq, q_weight=qw, k_weight=kw, row_offsets=ro)
    qo, ko = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_qk_norm_rope(qk, qo, ko)
    q2 = torch.empty_like(qo)
    dsa.dsa_kv4_append(cache, qk, q2, ws)
    assert q2.equal(qo)                                    # the same queries either way
    # the prompt over itself: dense over what it appended, and over the pages
    kr, vr = torch.empty_like(ko), torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_kv4_read(cache, ro, pos, kr, vr, ws)
    dp = dsa.DenseProblem.from_tensors(q=qo, k=kr, v=vr, offsets=ro, row_offsets=ro, row_len=pos + 1, softmax_scale=scale)
    dense = torch.empty_like(qo)
    dsa.dsa_dense_attn(dp, dense, None, dsa.alloc_dense_workspace(dp))
    kp = dsa.KV4Problem.from_tensors(cache=cache, q=qo, row_offsets=ro, row_len=pos + 1, softmax_scale=scale)
    paged = torch.empty_like(qo)
    dsa.dsa_kv4_attn(kp, paged, None, dsa.alloc_kv4_workspace(kp))
    t = dict(pages=cache._keep["pages"].cpu(), table=table.cpu(), q=qo.cpu(), row_offsets=ro.cpu(), row_len=(pos + 1).cpu(),
             dk=D, dv=D, ps=ps)
    H.check(t, scale, paged.cpu(), None)
    H.check(t, scale, dense.cpu(), None)
    # 4 bits are near the 16: half a scale of a group's largest value / 7
    err = (kr.float() - ko.float()).unflatten(-1, (-1, 64)).abs().amax(-1)
    assert bool((err <= 1.01 * ko.float().unflatten(-1, (-1, 64)).abs().amax(-1) / 7 * 1.07 / 2 + 2.0 ** -8).all())
    one = H.ints([0, 1, 2, 3], "cuda")
    for s in range(steps):
        q, k, v = _fused(3, [(hq, D), (hkv, D), (hkv, D)], torch.bfloat16, g)
        at = torch.tensor([n + s for n in lens], dtype=torch.int32, device="cuda")
        qk = dsa.QKProblem.from_tensors(q=q, k=k, v=v, positions=at, inv_freq=freq, q_weight=qw, k_weight=kw, row_offsets=one)
        qo = torch.empty(3, hq, D, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_kv4_append(cache, qk, qo, ws)
        kp = dsa.KV4Problem.from_tensors(cache=cache, q=qo, row_offsets=one, row_len=at + 1, softmax_scale=scale)
        out, lse = torch.empty_like(qo), torch.empty(3, hq, device="cuda")
        aws = dsa.alloc_kv4_workspace(kp)
        dsa.dsa_kv4_attn(kp, out, lse, aws)
        assert dsa.dsa_read_device_status(aws) == 0 and dsa.dsa_read_device_status(ws) == 0
        t = dict(t, pages=cache._keep["pages"].cpu(), q=qo.cpu(), row_offsets=one.cpu(), row_len=(at + 1).cpu())
        H.check(t, scale, out.cpu(), lse.cpu())
