"""The 4-bit cache's writer and reader at the ends of their ranges (dsa_kv4_append, dsa_kv4_read)."""
import math

import pytest

import kv4_harness as H
from test_gpu_kv4_cache import _append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(64, 64), (192, 128)])
def test_fp16_values_are_rounded_once(dk, dv):
    # Every scale from 2^-44 to the largest whose sevenfold fp16 holds, with every code.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    ps, hkv = 64, 2
    scales = torch.tensor([m * 2.0 ** (e - 3) for e in range(-44, 14) for m in range(8, 16)], dtype=torch.float64)
    scales = torch.cat([scales[scales * 7 <= 65504], torch.zeros(1, dtype=torch.float64)])
    n = -(-len(scales) // ps)
    t = H.make([0], [n * ps], hkv, hkv, dk, dv, ps, "fp16", seed=70, spare=0)
    g = torch.Generator().manual_seed(71)
    kc, vc, ks, vs = H.parts(t["pages"], dk, dv, ps)
    at = torch.arange(n * ps) % len(scales)
    for codes, s in ((kc, ks), (vc, vs)):
        lo, hi = (torch.randint(1, 16, codes.shape, generator=g, dtype=torch.uint8) for _ in range(2))
        codes.copy_(lo | hi << 4)
        s.copy_(scales[at].reshape(n, 1, 1, ps).bfloat16().expand(s.shape))
    kc[..., :8] = torch.tensor([0x21, 0x43, 0x65, 0x87, 0xA9, 0xCB, 0xED, 0x1F], dtype=torch.uint8)
    cache = dsa.KV4Cache.from_tensors(pages=t["pages"].cuda(), table=t["table"].cuda(), page_size=ps, D_k=dk, D_v=dv)
    pos = torch.arange(n * ps, dtype=torch.int32)
    ko = torch.zeros(n * ps, hkv, dk, dtype=torch.float16, device="cuda")
    vo = torch.zeros(n * ps, hkv, dv, dtype=torch.float16, device="cuda")
    ws = dsa.alloc_kv4_workspace()
    dsa.dsa_kv4_read(cache, H.prefix([n * ps]).cuda(), pos.cuda(), ko, vo, ws)
    assert dsa.dsa_read_device_status(ws) == 0
    K, V = H.values(t["pages"], dk, dv, ps)
    page = t["table"][0, pos.long() // ps].long()
    for got, want in ((ko, K), (vo, V)):
        want = want[page, pos.long() % ps].half()        # (eight significant bits: one rounding)
        assert bool(want.isfinite().all()) and got.cpu().equal(want)


def test_fp16_appended_and_read_back_in_the_smallest_steps():
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(72)
    x = (torch.randint(-40, 41, (64, 2, 64), generator=g).double() * 2.0 ** -24).half()
    x[:, :, 0] = 5 * 2.0 ** -24
    a = _append([64], [0], 0, 2, 64, 64, 16, "fp16", rot=0, norm=False, x=(x, x.flip(2)))
    assert a["cache"]._keep["pages"].cpu().equal(a["want"])
    ko, vo = (torch.zeros(64, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    dsa.dsa_kv4_read(a["cache"], a["ro"].cuda(), a["pos"].cuda(), ko, vo, a["ws"])
    assert ko.cpu().equal(H.held(x).half()) and vo.cpu().equal(H.held(x.flip(2)).half())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("c", [dict(), dict(adjacent=True)])
def test_neighbours_of_a_group_that_is_not_finite(bad, c):
    # The head's other group is rotated: its borders fall where exact arithmetic puts them all the same.
    import torch
    g = torch.Generator().manual_seed(73)
    k, v = (torch.randn(8200, 8, 128, generator=g).bfloat16() for _ in range(2))
    k[:, :, 100] = bad
    a = _append([8200], [0], 0, 8, 128, 128, 64, rot=64, norm=False, x=(k, v), **c)
    assert a["bits"] == 0
    page, at = a["table"][0, a["pos"].long() // 64].long(), a["pos"].long() % 64
    got, want = (H.parts(x, 128, 128, 64) for x in (a["cache"]._keep["pages"].cpu(), a["want"]))
    for i in (0, 2):                                     # codes and scales of K's first group
        assert bool((got[i][page, :, 0, at] == want[i][page, :, 0, at]).all())
    for i in (1, 3):
        assert got[i][page, :, :, at].equal(want[i][page, :, :, at])
    assert bool(got[2][page, :, 1, at].isnan().all())


def test_border_of_the_smallest_scale():
    # One rotated pair to a key, its larger column next to 7 * 31 / 32 * 2^-126, where a scale of 2^-126 begins: those within
    # 2^-22 of it out of forty million, on either side.
    import numpy as np
    import torch
    rng = np.random.default_rng(74)
    border, keep = 7 * 31 / 32 * 2.0 ** -126, []
    for _ in range(20):
        u, v = (torch.from_numpy(rng.uniform(-1, 1, 2_000_000) * 2.0 ** -123).bfloat16() for _ in range(2))
        pos = rng.integers(0, 1 << 15, 2_000_000)
        a, b = u.double().numpy(), v.double().numpy()
        c, s = np.cos(pos.astype(np.float64)), np.sin(pos.astype(np.float64))
        top = np.maximum(np.abs(a * c - b * s), np.abs(b * c + a * s))
        at = np.nonzero(np.abs(top / border - 1) < 2.0 ** -22)[0]
        keep += [(u[i].item(), v[i].item(), int(pos[i])) for i in at]
    n = len(keep)
    assert n >= 20
    k = torch.zeros(n, 1, 64, dtype=torch.bfloat16)
    k[:, 0, 0], k[:, 0, 32] = (torch.tensor([x[i] for x in keep]).bfloat16() for i in (0, 1))
    # (each key at its own position: a request to a key)
    a = _append([1] * n, [x[2] for x in keep], 0, 1, 64, 64, 128, norm=False, x=(k, k))
    assert a["bits"] == 0 and a["cache"]._keep["pages"].cpu().equal(a["want"])


@pytest.mark.parametrize("e,eps", [(-50, 0.0), (-40, 2.0 ** -90), (59, 0.0), (59, 1e-6)])
def test_ends_of_the_norms_range(e, eps):
    # Keys whose mean square is 2^-100 or 2^118: the bytes are exact arithmetic's there too, and the rotated rows within
    # their bound.
    import torch
    import dsa_sparse_attention_03_gb300 as dsa
    g = torch.Generator().manual_seed(75)
    k, v = torch.randn(600, 4, 128, generator=g), torch.randn(600, 4, 128, generator=g)
    k *= 2.0 ** e / (k * k).mean(dim=-1, keepdim=True).sqrt() * 1.01
    a = _append([600], [100], 0, 4, 128, 128, 64, x=(k, v), seed=76)
    a["cache"]._keep["pages"].copy_(a["before"])
    prob = a["prob"].set(eps=eps)
    dsa.dsa_kv4_append(a["cache"], prob, None, a["ws"])
    weight = prob._keep["k_weight"].cpu()
    y, size = H.turned(a["k"].cpu(), weight, a["pos"], a["freq"], eps=eps)
    want = a["before"].clone()
    for r, p in enumerate(a["pos"].tolist()):
        H.put(want, int(a["table"][0, p // 64]), p % 64, y[r], a["v"][r].cpu().double(), 128, 128, 64)
    assert dsa.dsa_read_device_status(a["ws"]) == 0 and a["cache"]._keep["pages"].cpu().equal(want)
    out = torch.zeros(600, 4, 128, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_qk_norm_rope(prob, None, out)
    assert bool(((out.cpu().double() - y).abs() <= H.turned_bound(y, size, torch.bfloat16)).all())
