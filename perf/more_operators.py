"""The operators around a paged K/V cache held in 4 bits, as they are measured.

Four operators of one serving path (see include/dsa_rope.h and include/dsa_kv4.h):

* qk: norms of queries and keys for each head and the position rotation, in one pass;
* append: the same on the way into the cache, K and V quantised to 4 bits and written
  into pages (the rows are then read back, which shows what the pages hold);
* read: rows of the pages back as 16-bit K and V;
* attn: softmax attention over the pages, for single tokens, drafted rows, chunks of
  prompts and whole prompts.

The cache: a page holds ``ps`` positions; for each K/V head it is one block of bytes, K's
codes [D_k / 64, ps, 32], V's codes [D_v / 64, ps, 32], K's scales [D_k / 64, ps] and V's
[D_v / 64, ps] in bf16.  A value is (code - 8) * scale, the code of an even column in
the low half of its byte; a scale belongs to 64 columns of one position.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits (what goes into 4 bits in 64: a value next to the border of two codes
has to fall on the right side); where it is true it calls the library's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_DEV = "cuda"


# ----------------------------------------------------------------- the cases

def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(v):
    return ",".join(str(int(x)) for x in v)


def _ints(s):
    return [int(x) for x in s.split(",")]


def _qk(name, rows, hq, hkv, d, rot, first=0, pairs="half", norm=True, far=0, dtype="bf16", fused=False):
    return {"name": name, "op": "qk", "rows": rows, "hq": hq, "hkv": hkv, "dk": d, "rot": rot, "first": first,
            "pairs": pairs, "norm": norm, "far": far, "dtype": dtype, "fused": fused}


def _append(name, rows, lens, hq, hkv, dk, dv, ps, rot, first=0, pairs="half", norm=True, dtype="bf16", fused=False):
    return {"name": name, "op": "append", "rows": _text(rows), "lens": _text(lens), "hq": hq, "hkv": hkv, "dk": dk,
            "dv": dv, "ps": ps, "rot": rot, "first": first, "pairs": pairs, "norm": norm, "dtype": dtype, "fused": fused}


def _read(name, rows, lens, hkv, dk, dv, ps, dtype="bf16"):
    return {"name": name, "op": "read", "rows": _text(rows), "lens": _text(lens), "hkv": hkv, "dk": dk, "dv": dv,
            "ps": ps, "dtype": dtype}


def _attn(name, rows, lens, hq, hkv, dk, dv, ps, dtype="bf16"):
    return {"name": name, "op": "attn", "rows": _text(rows), "lens": _text(lens), "hq": hq, "hkv": hkv, "dk": dk,
            "dv": dv, "ps": ps, "dtype": dtype}


_BATCH32 = [31807, 517, 9301, 0, 1024, 28672, 15003, 4099, 22222, 700, 32768, 129, 6143, 18001, 2500, 11111,
            256, 30001, 0, 8192, 26003, 2971, 13579, 1, 20480, 5005, 24601, 17000, 777, 12000, 29999, 10007]
_RAGGED = [2048, 1021, 77, 1536, 1, 1999, 640, 300]


def listed():
    return [
        # The smallest calls: the new token of one request, far into a long context; latency.
        _qk("qk_token", 1, 64, 8, 128, 128, far=300000),
        # The rows of a packed batch of prompts, read out of one fused projection.
        _qk("qk_prompts", 9601, 64, 8, 128, 128, fused=True),
        # A decode batch of 32 places, two of them unused: queries normed and rotated, K and V into the cache.
        _append("append_batch32", [1] * 32, _BATCH32, 64, 8, 128, 128, 64, 128),
        # Prompts as they are taken in: K and V alone (the queries went with dsa_qk_norm_rope), odd lengths.
        _append("append_prompts", [4096, 130, 1, 2047, 3001, 326], [4096, 130, 9000, 2047, 5003, 326], 0, 8, 128, 128, 16,
                64, fused=True),
        # A cached prefix of 10240 positions taken back into 16 bits for a prompt's chunk.
        _read("read_prefix", [10240], [10240], 8, 128, 128, 64),
        # The last positions of several short requests, narrow heads, fp16.
        _read("read_tails", [100, 1, 64, 333], [4096, 77, 2000, 333], 8, 64, 64, 32, "fp16"),
        # One new token of one short request, where latency counts.
        _attn("token_4k", [1], [4096], 64, 8, 128, 128, 64),
        # One new token at the end of a long context.
        _attn("token_300k", [1], [307200], 64, 8, 128, 128, 64),
        # A decode batch of 32 places, ragged contexts, two of the places unused (length 0).
        _attn("tokens_batch32", [1] * 32, _BATCH32, 64, 8, 128, 128, 16),
        # Drafted tokens being verified: a few rows for each request, 8 heads of width 64, fp16.
        _attn("verify_d64", [4, 3, 5, 4, 2, 4], [4096, 2000, 3333, 65, 1027, 4095], 8, 8, 64, 64, 32, "fp16"),
        # Whole prompts of ragged lengths over what was just appended, one K/V head for each query head, width 192 / 128.
        _attn("prompts_d192", _RAGGED, _RAGGED, 64, 64, 192, 128, 64),
        # A 2048-row chunk of a longer prompt over its cache.
        _attn("chunk_2048", [2048], [10240], 64, 8, 128, 128, 64),
    ]


def draw(rng):
    op = rng.choice(["qk", "append", "read", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "fp16"])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 8])
    ps = rng.choice([16, 32, 64, 128])
    pairs = rng.choice(["half", "adjacent"])
    norm = rng.random() < 0.7
    rot, first = rng.choice([(dk, 0), (64, 0), (64, dk - 64), (32, 0), (dk // 2, dk // 4), (0, 0)])
    n = rng.choice([1, 1, 2, 3, 7, 32])
    if op == "qk":
        c = _qk("", _spread(rng, 1, 9000), hq, hkv, dk, rot, first, pairs, norm, rng.choice([0, 1000, 1000000]), dtype,
                rng.random() < 0.4)
    elif op == "append":
        rows = [_spread(rng, 1, max(1, 9000 // n)) if rng.random() < 0.6 else 1 for _ in range(n)]
        lens = [r + rng.choice([0, 1, 1000, 30000]) for r in rows]
        c = _append("", rows, lens, rng.choice([0, hq]), hkv, dk, dv, ps, rot, first, pairs, norm, dtype,
                    rng.random() < 0.4)
    elif op == "read":
        lens = [_spread(rng, 1, max(64, 16384 // n)) for _ in range(n)]
        c = _read("", [_spread(rng, 1, x) for x in lens], lens, hkv, dk, dv, ps, dtype)
    else:
        kind = rng.choice(["tokens", "tokens", "prompts", "chunk"])
        if kind == "tokens":
            n = _spread(rng, 1, 32)
            lens = [_spread(rng, 1, 32768) for _ in range(n)]
            rows = [min(x, rng.choice([1, 1, 1, 2, 5])) for x in lens]
        elif kind == "prompts":
            n = rng.choice([1, 2, 4, 9])
            lens = [_spread(rng, 1, max(64, 4096 // n)) for _ in range(n)]
            rows = list(lens)
        else:
            n = rng.choice([1, 2])
            lens = [_spread(rng, 64, 10240) for _ in range(n)]
            rows = [max(1, min(x, _spread(rng, 1, 2048 // n))) for x in lens]
        c = _attn("", rows, lens, hq, hkv, dk, dv, ps, dtype)
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------- the inputs

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=_DEV, dtype=torch.float32, generator=g).to(dtype)


def _prefix(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device=_DEV)


def _heads(g, T, sizes, dtype, fused):
    """Tensors [T, heads, width] for each (heads, width): packed, or views of one
    fused projection [T, sum heads * width]."""
    if not fused:
        return [_normal(g, T, h, d, dtype=dtype) for h, d in sizes]
    x = _normal(g, T, sum(h * d for h, d in sizes), dtype=dtype)
    return [p.view(T, h, d) for p, (h, d) in zip(x.split([h * d for h, d in sizes], dim=1), sizes)]


def _quantise(x):
    """Codes + 8 and scales of x [..., 64], in x's precision: the scale is the largest magnitude / 7 to the
    nearest of four significant bits, ties to even.  (Divided by a tensor: a number would become a product.)"""
    top = x.abs().amax(dim=-1)
    m, e = torch.frexp(top / torch.full_like(top, 7))
    scale = torch.ldexp(torch.round(m * 16) / 16, e)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    codes = torch.where(scale[..., None] > 0, torch.round(x / scale[..., None]), torch.zeros_like(x)) + 8
    return codes.to(torch.uint8), scale


def _parts(pages, dk, dv, ps):
    """Views of the blocks [n, H, bytes]: K's and V's codes [n, H, groups, ps, 32] and scales [n, H, groups, ps]."""
    n, H = pages.shape[:2]
    gk, gv = dk // 64, dv // 64
    a, b = gk * ps * 32, (gk + gv) * ps * 32
    c = b + gk * ps * 2
    return (pages[..., :a].unflatten(2, (gk, ps, 32)), pages[..., a:b].unflatten(2, (gv, ps, 32)),
            pages[..., b:c].view(torch.bfloat16).unflatten(2, (gk, ps)),
            pages[..., c:].view(torch.bfloat16).unflatten(2, (gv, ps)))


def _cache(g, lens, hkv, dk, dv, ps):
    """A pool of pages that hold quantised normals, a few pages more than the requests need, and their table."""
    need = [-(-x // ps) for x in lens]
    n = sum(need) + 3
    pages = torch.empty(n, hkv, ps * (dk + dv) * 17 // 32, dtype=torch.uint8, device=_DEV)
    kc, vc, ks, vs = _parts(pages, dk, dv, ps)
    for first in range(0, n, 1024):
        at = slice(first, min(n, first + 1024))
        for codes, scales in ((kc, ks), (vc, vs)):
            c, s = _quantise(_normal(g, *codes[at].shape[:4], 64))
            codes[at] = c[..., 0::2] | (c[..., 1::2] << 4)
            scales[at] = s.to(torch.bfloat16)
    order = torch.randperm(n, device=_DEV, generator=g).int()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=_DEV)
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    return pages, table


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    dt, dk = _DT[case["dtype"]], case["dk"]
    s = {"case": case}
    if case["op"] in ("qk", "append"):
        # 1 / 10000^(2 i / rot), and norms' weights around 1.
        rot = case["rot"]
        s["inv_freq"] = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=_DEV) / max(rot, 1))
        for x in ("q_weight", "k_weight"):
            s[x] = (1 + 0.2 * _normal(g, dk)).to(dt) if case["norm"] else None
        s["eps"] = 1e-6
    if case["op"] == "qk":
        R = case["rows"]
        s["q"], s["k"] = _heads(g, R, [(case["hq"], dk), (case["hkv"], dk)], dt, case["fused"])
        s["positions"] = torch.arange(R, dtype=torch.int32, device=_DEV) + case["far"]
        s["q_out"], s["k_out"] = (torch.empty(x.shape, dtype=dt, device=_DEV) for x in (s["q"], s["k"]))
        return s
    rows, lens, dv, hkv = _ints(case["rows"]), _ints(case["lens"]), case["dv"], case["hkv"]
    R = sum(rows)
    s["pages"], s["table"] = _cache(g, lens, hkv, dk, dv, case["ps"])
    s["row_offsets"] = _prefix(rows)
    # Row i of a request's n rows is its position L - n + i (none where the place is unused).
    s["positions"] = torch.tensor([max(-1, L - n + i) for n, L in zip(rows, lens) for i in range(n)], dtype=torch.int32,
                                  device=_DEV)
    if case["op"] == "append":
        s["k"], s["v"] = _heads(g, R, [(hkv, dk), (hkv, dv)], dt, case["fused"])
        s["q"] = _normal(g, R, case["hq"], dk, dtype=dt) if case["hq"] else None
        s["q_out"] = torch.zeros(R, case["hq"], dk, dtype=dt, device=_DEV) if case["hq"] else None
    if case["op"] == "attn":
        s["q"] = _normal(g, R, case["hq"], dk, dtype=dt)
        s["row_len"] = s["positions"] + 1
        s["scale"] = 1.0 / math.sqrt(dk)
        s["out"] = torch.empty(R, case["hq"], dv, dtype=dt, device=_DEV)
        s["lse"] = torch.empty(R, case["hq"], dtype=torch.float32, device=_DEV)
    else:
        s["k_out"] = torch.zeros(R, hkv, dk, dtype=dt, device=_DEV)
        s["v_out"] = torch.zeros(R, hkv, dv, dtype=dt, device=_DEV)
    return s


# -------------------------------------------------------------- one pass

def _turned(s, x, weight, wide):
    """x [T, heads, width] normed and rotated, in the type `wide`."""
    case = s["case"]
    x = x.to(wide)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"]) * weight.to(wide)
    rot, first = case["rot"], case["first"]
    if rot == 0:
        return x
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos().to(wide), angle.sin().to(wide)
    part = x[..., first:first + rot]
    if case["pairs"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([x[..., :first], turned, x[..., first + rot:]], dim=-1)


def _qk_plain(s):
    dt = s["q"].dtype
    return {"q": _turned(s, s["q"], s["q_weight"], torch.float32).to(dt),
            "k": _turned(s, s["k"], s["k_weight"], torch.float32).to(dt)}


def _rows(s):
    """Page and place in it of each row that has a position, and which rows these are."""
    ps, row = s["case"]["ps"], torch.arange(s["positions"].shape[0], device=_DEV)
    live = s["positions"] >= 0
    row, pos = row[live], s["positions"][live].long()
    request = torch.bucketize(row, s["row_offsets"][1:].long(), right=True)
    return s["table"][request, pos // ps].long(), pos % ps, live


def _read_plain(s):
    case, out = s["case"], {}
    dk, dv, ps, hkv = case["dk"], case["dv"], case["ps"], case["hkv"]
    kc, vc, ks, vs = _parts(s["pages"], dk, dv, ps)
    page, place, live = _rows(s)
    for name, codes, scales, d in (("k", kc, ks, dk), ("v", vc, vs, dv)):
        c = codes[page, :, :, place].int()                                 # [rows, H, groups, 32]
        x = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).float().sub_(8) * scales[page, :, :, place, None].float()
        full = torch.zeros(live.shape[0], hkv, d, device=_DEV)
        full[live] = x.flatten(-2)
        out[name] = full.to(_DT[case["dtype"]])
    return out


def _append_plain(s):
    case = s["case"]
    dk, dv, ps = case["dk"], case["dv"], case["ps"]
    kc, vc, ks, vs = _parts(s["pages"], dk, dv, ps)
    page, place, live = _rows(s)
    for x, codes, scales in ((_turned(s, s["k"], s["k_weight"], torch.float64), kc, ks), (s["v"].double(), vc, vs)):
        c, scale = _quantise(x[live].unflatten(-1, (-1, 64)))
        codes[page, :, :, place] = c[..., 0::2] | (c[..., 1::2] << 4)
        scales[page, :, :, place] = scale.to(torch.bfloat16)
    out = _read_plain(s)
    if case["hq"]:
        q = _turned(s, s["q"], s["q_weight"], torch.float32) * live[:, None, None]
        out["q"] = q.to(s["q"].dtype)
    return out


def _attn_plain(s):
    case = s["case"]
    hkv, dk, dv, ps = case["hkv"], case["dk"], case["dv"], case["ps"]
    G = case["hq"] // hkv
    outs, lses = [], []
    r0 = 0
    for b, (n, L) in enumerate(zip(_ints(case["rows"]), _ints(case["lens"]))):   # requests have shapes of their own
        if L == 0:
            outs.append(torch.zeros(n, hkv * G, dv, device=_DEV))
            lses.append(torch.full((n, hkv * G), -math.inf, device=_DEV))
            r0 += n
            continue
        kc, vc, ks, vs = _parts(s["pages"][s["table"][b, :-(-L // ps)].long()], dk, dv, ps)

        def values(codes, scales):                                          # [H, L, width]
            x = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float().sub_(8).mul_(scales[..., None].float())
            return x.permute(1, 0, 3, 2, 4).flatten(3).flatten(1, 2)[:, :L]

        q = s["q"][r0:r0 + n].float().view(n, hkv, G, dk).permute(1, 2, 0, 3).reshape(hkv, G * n, dk)
        x = torch.matmul(q, values(kc, ks).transpose(1, 2)).mul_(s["scale"]).view(hkv, G, n, L)
        hidden = torch.arange(L, device=_DEV)[None, :] >= s["row_len"][r0:r0 + n, None]
        x.masked_fill_(hidden, -math.inf)
        m = x.amax(dim=-1, keepdim=True).clamp_(min=-3.0e38)
        p = x.sub_(m).exp_()
        z = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(hkv, G * n, L), values(vc, vs)).view(hkv, G, n, dv) / z.clamp(min=1e-37)
        outs.append(o.permute(2, 0, 1, 3).reshape(n, hkv * G, dv))
        lses.append((m + z.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hkv * G))
        r0 += n
    return {"out": torch.cat(outs).to(s["q"].dtype), "lse": torch.cat(lses)}


def _handle(s):
    """The problems, the cache and the workspace that a user's program keeps between calls."""
    import dsa_sparse_attention_03_gb300 as dsa
    case = s["case"]
    turn = dict(inv_freq=s.get("inv_freq"), rot_first=case.get("first", 0), interleaved=case.get("pairs") == "adjacent",
                q_weight=s.get("q_weight"), k_weight=s.get("k_weight"), eps=s.get("eps", 0.0), positions=s["positions"])
    if case["op"] == "qk":
        return dsa, None, dsa.QKProblem.from_tensors(q=s["q"], k=s["k"], **turn), None
    cache = dsa.KV4Cache.from_tensors(pages=s["pages"], table=s["table"], page_size=case["ps"], D_k=case["dk"],
                                      D_v=case["dv"])
    if case["op"] == "append":
        prob = dsa.QKProblem.from_tensors(q=s["q"], k=s["k"], v=s["v"], row_offsets=s["row_offsets"], **turn)
        return dsa, cache, prob, dsa.alloc_kv4_workspace(device=_DEV)
    if case["op"] == "read":
        return dsa, cache, None, dsa.alloc_kv4_workspace(device=_DEV)
    prob = dsa.KV4Problem.from_tensors(
        cache=cache, q=s["q"], row_offsets=s["row_offsets"], row_len=s["row_len"], softmax_scale=s["scale"],
        L_max=max(_ints(case["lens"])), rows_max=max(_ints(case["rows"])))
    return dsa, cache, prob, dsa.alloc_kv4_workspace(prob, device=_DEV)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"qk": _qk_plain, "append": _append_plain, "read": _read_plain, "attn": _attn_plain}[op](s)
    if "handle" not in s:
        s["handle"] = _handle(s)
    dsa, cache, prob, ws = s["handle"]
    if op == "qk":
        dsa.dsa_qk_norm_rope(prob, s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "attn":
        dsa.dsa_kv4_attn(prob, s["out"], s["lse"], ws)
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        dsa.dsa_kv4_append(cache, prob, s["q_out"], ws)
    dsa.dsa_kv4_read(cache, s["row_offsets"], s["positions"], s["k_out"], s["v_out"], ws)
    out = {"k": s["k_out"], "v": s["v_out"]}
    if s.get("q_out") is not None:
        out["q"] = s["q_out"]
    return out


# ------------------------------------------------- what a pass has to do

def work(case):
    dk = case["dk"]
    if case["op"] == "qk":
        n = case["rows"] * (case["hq"] + case["hkv"]) * dk
        return {"bytes": 4 * n, "flops": 8 * n}
    rows, lens = _ints(case["rows"]), _ints(case["lens"])
    dv, hkv = case["dv"], case["hkv"]
    if case["op"] == "attn":
        hq, R = case["hq"], sum(rows)
        pairs = sum(max(0, min(L, L - n + i + 1)) for n, L in zip(rows, lens) for i in range(n))
        return {"bytes": 2 * R * hq * (dk + dv) + sum(lens) * hkv * (dk + dv) * 17 // 32 + 4 * R * hq,
                "flops": 2 * pairs * hq * (dk + dv)}
    live = sum(min(n, L) for n, L in zip(rows, lens))
    n = live * hkv * (dk + dv)
    read = n * 17 // 32 + 2 * n                                  # out of the pages, into 16 bits
    if case["op"] == "read":
        return {"bytes": read, "flops": n}
    return {"bytes": read + 2 * n + n * 17 // 32 + 4 * live * case["hq"] * dk,
            "flops": 10 * n + 8 * live * case["hq"] * dk}


# ------------------------------------------------- the definitions in 64 bits

def _exact_turn(case, s, x, weight):
    """Head by head and pair by pair, as the definition reads."""
    x = x.double().clone()
    if weight is not None:
        for h in range(x.shape[1]):
            x[:, h] = x[:, h] / torch.sqrt((x[:, h] ** 2).sum(dim=1, keepdim=True) / x.shape[2] + s["eps"])
        x = x * weight.double()
    y = x.clone()
    for i in range(case["rot"] // 2):
        a, b = ((i, i + case["rot"] // 2) if case["pairs"] == "half" else (2 * i, 2 * i + 1))
        a, b = a + case["first"], b + case["first"]
        t = s["positions"].double()[:, None] * s["inv_freq"][i]
        y[..., a] = torch.cos(t) * x[..., a] - torch.sin(t) * x[..., b]
        y[..., b] = torch.sin(t) * x[..., a] + torch.cos(t) * x[..., b]
    return y


def _exact_held(x):
    """What 4 bits keep of x [..., width]: for each 64 columns a scale of four significant bits near a seventh of
    the largest magnitude, and a whole number of scales."""
    out = torch.zeros_like(x)
    for g in range(x.shape[-1] // 64):
        at = slice(64 * g, 64 * g + 64)
        top = x[..., at].abs().amax(dim=-1, keepdim=True)
        top = top / torch.full_like(top, 7.0)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 3)
        scale = torch.round(top / unit) * unit
        out[..., at] = torch.where(scale >= 2.0 ** -126, torch.round(x[..., at] / scale) * scale, 0.0)
    return out


def _exact_values(s, which, page, place):
    """K or V of the positions at (page, place), [positions, H, width]."""
    case = s["case"]
    dk, dv, ps = case["dk"], case["dv"], case["ps"]
    d, code0, scale0 = ((dk, 0, (dk + dv) * ps // 2) if which == "k"
                        else (dv, dk * ps // 2, (dk + dv) * ps // 2 + dk // 32 * ps))
    raw, head = s["pages"], torch.arange(case["hkv"], device=_DEV)

    def at(byte):
        return raw[page[:, None], head[None], byte[:, None]].int()

    cols = []
    for c in range(d):
        byte = at(code0 + (c // 64 * ps + place) * 32 + c % 64 // 2)
        cols.append((byte >> 4 if c % 2 else byte & 15).double() - 8)
    x = torch.stack(cols, dim=-1)
    for g in range(d // 64):
        first = scale0 + 2 * (g * ps + place)
        bits = (at(first) << 16) | (at(first + 1) << 24)
        x[..., 64 * g:64 * g + 64] *= bits.view(torch.float32).double()[..., None]
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return {x: _exact_turn(case, s, s[x], s[x + "_weight"]) for x in "qk"}
    rows, lens, ps = _ints(case["rows"]), _ints(case["lens"]), case["ps"]
    if case["op"] == "append":
        live = (s["positions"] >= 0).double()[:, None, None]
        out = {"k": _exact_held(_exact_turn(case, s, s["k"], s["k_weight"])) * live, "v": _exact_held(s["v"].double()) * live}
        if case["hq"]:
            out["q"] = _exact_turn(case, s, s["q"], s["q_weight"]) * live
        return out
    if case["op"] == "read":
        out = {x: torch.zeros(s[x + "_out"].shape, dtype=torch.float64, device=_DEV) for x in "kv"}
        r = 0
        for b, n in enumerate(rows):
            pos = s["positions"][r:r + n].long()
            for x in "kv":
                out[x][r:r + n] = _exact_values(s, x, s["table"][b, pos // ps].long(), pos % ps)
            r += n
        return out
    G = case["hq"] // case["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=_DEV)
    r0 = 0
    for b, (n, L) in enumerate(zip(rows, lens)):
        for first in range(r0, r0 + n, 1024):
            R = slice(first, min(first + 1024, r0 + n))
            far = int(s["row_len"][R].max())
            if far == 0:
                continue
            pos = torch.arange(far, device=_DEV)
            k, v = (_exact_values(s, x, s["table"][b, pos // ps].long(), pos % ps) for x in "kv")
            see = pos[None] < s["row_len"][R, None]
            for h in range(case["hq"]):
                x = s["q"][R, h].double() @ k[:, h // G].T * s["scale"]
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, dim=1)
                lse[R, h] = z
                w = torch.where(see, torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[:, None]), 0.0)
                out[R, h] = w @ v[:, h // G]
        r0 += n
    return {"out": out, "lse": lse}
