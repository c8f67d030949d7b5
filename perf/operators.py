"""The dense and linear attention operators of libdsa as they are measured.

Two families over one packed batch (see include/dsa_dense.h and
include/dsa_linear.h):

* dense attention: every visible position of a packed K/V cache, grouped
  heads, whole prompts, chunks of prompts and single tokens;
* linear attention with a decay for each head: chunked for prompts, recurrent
  for single tokens, over a pool of fp32 states.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits; where it is true it calls the library's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_DEV = "cuda"


# ----------------------------------------------------------------- the cases

def _ragged(rng, n, lo, hi):
    """n lengths between lo and hi, spread over their logarithm."""
    return [min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) for _ in range(n)]


def _text(v):
    return ",".join(str(int(x)) for x in v)


def _ints(s):
    return [int(x) for x in s.split(",")]


def _dense(name, rows, lens, hq, hkv, dk, dv, dtype="bf16", fused=False):
    return {"name": name, "op": "dense", "rows": _text(rows), "lens": _text(lens), "hq": hq, "hkv": hkv,
            "dk": dk, "dv": dv, "dtype": dtype, "fused": fused}


def _linear(name, rows, h, dk, dv, dtype="bf16", fused=False, state=True):
    return {"name": name, "op": "linear", "rows": _text(rows), "h": h, "dk": dk, "dv": dv, "dtype": dtype,
            "fused": fused, "state": state}


def _step(name, b, h, dk, dv, dtype="bf16"):
    return {"name": name, "op": "step", "b": b, "h": h, "dk": dk, "dv": dv, "dtype": dtype}


def listed():
    return [
        # The smallest call: one new token of one short request, where latency counts.
        _dense("token_4k", [1], [4096], 64, 8, 128, 128),
        # A decode batch of 32 places, ragged contexts, two of the places unused (length 0).
        _dense("tokens_batch32", [1] * 32,
               [31807, 517, 9301, 0, 1024, 28672, 15003, 4099, 22222, 700, 32768, 129, 6143, 18001, 2500, 11111,
                256, 30001, 0, 8192, 26003, 2971, 13579, 1, 20480, 5005, 24601, 17000, 777, 12000, 29999, 10007],
               64, 8, 128, 128),
        # Drafted tokens being verified: a few rows for each request, 8 heads of width 64, fp16.
        _dense("verify_d64", [4, 3, 5, 4, 2, 4], [4096, 2000, 3333, 65, 1027, 4095], 8, 8, 64, 64, "fp16"),
        # Whole prompts within the top-k (full attention), one head of K for each query head, width 192 / 128.
        _dense("prompts_d192", [2048, 1021, 77, 1536, 1, 1999, 640, 300], [2048, 1021, 77, 1536, 1, 1999, 640, 300],
               64, 64, 192, 128),
        # A 2048-row chunk of a longer prompt over its cache, q/k/v read out of one fused projection, fp16.
        _dense("chunk_2048", [2048], [10240], 64, 8, 128, 128, "fp16"),
        # One long prompt.
        _dense("prompt_16k", [16384], [16384], 16, 2, 128, 128, fused=True),
        # One token of one request: latency.
        _step("step_1", 1, 64, 128, 128),
        # A decode batch: the states' traffic.
        _step("step_96", 96, 64, 128, 128),
        # Short prompts of narrow heads from an empty state, fp16.
        _linear("prompts_d64", [311, 64, 1000, 17, 129], 8, 64, 64, "fp16", state=False),
        # Packed prompts of a serving batch, ragged, each going on from a state of its own.
        _linear("prompts_ragged", [4096, 130, 1, 2047, 3001, 640, 65, 1500, 2900, 1003, 777, 100], 32, 128, 128,
                fused=True),
        # One long prompt: 16 heads alone do not fill the GPU.
        _linear("prompt_64k", [65536], 16, 128, 128, state=False),
    ]


def draw(rng):
    op = rng.choice(["dense", "dense", "dense", "linear", "linear", "step"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "step":
        dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        h = rng.choice([4, 8, 16, 24, 32, 64])
        b = _ragged(rng, 1, 1, 96)[0]
        return {k: v for k, v in _step("", b, h, dk, dv, dtype).items() if k != "name"}
    if op == "linear":
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 64), (64, 128)])
        h = rng.choice([2, 5, 8, 16, 32])
        n = rng.choice([1, 1, 2, 3, 7, 12])
        top = max(2, min(32768, (65536 * 16) // (h * n)))
        rows = _ragged(rng, n, 1, top)
        return {k: v for k, v in _linear("", rows, h, dk, dv, dtype, rng.random() < 0.4, rng.random() < 0.6).items()
                if k != "name"}
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    kind = rng.choice(["tokens", "prompts", "chunk"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 8])
    if kind == "tokens":
        n = _ragged(rng, 1, 1, 32)[0]
        lens = _ragged(rng, n, 1, 32768)
        rows = [min(L, rng.choice([1, 1, 1, 2, 5])) for L in lens]
    elif kind == "prompts":
        n = rng.choice([1, 2, 4, 9])
        lens = _ragged(rng, n, 1, max(64, min(8192, 32768 // n)))
        rows = list(lens)
    else:
        n = rng.choice([1, 2, 3])
        lens = _ragged(rng, n, 64, 10240)
        rows = [max(1, min(L, _ragged(rng, 1, 1, 2048)[0])) for L in lens]
    return {k: v for k, v in _dense("", rows, lens, hq, hkv, dk, dv, dtype, rng.random() < 0.4 and rows == lens).items()
            if k != "name"}


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


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "dense":
        rows, lens = _ints(case["rows"]), _ints(case["lens"])
        R, L = sum(rows), sum(lens)
        hq, hkv, dk, dv = case["hq"], case["hkv"], case["dk"], case["dv"]
        if case["fused"]:
            s["q"], s["k"], s["v"] = _heads(g, L, [(hq, dk), (hkv, dk), (hkv, dv)], dt, True)
        else:
            s["q"] = _normal(g, R, hq, dk, dtype=dt)
            s["k"], s["v"] = _heads(g, L, [(hkv, dk), (hkv, dv)], dt, False)
        # Row i of a request's n rows sees its first L - n + i + 1 positions (none where the place is unused).
        seen = [max(0, min(L_b, L_b - n + i + 1)) for n, L_b in zip(rows, lens) for i in range(n)]
        s["row_len"] = torch.tensor(seen, dtype=torch.int32, device=_DEV)
        s["offsets"], s["row_offsets"] = _prefix(lens), _prefix(rows)
        s["scale"] = 1.0 / math.sqrt(dk)
        s["out"] = torch.empty(R, hq, dv, dtype=dt, device=_DEV)
        s["lse"] = torch.empty(R, hq, dtype=torch.float32, device=_DEV)
        return s
    h, dk, dv = case["h"], case["dk"], case["dv"]
    rows = _ints(case["rows"]) if case["op"] == "linear" else [1] * case["b"]
    T, B = sum(rows), len(rows)
    s["q"], s["k"], s["v"] = _heads(g, T, [(h, dk), (h, dk), (h, dv)], dt, case.get("fused", False))
    # Heads forget over from 1 / 4 of a token's weight to thousands of tokens: 1 - 2^-(2 .. 12).
    e = torch.linspace(2.0, 12.0, h, device=_DEV, dtype=torch.float64)
    s["log_decay"] = torch.log1p(-torch.exp2(-e)).float()
    s["row_offsets"] = _prefix(rows)
    s["scale"] = 1.0 / math.sqrt(dk)
    s["state_in"] = _normal(g, B, h, dk, dv) if case.get("state", True) else None
    s["state_out"] = torch.empty(B, h, dk, dv, dtype=torch.float32, device=_DEV)
    s["out"] = torch.empty(T, h, dv, dtype=dt, device=_DEV)
    return s


# -------------------------------------------------------------- one pass

def _dense_plain(s):
    case = s["case"]
    rows, lens = _ints(case["rows"]), _ints(case["lens"])
    hkv, dk, dv = case["hkv"], case["dk"], case["dv"]
    G = case["hq"] // hkv
    outs, lses = [], []
    r0 = l0 = 0
    for n, L in zip(rows, lens):            # requests have shapes of their own
        q = s["q"][r0:r0 + n].float().view(n, hkv, G, dk).permute(1, 2, 0, 3).reshape(hkv, G * n, dk)
        k = s["k"][l0:l0 + L].float().permute(1, 2, 0)                      # [hkv, dk, L]
        v = s["v"][l0:l0 + L].float().permute(1, 0, 2)                      # [hkv, L, dv]
        x = torch.matmul(q, k).mul_(s["scale"]).view(hkv, G, n, L)
        hidden = torch.arange(L, device=_DEV)[None, :] >= s["row_len"][r0:r0 + n, None]
        x.masked_fill_(hidden, -math.inf)
        if L == 0:
            outs.append(torch.zeros(n, hkv * G, dv, device=_DEV))
            lses.append(torch.full((n, hkv * G), -math.inf, device=_DEV))
        else:
            m = x.amax(dim=-1, keepdim=True).clamp_(min=-3.0e38)
            p = x.sub_(m).exp_()
            z = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p.view(hkv, G * n, L), v).view(hkv, G, n, dv) / z.clamp(min=1e-37)
            outs.append(o.permute(2, 0, 1, 3).reshape(n, hkv * G, dv))
            lses.append((m + z.log()).squeeze(-1).permute(2, 0, 1).reshape(n, hkv * G))
        r0, l0 = r0 + n, l0 + L
    return {"out": torch.cat(outs).to(s["q"].dtype), "lse": torch.cat(lses)}


def _linear_plain(s):
    """Chunks of 128 tokens: products within a chunk, and the chunks' states
    carried forward by one product with the decays between chunks."""
    case, C = s["case"], 128
    h, dk, dv = case["h"], case["dk"], case["dv"]
    ld = s["log_decay"].double()                                            # [h]
    i = torch.arange(C, device=_DEV, dtype=torch.float64)
    w = i[:, None] - i[None, :]
    within = torch.exp(ld[:, None, None] * w.clamp(min=0)).mul_(w >= 0).float()        # [h, C, C]
    reach = torch.exp(ld[:, None] * (i + 1)).float()                        # [h, C]
    outs, finals = [], []
    r0 = 0
    for b, n in enumerate(_ints(case["rows"])):                             # requests have lengths of their own
        N = -(-n // C)

        def part(t, d):
            x = t[r0:r0 + n].float()
            return torch.cat([x, x.new_zeros(N * C - n, h, d)]).view(N, C, h, d).permute(2, 0, 1, 3)  # [h, N, C, d]

        q, k, v = part(s["q"], dk), part(s["k"], dk), part(s["v"], dv)
        last = torch.full((N,), C, device=_DEV, dtype=torch.float64)
        last[-1] = n - (N - 1) * C
        left = last[None, :, None] - 1 - i[None, None, :]                   # tokens after i in its chunk
        fade = torch.exp(ld[:, None, None] * left.clamp(min=0)).mul_(left >= 0).float()
        add = torch.matmul((k * fade[..., None]).transpose(-1, -2), v)      # [h, N, dk, dv]
        start = s["state_in"][b].float() if s["state_in"] is not None else torch.zeros(h, dk, dv, device=_DEV)
        # State before chunk c (c = N: after the last): decays over the tokens in between.
        at = torch.cat([last.new_zeros(1), last.cumsum(0)])                 # [N + 1]
        gap = at[:, None] - at[None, :]                                     # row c, column c'
        keep = torch.exp(ld[:, None, None] * gap.clamp(min=0)).mul_(gap >= 0).float()
        terms = torch.cat([start[:, None], add], dim=1).view(h, N + 1, dk * dv)
        states = torch.matmul(keep, terms).view(h, N + 1, dk, dv)
        o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)).mul_(within[:, None]), v)
        o += torch.matmul(q, states[:, :N]) * reach[:, None, :, None]
        outs.append((o * s["scale"]).permute(1, 2, 0, 3).reshape(N * C, h, dv)[:n])
        finals.append(states[:, N])
        r0 += n
    return {"out": torch.cat(outs).to(s["q"].dtype), "state": torch.stack(finals)}


def _step_plain(s):
    q, k, v = (s[x].float() for x in "qkv")                                 # [B, h, d]
    state = s["state_in"] * torch.exp(s["log_decay"])[None, :, None, None] + k[..., :, None] * v[..., None, :]
    o = torch.matmul(q[..., None, :], state).squeeze(-2) * s["scale"]
    return {"out": o.to(s["q"].dtype), "state": state}


def _handle(s):
    """The problem and the workspace that a user's program keeps between calls."""
    import dsa_sparse_attention_03_gb300 as dsa
    case = s["case"]
    if case["op"] == "dense":
        rows, lens = _ints(case["rows"]), _ints(case["lens"])
        prob = dsa.DenseProblem.from_tensors(
            q=s["q"], k=s["k"], v=s["v"], offsets=s["offsets"], row_offsets=s["row_offsets"], row_len=s["row_len"],
            softmax_scale=s["scale"], L_max=max(lens), L_total=sum(lens), rows_max=max(rows))
        return dsa, prob, dsa.alloc_dense_workspace(prob)
    rows = _ints(case["rows"]) if case["op"] == "linear" else [1] * case["b"]
    prob = dsa.LinearProblem.from_tensors(
        q=s["q"], k=s["k"], v=s["v"], log_decay=s["log_decay"], row_offsets=s["row_offsets"], scale=s["scale"],
        rows_max=max(rows))
    return dsa, prob, dsa.alloc_linear_workspace(prob)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"dense": _dense_plain, "linear": _linear_plain, "step": _step_plain}[op](s)
    if "handle" not in s:
        s["handle"] = _handle(s)
    dsa, prob, ws = s["handle"]
    if op == "dense":
        dsa.dsa_dense_attn(prob, s["out"], s["lse"], ws)
        return {"out": s["out"], "lse": s["lse"]}
    call = dsa.dsa_linear_attn if op == "linear" else dsa.dsa_linear_step
    call(prob, s["state_in"], s["state_out"], s["out"], ws)
    return {"out": s["out"], "state": s["state_out"]}


# ------------------------------------------------- what a pass has to do

def work(case):
    if case["op"] == "dense":
        rows, lens = _ints(case["rows"]), _ints(case["lens"])
        hq, hkv, dk, dv = case["hq"], case["hkv"], case["dk"], case["dv"]
        pairs = sum(max(0, min(L, L - n + i + 1)) for n, L in zip(rows, lens) for i in range(n))
        R, L = sum(rows), sum(lens)
        return {"bytes": 2 * (R * hq * (dk + dv) + L * hkv * (dk + dv)) + 4 * R * hq,
                "flops": 2 * pairs * hq * (dk + dv)}
    rows = _ints(case["rows"]) if case["op"] == "linear" else [1] * case["b"]
    h, dk, dv = case["h"], case["dk"], case["dv"]
    T, states = sum(rows), len(rows) * h * dk * dv * 4
    return {"bytes": 2 * T * h * 2 * (dk + dv) + states * (2 if case.get("state", True) else 1),
            "flops": 4 * T * h * dk * dv}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    q, k, v = s["q"], s["k"], s["v"]
    if case["op"] == "dense":
        G = case["hq"] // case["hkv"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=_DEV)
        r = s["row_offsets"].tolist()
        o = s["offsets"].tolist()
        for b in range(len(r) - 1):
            for first in range(r[b], r[b + 1], 1024):
                R = slice(first, min(first + 1024, r[b + 1]))
                far = int(s["row_len"][R].max())
                if far == 0:
                    continue
                see = torch.arange(far, device=_DEV)[None] < s["row_len"][R, None]
                for h in range(case["hq"]):
                    x = q[R, h].double() @ k[o[b]:o[b] + far, h // G].double().T * s["scale"]
                    x = torch.where(see, x, torch.full_like(x, -math.inf))
                    z = torch.logsumexp(x, dim=1)
                    lse[R, h] = z
                    w = torch.where(see, torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[:, None]), 0.0)
                    out[R, h] = w @ v[o[b]:o[b] + far, h // G].double()
        return {"out": out, "lse": lse}
    # One token after the other, all requests abreast; a request that has ended stays as it is.
    rows = _ints(case["rows"]) if case["op"] == "linear" else [1] * case["b"]
    h, dk, dv = case["h"], case["dk"], case["dv"]
    B = len(rows)
    first = s["row_offsets"][:-1].long()
    n = torch.tensor(rows, device=_DEV)
    S = s["state_in"].double() if s["state_in"] is not None else torch.zeros(B, h, dk, dv, dtype=torch.float64, device=_DEV)
    lam = torch.exp(s["log_decay"].double())[None, :, None, None]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=_DEV)
    order = sorted(range(B), key=lambda b: -rows[b])
    for t in range(max(rows)):
        alive = B
        while rows[order[alive - 1]] <= t:
            alive -= 1
        if alive == B:
            at = first + t
            S = S * lam + k[at].double()[..., :, None] * v[at].double()[..., None, :]
            out[at] = torch.matmul(q[at].double()[..., None, :], S).squeeze(-2) * s["scale"]
        else:
            w = torch.tensor(order[:alive], device=_DEV) if alive > 1 else slice(order[0], order[0] + 1)
            at = first[w] + t
            X = S[w] * lam + k[at].double()[..., :, None] * v[at].double()[..., None, :]
            S[w] = X
            out[at] = torch.matmul(q[at].double()[..., None, :], X).squeeze(-2) * s["scale"]
    return {"out": out, "state": S}
