"""Norms, rotation and the 4-bit cache without a GPU: the structs' layout, what the host refuses, the
workspace, the binding's checks, and the definitions that the GPU tests use.  Nothing is launched."""
import ctypes

import pytest

import kv4_harness as H


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_sparse_attention_03_gb300 as m
    return m


FAKE = 1 << 20   # never read: the calls fail before any launch
BAD_WS = ctypes.c_void_p(FAKE + 16)   # (and were a check under test missing, this one would still refuse)


def _cache(dsa, **kw):
    return dsa.KV4Cache(**dict(dict(n_pages=100, page_size=64, H_kv=2, D_k=128, D_v=128, B=2, table_cols=64, pages=FAKE,
                                    table=FAKE), **kw))


def _qk(dsa, **kw):
    return dsa.QKProblem(**dict(dict(R=2, B=2, H_q=8, H_kv=2, D_k=128, D_v=128, rot=128, rot_first=0, eps=1e-6, q=FAKE, k=FAKE,
                                     v=FAKE, q_weight=FAKE, k_weight=FAKE, inv_freq=FAKE, positions=FAKE, row_offsets=FAKE),
                                **kw))


def _prob(dsa, **kw):
    return dsa.KV4Problem(**dict(dict(R=2, H_q=8, L_max=4096, rows_max=1, softmax_scale=0.1, q=FAKE, row_offsets=FAKE,
                                      row_len=FAKE), **kw))


def _attn(dsa, c, p, out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return dsa.lib().dsa_kv4_attn(ctypes.byref(c.c), ctypes.byref(p.c), out, lse, ctypes.c_void_p(ws), n, None)


def test_struct_layout(dsa):
    assert ctypes.sizeof(dsa.dsa_qk_problem) == 128 and dsa.dsa_qk_problem.q_stride.offset == 40
    assert dsa.dsa_qk_problem.q.offset == 64 and dsa.dsa_qk_problem.row_offsets.offset == 120
    assert ctypes.sizeof(dsa.dsa_kv4_cache) == 48 and dsa.dsa_kv4_cache.pages.offset == 32
    assert ctypes.sizeof(dsa.dsa_kv4_problem) == 56 and dsa.dsa_kv4_problem.q_stride.offset == 24


def test_headers_from_c(dsa, tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lib = os.path.dirname(dsa.LIB_PATH)
    for header in ("dsa_rope.h", "dsa_kv4.h"):
        src = tmp_path / "h.c"
        src.write_text(f'#include "{header}"\nint a[sizeof(dsa_qk_problem) == 128 ? 1 : -1];\n'
                       + ("int b[sizeof(dsa_kv4_cache) == 48 && sizeof(dsa_kv4_problem) == 56 ? 1 : -1];\n"
                          "int main(void) { return dsa_kv4_block_bytes(128, 128, 64) != 8704; }\n" if "kv4" in header else
                          "int main(void) { dsa_qk_problem p = {0}; return dsa_qk_norm_rope(&p, 0, 0, 0) == 0; }\n"))
        exe = str(tmp_path / "h")
        res = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                              exe, "-L", lib, "-ldsa", "-Wl,-rpath," + lib], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
        assert subprocess.run([exe], timeout=120).returncode == 0


@pytest.mark.parametrize("kw,status,text", [
    (dict(R=-1), 1, b"R=-1"), (dict(R=70000), 1, b"R="), (dict(H_q=0), 2, b"H_q"), (dict(H_q=129), 2, b"H_q"),
    (dict(H_kv=0), 2, b"H_kv"), (dict(H_kv=200), 2, b"H_kv"), (dict(D_k=96), 2, b"D_k"), (dict(D_k=512), 2, b"D_k"),
    (dict(rot=4), 2, b"rot="), (dict(rot=136), 2, b"rot="), (dict(rot=-8), 2, b"rot="), (dict(rot_first=4), 2, b"rot_first"),
    (dict(rot=64, rot_first=66), 2, b"rot_first"), (dict(rot=64, rot_first=-4), 2, b"rot_first"),
    (dict(eps=-1e-6), 1, b"eps"), (dict(eps=float("nan")), 1, b"eps"), (dict(eps=float("inf")), 1, b"eps"),
    (dict(flags=0x1), 1, b"flag"), (dict(q_stride=1000), 1, b"q_stride"), (dict(k_stride=260), 1, b"k_stride"),
    (dict(k_stride=-256), 1, b"k_stride"), (dict(q=FAKE + 2), 1, b"aligned"), (dict(k_weight=FAKE + 8), 1, b"aligned"),
    (dict(inv_freq=FAKE + 4), 1, b"inv_freq"), (dict(inv_freq=None), 1, b"inv_freq"), (dict(positions=None), 1, b"positions"),
    (dict(positions=FAKE + 2), 1, b"positions"),
])
def test_turn_refusals(dsa, kw, status, text):
    lib, p = dsa.lib(), _qk(dsa, **kw)
    assert lib.dsa_qk_norm_rope(ctypes.byref(p.c), FAKE, FAKE, None) == status
    assert text in lib.dsa_last_error_string()
    c = _cache(dsa)
    assert lib.dsa_kv4_append(ctypes.byref(c.c), ctypes.byref(p.c), FAKE, BAD_WS, 1 << 20, None) == status
    assert text in lib.dsa_last_error_string()


def test_turn_buffers_refused(dsa):
    lib, p = dsa.lib(), _qk(dsa)
    for q, k in ((None, FAKE), (FAKE, None), (FAKE + 8, FAKE), (FAKE, FAKE + 2)):
        assert lib.dsa_qk_norm_rope(ctypes.byref(p.c), q, k, None) == 1
    assert lib.dsa_qk_norm_rope(None, FAKE, FAKE, None) == 1


@pytest.mark.parametrize("kw,status,text", [
    (dict(D_k=256), 2, b"D_k"), (dict(D_v=64), 2, b"D_k"), (dict(D_k=64), 2, b"D_k"), (dict(page_size=8), 2, b"page_size"),
    (dict(page_size=48), 2, b"page_size"), (dict(page_size=256), 2, b"page_size"), (dict(n_pages=0), 1, b"n_pages"),
    (dict(H_kv=0), 2, b"H_kv"), (dict(H_kv=129), 2, b"H_kv"), (dict(B=0), 2, b"B=0"), (dict(B=5000), 2, b"B="),
    (dict(table_cols=0), 2, b"table_cols"), (dict(table_cols=1 << 25), 2, b"table_cols"), (dict(pages=None), 1, b"pages"),
    (dict(pages=FAKE + 8), 1, b"pages"), (dict(table=None), 1, b"table"), (dict(table=FAKE + 2), 1, b"table"),
])
def test_cache_refusals(dsa, kw, status, text):
    lib, c = dsa.lib(), _cache(dsa, **kw)
    q, p = _qk(dsa), _prob(dsa, H_q=129 // max(1, c.H_kv) * c.H_kv if 0 < c.H_kv <= 128 else 8)
    for got in (lib.dsa_kv4_append(ctypes.byref(c.c), ctypes.byref(q.c), FAKE, BAD_WS, 1 << 20, None),
                lib.dsa_kv4_read(ctypes.byref(c.c), 2, FAKE, FAKE, 0, FAKE, FAKE, BAD_WS, 1 << 20, None),
                _attn(dsa, c, p, ws=FAKE + 16)):
        assert got == status
        assert text in lib.dsa_last_error_string()
    assert lib.dsa_kv4_workspace_size(ctypes.byref(c.c), ctypes.byref(p.c)) == 0


@pytest.mark.parametrize("kw", [dict(H_kv=4), dict(D_k=64), dict(D_v=64), dict(B=3), dict(k=None), dict(v=None),
                                dict(row_offsets=None)])
def test_append_refuses_what_is_not_the_caches(dsa, kw):
    lib, p, c = dsa.lib(), _qk(dsa, **dict(dict(rot=64), **kw)), _cache(dsa)
    assert lib.dsa_kv4_append(ctypes.byref(c.c), ctypes.byref(p.c), FAKE, ctypes.c_void_p(FAKE), 255, None) == 1
    assert lib.dsa_kv4_append(ctypes.byref(c.c), ctypes.byref(p.c), FAKE, ctypes.c_void_p(FAKE), 256, None) == 1


def test_read_refusals(dsa):
    lib, c = dsa.lib(), _cache(dsa)
    ok = [2, FAKE, FAKE, 0, FAKE, FAKE, FAKE, 256, None]
    for at, x in ((0, -1), (1, None), (2, None), (1, FAKE + 2), (3, 0x800), (4, FAKE + 8), (5, FAKE + 2), (6, FAKE + 16), (7, 100)):
        args = list(ok)
        args[at] = x
        assert lib.dsa_kv4_read(ctypes.byref(c.c), *args) == 1, (at, x)


@pytest.mark.parametrize("kw,status,text", [
    (dict(R=-1), 1, b"R=-1"), (dict(R=70000), 1, b"R="), (dict(H_q=0), 2, b"H_q"), (dict(H_q=130), 2, b"H_q"),
    (dict(H_q=7), 2, b"H_kv"), (dict(L_max=-1), 1, b"L_max"), (dict(rows_max=-1), 1, b"rows_max"),
    (dict(q_stride=1000), 1, b"q_stride"), (dict(q_stride=1028), 1, b"q_stride"), (dict(softmax_scale=0.0), 1, b"softmax_scale"),
    (dict(softmax_scale=float("nan")), 1, b"softmax_scale"), (dict(softmax_scale=float("inf")), 1, b"softmax_scale"),
    (dict(flags=0x800), 1, b"flag"), (dict(q=None), 1, b"q/out"), (dict(q=FAKE + 8), 1, b"16-byte"), (dict(row_offsets=None), 1, b"row_offsets"),
    (dict(row_len=FAKE + 2), 1, b"4-byte"),
])
def test_attention_refusals(dsa, kw, status, text):
    assert _attn(dsa, _cache(dsa), _prob(dsa, **kw)) == status
    assert text in dsa.lib().dsa_last_error_string()


def test_attention_buffers_refused(dsa):
    c, p = _cache(dsa), _prob(dsa)
    n = dsa.lib().dsa_kv4_workspace_size(ctypes.byref(c.c), ctypes.byref(p.c))
    assert n % 256 == 0 and n > 0
    assert _attn(dsa, c, p, out=None) == 1 and _attn(dsa, c, p, out=FAKE + 8) == 1 and _attn(dsa, c, p, lse=FAKE + 2) == 1
    assert _attn(dsa, c, p, ws=FAKE + 16) == 1 and _attn(dsa, c, p, n=n - 1) == 1
    assert b"required" in dsa.lib().dsa_last_error_string()
    for limit in (0, -5, 10 ** 11):
        assert dsa.lib().dsa_test_kv4_missing_stage(ctypes.byref(c.c), ctypes.byref(p.c), FAKE, None, ctypes.c_void_p(FAKE),
                                                    1 << 40, limit, None) == 1


def test_block_bytes(dsa):
    for dk, dv in ((64, 64), (128, 128), (192, 128)):
        for ps in (16, 32, 64, 128):
            n = dsa.dsa_kv4_block_bytes(dk, dv, ps)
            assert n == H.block_bytes(dk, dv, ps) == ps * (dk + dv) // 2 + ps * (dk + dv) // 32 and n % 16 == 0
    for bad in ((128, 64, 64), (256, 256, 64), (128, 128, 0), (128, 128, 24)):
        with pytest.raises(dsa.DsaError):
            dsa.dsa_kv4_block_bytes(*bad)


def test_binding_checks(dsa):
    import torch
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    h = torch.float16
    pages, table = torch.zeros(9, 2, 8704, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    size = dict(page_size=64, D_k=128, D_v=128)
    cache = dsa.KV4Cache.from_tensors(pages=pages, table=table, **size)
    assert (cache.n_pages, cache.H_kv, cache.B, cache.table_cols) == (9, 2, 2, 4)
    for bad in (dict(pages=pages.int()), dict(pages=pages[:, :, :8000]), dict(pages=pages.transpose(0, 1)), dict(table=table.long()),
                dict(table=table[0]), dict(table=table.t()), dict(pages=pages[0])):
        with pytest.raises(ValueError):
            dsa.KV4Cache.from_tensors(**dict(dict(pages=pages, table=table, **size), **bad))
    with pytest.raises(dsa.DsaError):
        dsa.KV4Cache.from_tensors(pages=pages, table=table, page_size=64, D_k=128, D_v=64)
    f = torch.zeros(64, dtype=torch.float64)
    ok = dict(q=mk(3, 8, 128), k=mk(3, 2, 128), v=mk(3, 2, 128), positions=H.ints([0, 1, 2]), inv_freq=f, q_weight=mk(128),
              k_weight=mk(128), row_offsets=H.ints([0, 1, 3]))
    p = dsa.QKProblem.from_tensors(**ok)
    assert (p.R, p.B, p.H_q, p.H_kv, p.D_k, p.D_v, p.rot, p.flags) == (3, 2, 8, 2, 128, 128, 128, 0)
    x = mk(3, 12 * 128)
    p = dsa.QKProblem.from_tensors(**dict(ok, q=x[:, :1024].unflatten(1, (8, 128)), k=x[:, 1024:1280].unflatten(1, (2, 128)),
                                          interleaved=True))
    assert p.q_stride == p.k_stride == 1536 and p.flags == dsa.DSA_FLAG_ROPE_ADJACENT
    for bad in (dict(q=mk(3, 8, 128, dt=h)), dict(q=mk(2, 8, 128)), dict(k=mk(3, 2, 64)), dict(v=mk(3, 1, 128)), dict(k=None),
                dict(positions=H.ints([0, 1])), dict(positions=torch.arange(3)), dict(inv_freq=f.float()), dict(inv_freq=f[None]),
                dict(q_weight=mk(64)), dict(k_weight=mk(128, dt=h)), dict(k=mk(1, 2, 128).expand(3, 2, 128)),
                dict(q=None, k=None, v=None)):
        with pytest.raises(ValueError):
            dsa.QKProblem.from_tensors(**dict(ok, **bad))
    a = dict(cache=cache, q=mk(3, 8, 128), row_offsets=H.ints([0, 1, 3]), row_len=H.ints([5, 6, 7]), softmax_scale=0.1)
    kp = dsa.KV4Problem.from_tensors(**a)
    assert (kp.R, kp.H_q, kp.L_max, kp.rows_max, kp.flags) == (3, 8, 7, 2, 0)
    for bad in (dict(q=mk(3, 8, 64)), dict(q=mk(3, 8, 128, dt=torch.float32)), dict(row_offsets=H.ints([0, 3])),
                dict(row_len=H.ints([5, 6])), dict(q=mk(8, 3, 128).transpose(0, 1))):
        with pytest.raises(ValueError):
            dsa.KV4Problem.from_tensors(**dict(a, **bad))
    # tensors that are not on a CUDA device, outputs of another shape or type
    ws = torch.empty(256, dtype=torch.uint8)
    for out in (mk(3, 8, 128), mk(3, 8, 64)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_kv4_attn(kp, out, None, ws)
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_kv4_append(cache, p, out, ws)
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_qk_norm_rope(p, out, out)
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_kv4_read(cache, a["row_offsets"], ok["positions"], out, None, ws)


def test_changed_cache_is_looked_over_again(dsa):
    import torch
    pages, table = torch.zeros(9, 2, 8704, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    cache = dsa.KV4Cache.from_tensors(pages=pages, table=table, page_size=64, D_k=128, D_v=128)
    kp = dsa.KV4Problem.from_tensors(cache=cache, q=torch.zeros(3, 8, 128).bfloat16(), row_offsets=H.ints([0, 1, 3]),
                                     row_len=H.ints([5, 6, 7]), softmax_scale=0.1)
    kp._on = cache._on = -1          # (as if looked over on a device)
    cache.set(B=3, table=torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="row_offsets"):
        dsa.dsa_kv4_attn(kp, torch.zeros(3, 8, 128).bfloat16(), None, torch.empty(1 << 20, dtype=torch.uint8))


def test_definitions():
    """The 64-bit definitions against what they have to satisfy."""
    import torch
    g = torch.Generator().manual_seed(1)
    x = torch.randn(50, 3, 128, generator=g, dtype=torch.float64)
    codes, scale = H.quantised(x)
    assert int(codes.min()) >= 1 and int(codes.max()) <= 15
    assert scale.to(torch.bfloat16).double().equal(scale)
    m, _ = torch.frexp(scale)
    assert (m * 16).equal((m * 16).round())
    err = (H.held(x) - x).abs()
    assert bool((err <= scale.repeat_interleave(64, -1) / 2).all())
    assert H.held(x).to(torch.bfloat16).double().equal(H.held(x)) and H.held(x).half().double().equal(H.held(x))
    pages = torch.zeros(2, 3, H.block_bytes(128, 128, 16), dtype=torch.uint8)
    H.put(pages, 1, 5, x[0], x[1], 128, 128, 16)
    k, v = H.values(pages, 128, 128, 16)
    assert k[1, 5].equal(H.held(x[0])) and v[1, 5].equal(H.held(x[1])) and not k[0].any()
    y, size = H.turned(x, None, torch.arange(50).int(), H.inv_freq(128))
    assert torch.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and y[0].equal(x[0])
    n, _ = H.turned(x, torch.ones(128), torch.zeros(50).int(), None, eps=0.0)
    assert torch.allclose((n ** 2).mean(-1), torch.ones(50, 3, dtype=torch.float64))
    # a rotated pair's product depends on the distance alone
    a, b = (H.turned(x[:1].expand(2, 3, 128), None, H.ints(p), H.inv_freq(128))[0] for p in ([3, 10], [1003, 1010]))
    assert torch.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1))
