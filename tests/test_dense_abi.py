"""dsa_dense_attn without a GPU: the struct's layout, what the host refuses, the
workspace, and the binding's checks.  Nothing is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_sparse_attention_03_gb300 as m
    return m


FAKE = 1 << 20   # never read: the calls fail before any launch


def _prob(dsa, **kw):
    base = dict(R=2, B=2, H_q=8, H_kv=2, D_k=128, D_v=128, L_max=4096, rows_max=1, L_total=8192, softmax_scale=0.1,
                q=FAKE, k=FAKE, v=FAKE, offsets=FAKE, row_offsets=FAKE, row_len=FAKE)
    base.update(kw)
    return dsa.DenseProblem(**base)


def _call(dsa, p, out=FAKE, lse=None, ws=FAKE, n=1 << 40):
    return dsa.lib().dsa_dense_attn(ctypes.byref(p.c), out, lse, ctypes.c_void_p(ws), n, None)


def test_struct_layout(dsa):
    s = dsa.dsa_dense_problem
    assert ctypes.sizeof(s) == 120 and s.L_total.offset == 32 and s.softmax_scale.offset == 64 and s.q.offset == 72


@pytest.mark.parametrize("kw,status,text", [
    (dict(R=-1), 1, b"R=-1"), (dict(R=70000), 1, b"R="), (dict(B=0), 2, b"B=0"), (dict(B=5000), 2, b"B="),
    (dict(H_q=0), 2, b"H_q"), (dict(H_q=129, H_kv=1), 2, b"H_q"), (dict(H_kv=3), 2, b"H_kv"), (dict(H_kv=0), 2, b"H_kv"),
    (dict(D_k=96), 2, b"D_k"), (dict(D_v=64), 2, b"D_k"), (dict(D_k=192, D_v=192), 2, b"D_k"),
    (dict(L_max=-1), 1, b"L_max"), (dict(rows_max=-1), 1, b"rows_max"), (dict(L_total=1 << 31), 2, b"L_total"),
    (dict(L_total=-1), 2, b"L_total"), (dict(q_stride=1000), 1, b"q_stride"), (dict(k_stride=260), 1, b"k_stride"),
    (dict(v_stride=128), 1, b"v_stride"), (dict(v_stride=-256), 1, b"v_stride"), (dict(softmax_scale=0.0), 1, b"softmax_scale"),
    (dict(softmax_scale=float("nan")), 1, b"softmax_scale"), (dict(softmax_scale=float("inf")), 1, b"softmax_scale"),
    (dict(flags=0x1), 1, b"flag"), (dict(q=None), 1, b"q/k/v/out"), (dict(k=None), 1, b"q/k/v/out"),
    (dict(v=FAKE + 8), 1, b"16-byte"), (dict(q=FAKE + 2), 1, b"16-byte"), (dict(offsets=None), 1, b"offsets"),
    (dict(row_len=None), 1, b"row_len"), (dict(row_len=FAKE + 2), 1, b"4-byte"),
])
def test_refusals(dsa, kw, status, text):
    assert _call(dsa, _prob(dsa, **kw)) == status
    assert text in dsa.lib().dsa_last_error_string()


def test_buffers_refused(dsa):
    p = _prob(dsa)
    n = dsa.dsa_dense_workspace_size(p)
    assert n % 256 == 0
    assert _call(dsa, p, out=None) == 1 and _call(dsa, p, out=FAKE + 8) == 1 and _call(dsa, p, lse=FAKE + 2) == 1
    assert _call(dsa, p, ws=FAKE + 16) == 1 and _call(dsa, p, n=n - 1) == 1
    assert b"required" in dsa.lib().dsa_last_error_string()
    assert dsa.lib().dsa_dense_workspace_size(ctypes.byref(_prob(dsa, H_kv=3).c)) == 0


def test_hook_limit_refused(dsa):
    p = _prob(dsa)
    for limit in (0, -5, 10 ** 11):
        assert dsa.lib().dsa_test_dense_missing_tile(ctypes.byref(p.c), FAKE, None, ctypes.c_void_p(FAKE), 1 << 40,
                                                     limit, None) == 1
        assert b"limit_ns" in dsa.lib().dsa_last_error_string()


def test_workspace_holds_parts_only_where_the_cache_is_split(dsa):
    base = dsa.dsa_dense_workspace_size(_prob(dsa, R=0))
    few = dsa.dsa_dense_workspace_size(_prob(dsa, R=1, B=1, L_max=65536, L_total=65536))
    assert few > base + 8 * 128 * 4
    assert dsa.dsa_dense_workspace_size(_prob(dsa, R=1, B=1, L_max=128, L_total=128)) == base
    assert dsa.dsa_dense_workspace_size(_prob(dsa, R=65535, B=1, rows_max=0, L_max=65535, L_total=65535)) == base


def test_binding_checks(dsa):
    import torch
    i = lambda *a: torch.tensor(a, dtype=torch.int32)
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    ok = dict(q=mk(2, 8, 128), k=mk(30, 2, 128), v=mk(30, 2, 128), offsets=i(0, 10, 30), row_offsets=i(0, 1, 2),
              row_len=i(10, 20), softmax_scale=0.1)
    p = dsa.DenseProblem.from_tensors(**ok)
    assert (p.R, p.B, p.H_q, p.H_kv, p.L_max, p.L_total, p.rows_max, p.flags) == (2, 2, 8, 2, 20, 30, 1, 0)
    x = mk(30, 2 * 128 * 2 + 64)
    views = dict(ok, k=x[:, :256].unflatten(1, (2, 128)),
                 v=x[:, 256:512].unflatten(1, (2, 128)))
    p = dsa.DenseProblem.from_tensors(**views)
    assert p.k_stride == p.v_stride == 576
    h = torch.float16
    p = dsa.DenseProblem.from_tensors(**dict(ok, q=mk(2, 8, 128, dt=h), k=mk(30, 2, 128, dt=h), v=mk(30, 2, 128, dt=h)))
    assert p.flags == dsa.DSA_FLAG_FP16
    for bad in (dict(q=mk(2, 8, 128, dt=h)), dict(q=mk(2, 8, 64)), dict(v=mk(30, 1, 128)), dict(v=mk(29, 2, 128)),
                dict(k=mk(30, 128, 2).transpose(1, 2)), dict(q=mk(8, 2, 128).transpose(0, 1)), dict(row_len=i(1)),
                dict(row_len=torch.tensor([10, 20])), dict(L_total=31)):
        with pytest.raises(ValueError):
            dsa.DenseProblem.from_tensors(**dict(ok, **bad))
    # tensors that are not on the current device, outputs of another shape or type
    p = dsa.DenseProblem.from_tensors(**ok)
    ws = torch.empty(256, dtype=torch.uint8)
    for out in (mk(2, 8, 128), mk(2, 8, 64), mk(2, 8, 128, dt=h), mk(8, 2, 128).transpose(0, 1)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_dense_attn(p, out, None, ws)


def test_headers_from_c(dsa, tmp_path):
    # The new headers are C99, alone and together, and lay the structs out as the binding does.
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "h.c"
    src.write_text('#include "dsa_linear.h"\n#include "dsa_dense.h"\n#include "dsa_testing.h"\n'
                   "int a[sizeof(dsa_dense_problem) == %d ? 1 : -1];\nint b[sizeof(dsa_linear_problem) == %d ? 1 : -1];\n"
                   "int main(void) { dsa_dense_problem p = {0}; return dsa_dense_workspace_size(&p) != 0; }\n"
                   % (ctypes.sizeof(dsa.dsa_dense_problem), ctypes.sizeof(dsa.dsa_linear_problem)))
    lib = os.path.dirname(dsa.LIB_PATH)
    exe = str(tmp_path / "h")
    res = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"), str(src),
                          "-o", exe, "-L", lib, "-ldsa", "-Wl,-rpath," + lib], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert subprocess.run([exe], timeout=120).returncode == 0


def test_expanded_tokens_are_refused(dsa):
    # A token stride of 0 (expand) would read as "packed" and run past the storage.
    import torch
    i = lambda *a: torch.tensor(a, dtype=torch.int32)
    one = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    ok = dict(q=one.expand(2, 2, 128).contiguous(), k=one.expand(30, 2, 128).contiguous(),
              v=one.expand(30, 2, 128).contiguous(), offsets=i(0, 30), row_offsets=i(0, 2), row_len=i(29, 30),
              softmax_scale=0.1)
    dsa.DenseProblem.from_tensors(**ok)
    wide = torch.zeros(30 * 256 + 256, dtype=torch.bfloat16)
    for bad in (dict(k=one.expand(30, 2, 128)), dict(q=one.expand(2, 2, 128)), dict(v=one.expand(30, 2, 128)),
                dict(k=wide.as_strided((30, 2, 128), (128, 128, 1)))):
        with pytest.raises(ValueError, match="overlap"):
            dsa.DenseProblem.from_tensors(**dict(ok, **bad))
    ln = dict(q=ok["k"], k=ok["k"], v=ok["v"], log_decay=torch.zeros(2), row_offsets=i(0, 30), scale=0.1)
    dsa.LinearProblem.from_tensors(**ln)
    for name in "qkv":
        with pytest.raises(ValueError, match="overlap"):
            dsa.LinearProblem.from_tensors(**dict(ln, **{name: one.expand(30, 2, 128)}))


def test_longest_cache(dsa):
    # Positions are rounded up to whole tiles in 32 bits.
    top = (1 << 31) - 256
    assert dsa.dsa_dense_workspace_size(_prob(dsa, L_total=top)) > 0
    assert _call(dsa, _prob(dsa, L_total=top + 1)) == 2
    assert b"L_total" in dsa.lib().dsa_last_error_string()
