"""dsa_linear_attn and dsa_linear_step without a GPU: the struct's layout, what the
host refuses, the workspace, and the binding's checks.  Nothing is launched."""
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
    base = dict(R=2, B=2, H=4, D_k=128, D_v=64, rows_max=1, n_states=2, scale=0.1, q=FAKE, k=FAKE, v=FAKE,
                log_decay=FAKE, row_offsets=FAKE)
    base.update(kw)
    return dsa.LinearProblem(**base)


def _call(dsa, p, step=False, sin=FAKE, sout=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
    f = dsa.lib().dsa_linear_step if step else dsa.lib().dsa_linear_attn
    return f(ctypes.byref(p.c), sin, sout, out, ctypes.c_void_p(ws), n, None)


def test_struct_layout(dsa):
    s = dsa.dsa_linear_problem
    assert ctypes.sizeof(s) == 112 and s.q_stride.offset == 32 and s.scale.offset == 56 and s.q.offset == 64


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("kw,status,text", [
    (dict(R=-1), 1, b"R=-1"), (dict(B=0), 2, b"B=0"), (dict(B=5000), 2, b"B="), (dict(H=0), 2, b"H=0"),
    (dict(H=257), 2, b"H=257"), (dict(D_k=96), 2, b"D_k"), (dict(D_v=256), 2, b"D_v"), (dict(rows_max=-2), 1, b"rows_max"),
    (dict(n_states=-1), 1, b"n_states"), (dict(q_stride=64), 1, b"q_stride"), (dict(k_stride=516), 1, b"k_stride"),
    (dict(v_stride=-8), 1, b"v_stride"), (dict(scale=float("nan")), 1, b"scale"), (dict(flags=0x2), 1, b"flag"),
    (dict(q=None), 1, b"q/k/v/out"), (dict(k=FAKE + 8), 1, b"16-byte"), (dict(log_decay=None), 1, b"log_decay"),
    (dict(log_decay=FAKE + 2), 1, b"4-byte"), (dict(state_idx=FAKE + 1), 1, b"4-byte"),
])
def test_refusals(dsa, kw, status, text, step):
    assert _call(dsa, _prob(dsa, **kw), step) == status
    assert text in dsa.lib().dsa_last_error_string()


def test_buffers_refused(dsa):
    p = _prob(dsa)
    n = dsa.dsa_linear_workspace_size(p)
    assert n == 256
    for step in (False, True):
        assert _call(dsa, p, step, out=None) == 1 and _call(dsa, p, step, out=FAKE + 2) == 1
        assert _call(dsa, p, step, sin=FAKE + 4) == 1 and _call(dsa, p, step, sout=FAKE + 8) == 1
        assert _call(dsa, p, step, ws=FAKE + 16) == 1 and _call(dsa, p, step, n=n - 1) == 1
        assert _call(dsa, p, step, sin=FAKE, sout=FAKE + 4096) == 1
        assert b"overlap" in dsa.lib().dsa_last_error_string()
    assert _call(dsa, _prob(dsa, row_offsets=None)) == 1 and b"row_offsets" in dsa.lib().dsa_last_error_string()
    assert _call(dsa, _prob(dsa, R=3), step=True) == 1 and b"one token" in dsa.lib().dsa_last_error_string()
    assert _call(dsa, p, step=True, sout=None) == 1 and b"state_out" in dsa.lib().dsa_last_error_string()


def test_workspace_holds_segment_states_only_for_long_requests(dsa):
    long = dsa.dsa_linear_workspace_size(_prob(dsa, R=60000, B=1, rows_max=60000))
    assert long > 256 + 4 * 128 * 64 * 4
    assert dsa.dsa_linear_workspace_size(_prob(dsa, R=60000, B=4000, rows_max=20)) == 256


def test_binding_checks(dsa):
    import torch
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    ro = torch.tensor([0, 10, 30], dtype=torch.int32)
    ok = dict(q=mk(30, 4, 64), k=mk(30, 4, 64), v=mk(30, 4, 128), log_decay=torch.zeros(4), row_offsets=ro, scale=0.1)
    p = dsa.LinearProblem.from_tensors(**ok)
    assert (p.R, p.B, p.H, p.D_k, p.D_v, p.rows_max, p.n_states, p.flags) == (30, 2, 4, 64, 128, 20, 2, 0)
    assert dsa.LinearProblem.from_tensors(**dict(ok, row_offsets=None)).B == 30
    x = mk(30, 4 * 256 + 8)
    p = dsa.LinearProblem.from_tensors(**dict(ok, q=x[:, :256].unflatten(1, (4, 64))))
    assert p.q_stride == 1032
    h = torch.float16
    for bad in (dict(q=mk(30, 4, 64, dt=h)), dict(k=mk(30, 4, 128)), dict(v=mk(30, 5, 128)), dict(v=mk(29, 4, 128)),
                dict(log_decay=torch.zeros(3)), dict(log_decay=torch.zeros(4, dtype=torch.float64)),
                dict(row_offsets=ro.long()), dict(state_idx=torch.zeros(2, dtype=torch.int32)),
                dict(state_idx=torch.zeros(3, dtype=torch.int32), n_states=4), dict(q=mk(30, 64, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            dsa.LinearProblem.from_tensors(**dict(ok, **bad))
    p = dsa.LinearProblem.from_tensors(**ok)
    ws, st = torch.empty(256, dtype=torch.uint8), torch.zeros(2, 4, 64, 128)
    for s_, o in ((st, mk(30, 4, 128)), (torch.zeros(2, 4, 128, 64), mk(30, 4, 128)), (st, mk(30, 4, 64))):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dsa.dsa_linear_attn(p, None, s_, o, ws)
