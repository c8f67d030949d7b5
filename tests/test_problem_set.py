"""Fields of a dense or linear problem changed by ``set``: what no longer fits is refused before
anything is launched."""
import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_sparse_attention_03_gb300 as m
    return m


def _dense(dsa):
    import torch
    i = lambda *a: torch.tensor(a, dtype=torch.int32)
    mk = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    return dsa.DenseProblem.from_tensors(q=mk(2, 8, 128), k=mk(30, 2, 128), v=mk(30, 2, 128), offsets=i(0, 10, 30),
                                         row_offsets=i(0, 1, 2), row_len=i(10, 20), softmax_scale=0.1)


def _linear(dsa):
    import torch
    mk = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    return dsa.LinearProblem.from_tensors(q=mk(30, 4, 64), k=mk(30, 4, 64), v=mk(30, 4, 128), scale=0.1,
                                          log_decay=torch.zeros(4), row_offsets=torch.tensor([0, 10, 30], dtype=torch.int32))


def _call(dsa, p):
    import torch
    ws = torch.empty(256, dtype=torch.uint8)
    if isinstance(p, dsa.DenseProblem):
        dsa.dsa_dense_attn(p, torch.zeros(p.R, p.H_q, p.D_v, dtype=torch.bfloat16), None, ws)
    else:
        out = torch.zeros(p.R, p.H, p.D_v, dtype=torch.bfloat16)
        dsa.dsa_linear_attn(p, None, torch.zeros(p.n_states, p.H, p.D_k, p.D_v), out, ws)


def test_what_does_not_fit_is_refused(dsa):
    import torch
    mk = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    for make, cases in (
            (_dense, (dict(q=mk(1, 8, 128)), dict(k=mk(29, 2, 128)), dict(v=mk(30, 2, 64)), dict(q=mk(2, 4, 128)),
                      dict(k=mk(30, 4, 128)[:, ::2]), dict(k=mk(30, 2, 256)[:, :, :128]), dict(k=mk(60, 2, 128)[::2]),
                      dict(q=mk(2, 8, 128, dt=torch.float16)), dict(row_len=i32(1)), dict(offsets=i32(2)),
                      dict(row_len=torch.zeros(2)), dict(R=3), dict(L_total=31), dict(B=3), dict(H_q=16),
                      dict(flags=dsa.DSA_FLAG_FP16), dict(k_stride=512))),
            (_linear, (dict(q=mk(29, 4, 64)), dict(v=mk(30, 4, 64)), dict(k=mk(60, 4, 64)[::2]), dict(R=31),
                       dict(log_decay=torch.zeros(3)), dict(log_decay=torch.zeros(4, dtype=torch.float64)),
                       dict(state_idx=i32(1)), dict(row_offsets=i32(2)), dict(B=3), dict(D_k=128),
                       dict(k=mk(30, 4, 64, dt=torch.float16))))):
        for kw in cases:
            p = make(dsa).set(**kw)
            for _ in range(2):             # (and again: a refused call leaves nothing behind)
                with pytest.raises(ValueError) as e:
                    _call(dsa, p)
                assert "device" not in str(e.value), (kw, str(e.value))


def test_what_fits_is_taken(dsa):
    # As far as the check of the devices, which nothing here passes.
    import torch
    mk = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    for make, cases in ((_dense, (dict(), dict(q=mk(2, 8, 128)), dict(k=mk(64, 2, 128)), dict(rows_max=7), dict(R=1, B=1),
                                  dict(k=mk(30, 2, 256).view(30, 4, 128)[:, :2], k_stride=512))),
                        (_linear, (dict(), dict(v=mk(30, 4, 128)), dict(state_idx=torch.zeros(2, dtype=torch.int32), n_states=5),
                                   dict(rows_max=30)))):
        for kw in cases:
            with pytest.raises(ValueError, match="device"):
                _call(dsa, make(dsa).set(**kw))
