"""How dsa_dense_attn cuts its work, as far as the host's workspace shows it.  Nothing is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_sparse_attention_03_gb300 as m
    return m


def parts(dsa, **kw):
    """Parts that each row of a split call leaves in the workspace (1: not split)."""
    base = dict(R=32, B=32, H_q=64, H_kv=8, D_k=128, D_v=128, L_max=8000, rows_max=1, L_total=32 * 8000,
                softmax_scale=0.1)
    base.update(kw)
    size = lambda **over: dsa.lib().dsa_dense_workspace_size(ctypes.byref(dsa.DenseProblem(**dict(base, **over)).c))
    n = (size() - size(R=0)) // (base["R"] * base["H_q"] * (base["D_v"] + 2) * 4)
    return max(1, n)


@pytest.mark.parametrize("longest", [5000, 6144, 8000])
@pytest.mark.parametrize("requests", [32, 64])
def test_ragged_single_tokens_below_8192_positions_are_split(dsa, longest, requests):
    # One long request among short ones: walked in one part it would end last, alone.
    n = parts(dsa, R=requests, B=requests, L_max=longest, L_total=longest + 100 * (requests - 1))
    assert n == longest // (16 * 128) + (longest % (16 * 128) > 15 * 128)
    assert n == parts(dsa, R=requests, B=requests, L_max=longest, L_total=longest * requests)   # (however the cache is laid out)


def test_single_tokens_that_are_not_split(dsa):
    assert parts(dsa, R=64, B=64, L_max=4096, L_total=64 * 4096) == 1


def test_declared_bounds_above_what_the_call_holds(dsa):
    # L_max and rows_max are upper bounds: the largest int32 (2^31 tiles of positions past 32
    # bits) cuts the work as the true values do.
    top = (1 << 31) - 1
    for kw in (dict(R=1, B=1, L_total=32768), dict(R=32, B=32, L_total=8000), dict(R=700, B=1, rows_max=0, L_total=700),
               dict(R=4, B=2, H_q=8, H_kv=8, rows_max=2, L_total=20000)):
        n = parts(dsa, L_max=kw["L_total"], **kw)
        assert parts(dsa, L_max=top, **kw) == n
        if kw.get("rows_max") != 0:
            assert parts(dsa, **dict(kw, L_max=top, rows_max=kw["R"])) == parts(dsa, **dict(kw, L_max=top, rows_max=top))
    assert parts(dsa, R=1, B=1, L_total=32768, L_max=top) > 10
