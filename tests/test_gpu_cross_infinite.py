"""Cross attention with infinities among the states, against a float64 softmax.

A score of minus infinity has weight 0 wherever it stands: a whole first tile,
a part of split states, the last state.  A row with a score of plus infinity,
and one whose scores are all minus infinity, is NaN (inf - inf).  Rows that
the formula leaves finite keep the tolerance of tests/test_gpu_cross.py; its
term for the error of the finite scores is taken over the finite products.
"""

import pytest
import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_gpu_cross import BF16, F16, F32, FP8, Case, half

pytestmark = pytest.mark.gpu

INF = float("inf")


def definition(c, s, pool):
    """(out, tolerance) of sequence s over the pool's values (float64)."""
    n, b, G = c.lens[s], c.b, c.H // c.Hk
    q = c.q[c.starts[s]:c.starts[s + 1]].double().transpose(0, 1)
    blk = c.tables[s, :-(-n // b)].long()
    k, v = (x[blk].permute(1, 0, 2, 3).reshape(c.Hk, -1, c.D)[:, :n].repeat_interleave(G, 0)
            for x in pool)
    p = torch.softmax(q @ k.transpose(1, 2) * c.scale, dim=2)
    out, mass = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
    finite = torch.where(torch.isfinite(k), k, 0.0)
    dz = (q.abs() @ finite.abs().transpose(1, 2)).amax(2) * abs(c.scale) * (c.D + 4) * 2.0 ** -24
    hp = 0.0 if c.dtype == F32 or (c.dtype == FP8 and c.D == 64) else \
        half(F16 if c.dtype == FP8 else c.dtype)
    rel = hp + 2 * dz.t()[..., None] + 2.0 ** -20 + 2 * (n + 16) * 2.0 ** -24
    tol = half(c.io) * out.abs() + mass * rel * (1 + half(c.io)) + \
        torch.finfo(c.io).smallest_normal * torch.finfo(c.io).eps
    return out, tol


def check(c, out):
    """The finite elements within their tolerance; the others equal (NaN where
    the definition has NaN, infinities with their sign)."""
    out, pool = out.detach().cpu(), []
    for x, sc in zip(c.kv, (c.ks, c.vs)):
        x = x.float().double()
        pool.append(x if sc is None else x * sc.double()[None, :, None, None])
    for s in range(len(c.lens)):
        if c.lens[s] == 0:
            continue
        ref, tol = definition(c, s, pool)
        got = out[c.starts[s]:c.starts[s + 1]].double()
        fine = torch.isfinite(ref)
        err = (got - ref).abs()[fine]
        assert (err <= tol[fine]).all(), (s, float(err.max()))      # (a NaN fails here)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), s
        assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), s
    assert pkv.paged_get_device_error() == 0


def plant(c, which, s, where, value, dim=0):
    """``value`` in element ``dim`` of states ``where`` of sequence s."""
    t = torch.as_tensor(list(where))
    c.kv[which][c.tables[s].long()[t // c.b], :, t % c.b, dim] = value


def positive(c):
    """Queries whose element 0 is positive: an infinity there in a key makes
    a score of its sign."""
    c.q[..., 0] = c.q[..., 0].abs() + 0.25


POOLS = [(F16, 64), (F16, 128), (BF16, 64), (BF16, 128), (F32, 64), (F32, 128)]
# states with a score of minus infinity, of (states, queries): the first tile of
# 64, more than it, a lone state in a part of its own, a whole part of several,
# the last states, all but one state, every other one
WHERE = [(200, 3, range(64)), (200, 130, range(64)), (200, 3, range(150)), (129, 1, [128]),
         (129, 40, [128]), (65, 2, [64]), (1000, 1, range(256, 384)), (1000, 2, range(0, 900)),
         (200, 5, range(190, 200)), (77, 3, range(76)), (77, 3, range(1, 77)),
         (300, 9, range(0, 300, 2)), (1, 2, [])]


@pytest.mark.parametrize("dtype,D", POOLS)
@pytest.mark.parametrize("n,Q,where", WHERE, ids=lambda x: str(x) if isinstance(x, int) else str(len(x)))
def test_scores_of_minus_infinity_weigh_nothing(dtype, D, n, Q, where):
    c = Case([Q, 2], [n, 50], 4, 2, D, dtype, seed=n + Q)
    positive(c)
    if len(where):
        plant(c, 0, 0, where, -INF)
    out = c.call()
    assert torch.isfinite(out).all()
    check(c, out)


@pytest.mark.parametrize("dtype,D", POOLS)
@pytest.mark.parametrize("n,Q", [(1, 1), (40, 3), (64, 2), (129, 1), (200, 130), (1000, 2)])
def test_a_row_of_minus_infinities_alone_is_nan(dtype, D, n, Q):
    """0 / 0, in one part or in several."""
    c = Case([Q, 2], [n, 50], 4, 2, D, dtype, seed=n)
    positive(c)
    plant(c, 0, 0, range(n), -INF)
    out = c.call()
    assert torch.isnan(out[:Q]).all()
    check(c, out)


@pytest.mark.parametrize("dtype,D", POOLS)
@pytest.mark.parametrize("n,Q,where", [(200, 6, [3]), (200, 6, [199]), (129, 1, [128]), (1000, 2, [500]),
                                       (64, 40, range(64))])
def test_infinite_keys_of_either_sign(dtype, D, n, Q, where):
    """Queries of both signs: rows with a score of plus infinity are NaN, the
    others lose the state."""
    c = Case([Q, 2], [n, 50], 8, 2, D, dtype, seed=n + Q + 1)
    plant(c, 0, 0, where, INF)
    check(c, c.call())


@pytest.mark.parametrize("dtype,D", POOLS)
@pytest.mark.parametrize("n,Q", [(60, 3), (129, 1), (1000, 2)])
def test_infinite_values(dtype, D, n, Q):
    """They reach their element of every row with their sign, and NaN where
    both meet."""
    c = Case([Q, 2], [n, 50], 4, 2, D, dtype, seed=n + 2)
    plant(c, 1, 0, [n // 2], INF, 5)
    plant(c, 1, 0, [n - 1], -INF, 7)
    plant(c, 1, 0, [0, n - 1], INF, 9)
    plant(c, 1, 0, [1], INF, 11)
    plant(c, 1, 0, [n - 2], -INF, 11)
    out = c.call()
    assert (out[:Q, :, 5] == INF).all() and (out[:Q, :, 7] == -INF).all()
    assert torch.isnan(out[:Q, :, 11]).all()
    check(c, out)


@pytest.mark.parametrize("dtype,D", POOLS)
@pytest.mark.parametrize("n,where", [(200, range(64)), (1000, range(128, 256)), (129, [128])])
@pytest.mark.parametrize("value", [INF, float("nan")])
def test_a_value_that_is_not_finite_under_a_weight_of_zero(dtype, D, n, where, value):
    """0 times it is NaN, in its own tile or in a part that weighs nothing."""
    c = Case([2, 2], [n, 50], 4, 2, D, dtype, seed=n + 3)
    positive(c)
    plant(c, 0, 0, where, -INF)
    plant(c, 1, 0, [list(where)[-1]], value, 3)
    out = c.call()
    assert torch.isnan(out[:2, :, 3]).all()
    check(c, out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [70, 1000])
def test_a_query_that_is_not_finite_over_an_fp8_pool(D, n):
    """It makes its own row NaN and no other."""
    c = Case([3, 2], [n, 50], 4, 2, D, FP8, BF16, seed=n)
    c.q[1, 2, 4] = INF
    out = c.call()
    assert torch.isnan(out[1, 2]).all()
    out[1, 2] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64)])
def test_a_bad_table_is_zeroes_whatever_the_states_hold(dtype, D):
    """Split states: every part of the row is zeroed, none is NaN."""
    c = Case([2, 1], [1000, 900], 4, 2, D, dtype, seed=4)
    positive(c)
    plant(c, 0, 0, range(1000), -INF)
    c.tables[0, 40] = -1
    out = c.call()
    assert pkv.paged_get_device_error() == pkv.PKV_DEV_TABLE_RANGE
    assert (out[:2] == 0).all() and torch.isfinite(out).all()
