"""Paged cache, attention: rows all of whose scores are -inf because of infinite
keys.  They see something, so their softmax is NaN by definition; only rows that see
nothing are 0.  Where one score is finite the infinite ones have weight 0."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle
from tests import kv_cases
from tests.test_gpu_kv_attention import bounds
from tests.test_gpu_kv_edges import on_gpu, status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("S", [1, 5, 10, 20, 40, 300])
def test_rows_of_minus_infinity_are_nan(S, window):
    rng = np.random.default_rng(330)
    # every key of the first (long: joined from many parts) and the second sequence,
    # the newest keys of the third, one in the middle of the fourth; the last two
    # have rows in front of their first token
    lens, d, block = [5000, 1, 400 + S, 400 + S, max(1, S - 2)], 64, 32
    new = [S, 1, S, S, S]
    t, ref, table = kv_cases.rand_cache(rng, lens, 2, d, block, False)
    finite = {n: x.copy() for n, x in ref.items()}
    first = {0: 0, 1: 0, 2: 396, 3: 200}
    for b, lo in first.items():
        for p in range(lo, 201 if b == 3 else lens[b]):
            blk = int(table[b, p // block])
            t["k_cache"][blk, 0, p % block, 3] = float("inf")
            ref["k"][blk, 0, p % block, 3] = np.inf
            finite["k"][blk, 0, p % block, 3] = 0.0
    q = kv_cases.bf16(rng, (5, 4, S, d))
    q[:, :, :, 3] = -q[:, :, :, 3].abs() - 0.5               # scores -inf
    q[2, 1, S - 1, 3] = 2.0                                  # +inf: NaN in any case
    out, lse = on_gpu(t, table, lens, q, new, window)()
    status_ok()
    with np.errstate(invalid="ignore"):
        want, wlse, spread = kv_oracle.attention(q.double().numpy(), ref, table, lens, new, window)
    tol, eps = bounds(q.double().numpy(), finite, spread, want, lens, False)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(want[0, :2]).all() and np.isnan(want[1, :2, 0]).all()
    assert not np.isnan(want[0, 2:, 0]).any() and not np.isnan(want[4]).any()
    for b in range(5):
        f = new[b]
        w, g, wl, gl = want[b, :, :f], got[b, :, :f], wlse[b, :, :f], glse[b, :, :f]
        assert np.array_equal(np.isnan(g), np.isnan(w)), b
        assert np.array_equal(np.isnan(gl), np.isnan(wl)), b
        ok = ~np.isnan(w)
        assert (np.abs(g - w)[ok] <= tol[b, :, :f][ok]).all()
        gone = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), gone)
        ok = ~gone & ~np.isnan(wl)
        assert (np.abs(gl[ok] - wl[ok]) <= eps + 2.0 ** -22 * np.abs(wl[ok])).all()
