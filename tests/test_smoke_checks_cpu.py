"""The smoke step's own arithmetic without a GPU: what its checks let through and what they stop,
against tests/step_model.py and sums written out."""
import numpy as np
import pytest

import __graft_entry__ as entry
import step_model as model


def test_an_error_that_is_not_a_number_stops():
    want = np.ones((3, 4))
    assert entry.error("x", want + 0.001, want, 0.002) == pytest.approx(0.001)
    for bad in (np.nan, np.inf, -np.inf, 1.0021):
        got = want.copy()
        got[1, 2] = bad
        with pytest.raises(RuntimeError):
            entry.error("x", got, want, 0.002)
    with pytest.raises(RuntimeError):
        entry.error("x", want[:1], want, 0.002)           # not one row in the place of three


def test_a_value_may_be_off_by_its_own_rounding():
    want = np.array([100.0, 1.0])
    assert entry.error("x", want * (1 + 2.0 ** -9), want, 0.0, 2.0 ** -8) > 0
    with pytest.raises(RuntimeError):
        entry.error("x", want + 0.1, want, 0.0, 2.0 ** -8)


def test_rotation():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((7, 3, 64)), rng.integers(0, 5000, 7)
    for dim in (64, 32):
        f = model.frequencies(dim)
        want = model.turn(x, pos, f, False)[0]
        got = entry.rotated(x, pos, f)
        assert np.allclose(got, want, atol=1e-12)
        # nothing turned, another angle, a pair the other way round: each stops the step
        for wrong in (x, entry.rotated(x, pos + 1, f), entry.rotated(x, -pos, f)):
            with pytest.raises(RuntimeError):
                entry.error("x", wrong, want, 2e-5, 2.0 ** -8)


@pytest.mark.parametrize("n,m,window,sinks", [(50, 50, 7, 3), (40, 5, 1, 0), (30, 30, 100, 0), (64, 1, 16, 16), (45, 9, 4, 40)])
def test_windowed_attention(n, m, window, sinks):
    rng = np.random.default_rng(n + window)
    q, k, v = rng.standard_normal((m, 4, 8)), rng.standard_normal((n, 2, 8)), rng.standard_normal((n, 2, 8))
    got = entry.windowed(q, k, v, 0.3, window, sinks)
    want = np.zeros(q.shape)
    for i in range(m):
        seen = model.seen(n - m + i, window, sinks)
        for h in range(4):
            e = [np.exp(0.3 * float(q[i, h] @ k[j, h // 2])) for j in seen]
            want[i, h] = sum(w * v[j, h // 2] for w, j in zip(e, seen)) / sum(e)
    assert entry.error("x", got, want, 1e-12) >= 0
    if window < n and (sinks < n - window):                 # a token too many or too few shows
        for other in (entry.windowed(q, k, v, 0.3, window + 1, sinks), entry.windowed(q, k, v, 0.3, window, sinks + 1)):
            with pytest.raises(RuntimeError):
                entry.error("x", other, want, 2e-3)
