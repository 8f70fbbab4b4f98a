"""Cosines and sines at any position to the bound that the header states, against angles reduced
in integers of 300 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_310_gb300 as pkv
import step_model as model

pytestmark = pytest.mark.gpu

BITS = 300


def pi_bits():
    """pi * 2^BITS, by 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inverse(n):
        one = 1 << (BITS + 20)
        total, term, i = 0, one // n, 1
        while term:
            total += term // i if i % 4 == 1 else -(term // i)
            term //= n * n
            i += 2
        return total
    return (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 20


def turn_of(position, frequency):
    """The angle position * frequency in radians, whole turns taken off, from -pi to pi."""
    top, bottom = float(frequency).as_integer_ratio()
    whole = 2 * pi_bits()                                    # a turn
    angle = (position * top << BITS) // bottom % whole
    if angle > whole // 2:
        angle -= whole
    return math.ldexp(float(angle >> (BITS - 100)), -100)


# The stated angle: 2^-28 + 2^-31 turns.  sincospi: two steps of 2^-24 for values up to 1.
TOL = 2 * math.pi * (2.0 ** -28 + 2.0 ** -31) + 2 * 2.0 ** -24


def test_the_reduction_itself():
    for p, f in ((0, 1.0), (1, 1.0), (7, 0.25), (123_456, 10000.0 ** -0.3)):
        want = math.remainder(p * f, 2 * math.pi)
        assert abs(turn_of(p, f) - want) < 1e-10


@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines_at_any_position(interleaved):
    rng = np.random.default_rng(316_300)
    pos = np.concatenate([[0, 1, 2, 3, 1 << 20, (1 << 24) + 1, 1 << 30, (1 << 31) - 1], rng.integers(0, 1 << 31, 100),
                          rng.integers(0, 1 << 20, 92)])
    freq = np.concatenate([[1.0, 0.5, 1 / 3, math.pi / 4, 1e-9], rng.random(11), model.frequencies(32, 1e6)])
    q = torch.zeros(len(pos), 1, 64)
    if interleaved:
        q[..., ::2] = 1
    else:
        q[..., :32] = 1
    out, none = torch.empty_like(q, device="cuda"), torch.empty(len(pos), 0, 64, device="cuda")
    pkv.paged_qk_rotary(q.cuda(), none, torch.tensor(pos, dtype=torch.int32).cuda(), out, none, torch.tensor(freq).cuda(),
                        interleaved=interleaved)
    got = out.cpu().double().numpy()[:, 0]
    c, s = (got[:, ::2], got[:, 1::2]) if interleaved else (got[:, :32], got[:, 32:])
    angle = np.array([[turn_of(int(p), f) for f in freq] for p in pos])
    assert np.abs(c - np.cos(angle)).max() <= TOL and np.abs(s - np.sin(angle)).max() <= TOL
    assert pkv.device_error() == 0
