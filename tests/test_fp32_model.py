"""The fp32 bounds tell a lost rounding or a sum that is not folded from what is there: the
mistakes are made here, in sums of 7200 terms formed in fp32 on the host."""
import math

import numpy as np
import pytest

import fp32_model as M

N, D = 7200, 64


def fma32(acc, a, b):
    """a b + acc rounded once to fp32 (the product is exact in 64 bits)."""
    return (acc.astype(np.float64) + a.astype(np.float64) * b).astype(np.float32)


def add_up(p, v, fold):
    """sum_u p_u v_u, one after another; with `fold`, that many terms apart and then to the
    total."""
    total, acc = np.zeros(v.shape[1:], np.float32), np.zeros(v.shape[1:], np.float32)
    for u in range(len(v)):
        acc = fma32(acc, p[u], v[u])
        if fold and (u + 1) % fold == 0:
            total, acc = (total + acc).astype(np.float32), np.zeros_like(acc)
    return (total + acc).astype(np.float32) if fold else acc


@pytest.fixture(scope="module")
def terms():
    rng = np.random.default_rng(0)
    p = np.exp(rng.standard_normal((N, 1)) * 0.25).astype(np.float32)
    v = rng.standard_normal((N, 4000)).astype(np.float32)
    return p, v, (p.astype(np.float64) * v).sum(0)


def off(x, want):
    return np.linalg.norm(x - want) / np.linalg.norm(want)


def bounds():
    z = 0.25 * 1.4427
    return M.forward(N, D, z), M.gradient(N, D, z, math.log2(N))


def test_folded_sums_are_within_the_bounds(terms):
    p, v, want = terms
    forward, gradient = bounds()
    assert 1.2 * off(add_up(p, v, 512), want) <= forward
    assert 1.2 * off(add_up(p, v, 64), want) <= gradient


def test_a_running_sum_is_not(terms):
    p, v, want = terms
    running = off(add_up(p, v, 0), want)
    assert all(running >= 1.2 * b for b in bounds()), (running, bounds())


@pytest.mark.parametrize("n", [64, 500, N])
def test_an_operand_of_13_bits_is_not(terms, n):
    p, v, _ = terms
    p, v = p[:n], v[:n]
    want = (p.astype(np.float64) * v).sum(0)
    m, e = np.frexp(v)
    short = np.ldexp(np.round(np.ldexp(m, 13)), e - 13)
    lost = off((p.astype(np.float64) * short).sum(0), want)
    assert lost >= M.LOST
    for z in (0.36, 1.5, 3.0):
        assert 4 * M.forward(n, 128, z) <= M.LOST and 4 * M.gradient(n, 128, z, 20.0) <= M.LOST
