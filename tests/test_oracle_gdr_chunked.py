"""CPU pins of the chunk form's oracle (oracle/gdr_chunked.py) against the
token-by-token one, and of the GPU tests' tolerances (tests/_gdr_bars.py): the
algebra the kernels keep passes them, planted mistakes do not.

The mistakes stand in the oracle: states, residuals or cotangents held in two
bf16 parts in place of three, and gradients of the decay with one of their
terms left out."""
import numpy as np
import pytest
import torch

from oracle.gdr import gdr_recurrent, gdr_recurrent_vjp
from oracle.gdr_chunked import DG_TERMS, gdr_chunked_vjp, growth, parts
from tests._gdr_bars import GRADS, bars, misses, misses_bf16, walk

BF = torch.bfloat16


def batch(seed, T, Hk, Hv, dk, dv, gates="usual", noise=None, beta=None, s0=True):
    """noise: keys are a common direction and so much of one of their own."""
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)      # noqa: E731
    bf = lambda x: parts(x, 1)                                          # noqa: E731
    k = unit(r.standard_normal((T, Hk, dk)))
    if noise is not None:
        k = unit(unit(r.standard_normal((1, Hk, dk))) + noise * k)
    b = dict(q=bf(unit(r.standard_normal((T, Hk, dk)))), k=bf(k), v=bf(r.standard_normal((T, Hv, dv))))
    if gates == "usual":
        b["g"] = -np.exp(r.uniform(-6, 1.5, (T, Hv)))
    elif gates == "slow":
        b["g"] = -1e-4 * r.random((T, Hv))
    else:
        b["g"] = -60 * r.random((T, Hv))
        b["g"][r.random((T, Hv)) < 0.1] = -np.inf
    b["beta"] = 1 / (1 + np.exp(-r.standard_normal((T, Hv)))) if beta is None else np.full((T, Hv), beta)
    b["dO"] = bf(r.standard_normal((T, Hv, dv)))
    b["scale"] = dk ** -0.5
    b["S0"] = 0.3 * r.standard_normal((Hv, dk, dv)) if s0 else None
    b["dS_T"] = 0.3 * r.standard_normal((Hv, dk, dv)) if s0 else None
    return b


def chunked(b, **kw):
    return gdr_chunked_vjp(*(b[x] for x in ("q", "k", "v", "g", "beta", "dO", "scale", "S0", "dS_T")), **kw)


def tokens(b):
    return (gdr_recurrent(*(b[x] for x in ("q", "k", "v", "g", "beta", "scale", "S0"))),
            gdr_recurrent_vjp(*(b[x] for x in ("q", "k", "v", "g", "beta", "dO", "scale", "S0", "dS_T"))))


@pytest.mark.parametrize("C", [32, 64])
@pytest.mark.parametrize("T,Hk,Hv,gates,s0", [(130, 2, 4, "usual", True), (63, 1, 3, "slow", True),
                                              (200, 1, 1, "fast", False), (1, 1, 2, "usual", True)])
def test_equals_the_recurrence(T, Hk, Hv, gates, s0, C):
    b = batch(T, T, Hk, Hv, 16, 24, gates, s0=s0)
    fwd, grads, _ = chunked(b, C=C)
    rf, rg = tokens(b)
    for x, y in zip(fwd + grads, rf + rg):
        assert np.linalg.norm(x - y) <= 1e-12 * max(np.linalg.norm(y), 1e-30)


def outputs(b, dtype=BF, **kw):
    """The outputs that miss their tolerances."""
    (o, S), grads, _ = chunked(b, **kw)
    rf, rg = tokens(b)
    _, _, norms = chunked(b)
    T, dk, dv = b["v"].shape[0], b["k"].shape[2], b["v"].shape[2]
    tol = bars(dtype, dk, dv, T, growth([norms]))
    got = dict(zip(GRADS, grads), S_T=S)
    return {x for x, y in zip(("S_T",) + GRADS[3:], (rf[1],) + rg[3:]) if misses(got[x], y, tol[x])}


def test_parts():
    x = np.random.default_rng(0).standard_normal(1000)
    left = [np.abs(parts(x, n) / x - 1).max() for n in (1, 2, 3)]
    assert left[0] <= 2.0 ** -8 and left[1] <= 2.0 ** -16 and left[2] <= 2.0 ** -24
    assert parts(x, None) is x


@pytest.mark.parametrize("T", [700, 1500])
def test_three_parts_pass_and_two_do_not(T):
    """Few chains with slow decays, where a state's error lasts longest."""
    b = batch(T, T, 1, 1, 128, 128, "slow")
    assert outputs(b, held={x: 3 for x in ("S", "L", "U", "Yb")}) == set()
    assert {"S_T", "dbeta"} <= outputs(b, held={"S": 2})
    assert {"dS0", "dbeta"} <= outputs(b, held={"L": 2})
    assert {"S_T", "dS0", "dbeta"} <= outputs(b, held={"S": 2, "L": 2, "U": 2})


@pytest.mark.parametrize("gates,T,d,dscale,held", [("usual", 300, 64, 1, "U"), ("usual", 700, 128, 1, "U"),
                                                   ("fast", 300, 64, 1, "U"), ("slow", 300, 64, 2.0 ** -10, "Yb")])
def test_two_parts_show_in_dg(gates, T, d, dscale, held):
    """Yb where the final state's cotangent is the larger one."""
    b = batch(3, T, 1, 1, d, d, gates)
    b["dO"] *= dscale
    assert outputs(b) == set()
    assert outputs(b, held={held: 2}) == {"dg"}


@pytest.mark.parametrize("gates,noise,beta", [("usual", None, None), ("slow", None, None), ("slow", 0.1, 0.9)])
def test_a_dg_without_one_of_its_terms_is_rejected(gates, noise, beta):
    b = batch(5, 200, 1, 2, 128, 128, gates, noise, beta)
    assert outputs(b) == set()
    for name in DG_TERMS:
        assert outputs(b, drop=(name,)) == {"dg"}, name


def test_growth_of_nearly_repeated_keys():
    """Rows that nearly repeat grow dg's terms to several times dg and F to
    several times Ub: far from the thousands of exactly repeated keys, whose
    dg no arithmetic in fp32 knows."""
    _, _, n = chunked(batch(8, 200, 1, 2, 128, 128, "slow", 0.1, 0.9, s0=False))
    gr = growth([n])
    assert 2 < gr["dg"] < 40 and 1.5 < gr["F"] < 10
    assert growth([]) == {"Y": 1.0, "F": 1.0, "dg": 1.0}


def test_what_the_tolerances_come_to():
    """At the largest heads: below 6e-7 for states in chunks, below 1.5e-6
    token by token.  A rounding to bf16 passes, a truncation does not."""
    assert 2 * walk(BF, 128, 128, 10 ** 6) < 6e-7 and 2 * walk(torch.float32, 128, 128, 10 ** 6) < 1.5e-6
    x = np.random.default_rng(1).standard_normal((64, 128))
    assert misses_bf16(parts(x, 1), x) is None
    cut = (x.astype(np.float32).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
    assert misses_bf16(cut, x)
    assert misses_bf16(parts(x * (1 + 2.0 ** -9), 1), x)
