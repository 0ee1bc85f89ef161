"""Tolerances of the gated delta rule's outputs, from the arithmetic that the
kernels keep, and the comparison that applies them.

An operation in fp32 rounds by at most 2^-24 of its value; over random values
the rounding's standard deviation is 2^-24 / sqrt 3.  The roundings that reach
an element of a state, counted along what it remembers:
- in chunks of 64 (bf16 inputs, d_k, d_v >= 64), where operands are held in
  three bf16 parts (24 bits): a row of residuals has 3 d_k / 32 accumulations
  of K S, 3 operations on top and 3 x 6 accumulations of the substitution; a
  chunk's update is one decay and 6 accumulations; the delta rule rewrites a
  key direction about every d_k / beta tokens, so a state remembers some
  min(T, 2 d_k) tokens.  d_k = 128: 33 + 7 (4 + 1) = 68;
- token by token (fp32, small heads): 3 operations a pair of tokens and some 20
  in a residual.  d_k = 128: 20 + 1.5 * 256 = 404.
A decay factor is one such rounding, to either side as often.
Their random walk is e = sqrt(count) 2^-24 / sqrt 3 (2.8e-7, 6.9e-7); twice
that is allowed, for walks that are not quite random:
- S_T, o in fp32: 2 e, times the size of the rows that a residual is the
  difference of over the residual's ("Y");
- dS0, and dv in fp32: the same of the reverse sweep ("F" in place of "Y");
- dbeta = Ub . R, and dq, dk in fp32, which are products of two such: 2 sqrt 2 e
  times the larger of the two growths;
- dg: as dbeta, times the size of the terms that it is a sum of over its own
  ("dg").
The growths come from the fp64 oracle (oracle/gdr_chunked.py); on the usual
inputs they are 1 to 2.  One element is off by at most 40 times the 2-norm's
tolerance, of the rms or of itself (5 deviations, 8 for tails).

An output in bf16 is rounded once, by 2^-8 of its value at most and 2^-8 /
sqrt 3 in the rms; before that it comes from operands held in two parts at
least (2^-16), some of three: an element is off by its half step and at most
2^-11 of the rms or of itself.
"""
import numpy as np
import torch

from oracle.gdr import gdr_recurrent, gdr_recurrent_vjp, packed
from oracle.gdr_chunked import gdr_chunked_vjp, growth
from tests._gpu_util import half_ulp_bf16

GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def in_chunks(dtype, dk, dv):
    return dtype == torch.bfloat16 and dk >= 64 and dv >= 64


def walk(dtype, dk, dv, T):
    """Relative error of a state element, T tokens at most."""
    memory = min(T, 2 * dk)
    n = 3 * dk / 32 + 3 + 18 + 7 * (memory / 64 + 1) if in_chunks(dtype, dk, dv) else 20 + 1.5 * memory
    return np.sqrt(n) * 2.0 ** -24 / np.sqrt(3)


def bars(dtype, dk, dv, T, gr):
    """{output: tolerance on the 2-norm} of the fp32 outputs; gr: growth()."""
    e = walk(dtype, dk, dv, T)
    both = 2 * np.sqrt(2) * e * max(gr["Y"], gr["F"])
    return {"o": 2 * e * gr["Y"], "S_T": 2 * e * gr["Y"], "dS0": 2 * e * gr["F"], "dv": 2 * e * gr["F"],
            "dq": both, "dk": both, "dbeta": both, "dg": both * gr["dg"]}


def misses(got, ref, tol):
    """None, or what is wrong with an fp32 output at this tolerance."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    if got.shape != ref.shape or not np.array_equal(np.isfinite(got), np.isfinite(ref)):
        return "shape or finiteness"
    norm = np.linalg.norm(ref)
    d = np.abs(got - ref)
    if norm == 0:
        return None if d.max(initial=0.0) == 0 else "not zero"
    rel = np.linalg.norm(d) / norm
    off = (d / np.maximum(np.abs(ref), norm / np.sqrt(ref.size))).max()
    print(f"    rel {rel:.2e} (<= {tol:.1e}) most {off:.2e} (<= {40 * tol:.1e})", flush=True)
    return None if rel <= tol and off <= 40 * tol else f"rel {rel:.2e} most {off:.2e} over {tol:.1e}"


def misses_bf16(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    if got.shape != ref.shape or not np.array_equal(np.isfinite(got), np.isfinite(ref)):
        return "shape or finiteness"
    norm = np.linalg.norm(ref)
    d = np.abs(got - ref)
    if norm == 0:
        return None if d.max(initial=0.0) == 0 else "not zero"
    rel = np.linalg.norm(d) / norm
    tol = 2.0 ** -8 * min(1.0, 1 / np.sqrt(3) + 1 / np.sqrt(ref.size)) + 2.0 ** -16
    off = (np.maximum(d - half_ulp_bf16(ref), 0) / np.maximum(np.abs(ref), norm / np.sqrt(ref.size))).max()
    print(f"    rel {rel:.2e} (<= {tol:.1e}) beyond a half step {off:.2e} (<= {2.0 ** -11:.1e})", flush=True)
    return None if rel <= tol and off <= 2.0 ** -11 else f"rel {rel:.2e} beyond a half step {off:.2e}"


def check(name, x, ref, tol):
    """A device output against fp64."""
    print(f"  {name}", flush=True)
    got = x.detach().double().cpu().numpy()
    bad = misses_bf16(got, ref) if x.dtype == torch.bfloat16 else misses(got, ref, tol[name])
    assert bad is None, (name, bad)


def reference(h, cu, scale, dtype, grads=True):
    """((o, S_T), gradients or None, bars) of a packed batch of fp64 arrays h."""
    dk, dv = h["q"].shape[2], h["v"].shape[2]
    fwd = packed(lambda q, k, v, g, b, S0: gdr_recurrent(q, k, v, g, b, scale, S0), cu,
                 [h[x] for x in ("q", "k", "v", "g", "beta")], (h["S0"],))
    bwd, norms = None, []
    rows = [h[x] for x in ("q", "k", "v", "g", "beta", "dO")]
    if grads:
        bwd = packed(lambda q, k, v, g, b, dO, S0, dS: gdr_recurrent_vjp(q, k, v, g, b, dO, scale, S0, dS), cu, rows,
                     (h["S0"], h["dS_T"]))
    for n in range(len(cu) - 1):
        norms.append(gdr_chunked_vjp(*(x[cu[n]:cu[n + 1]] for x in rows), scale,
                                     *(None if h[x] is None else h[x][n] for x in ("S0", "dS_T")),
                                     C=64 if in_chunks(dtype, dk, dv) else 32)[2])
    longest = max((b - a for a, b in zip(cu, cu[1:])), default=0)
    gr = growth(norms)
    print("  growth", {x: round(y, 2) for x, y in gr.items()}, flush=True)
    return fwd, bwd, bars(dtype, dk, dv, longest, gr)


def compare(b, dtype, grads=True):
    """A batch of tests/test_gpu_gdr.py's make() through the forward and the
    backward, against the oracle."""
    from tests.test_gpu_gdr import bwd, fwd, host
    ref, rg, tol = reference(host(b), b["cu"].tolist(), b["scale"], dtype, grads)
    for name, x, y in zip(("o", "S_T"), fwd(b), ref):
        check(name, x, y, tol)
    if grads:
        for name, x, y in zip(GRADS, bwd(b), rg):
            check(name, x, y, tol)
    return tol
