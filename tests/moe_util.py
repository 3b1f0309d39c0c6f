"""Plain float64 forms of the grouped products, the fused epilogues and the
router, written from their definitions, with the bounds their results are
held to."""
import math

import numpy as np

from mlp_huffman_coded_b200 import synth
from oracle import uw_oracle as O

HALF_ULP = 2.0 ** -8  # largest relative error of one BF16 rounding
F32 = 2.0 ** -24      # of one FP32 operation


def act_f64(v, name):
    v = np.asarray(v, dtype=np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return O.silu(v)
    if name == "gelu":
        return 0.5 * v * np.array([math.erfc(-t / math.sqrt(2)) for t in v.ravel()]).reshape(v.shape)
    assert name == "gelu_tanh"
    return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def sum_bound(absdot, K):
    """|FP32 sum of K exact BF16 products - exact sum| <= K 2^-23 sum |w x|:
    K additions, each off by at most 2^-23 of the partial sum it forms (which
    covers an adder that cuts off instead of rounding), and no partial sum
    exceeds sum |w x|.  Joining the partial sums of several issuers or CTAs
    only replaces additions of the same kind."""
    return K * 2.0 ** -23 * absdot


def epilogue_bound(v, dv, bias, act, residual, bf16):
    """(value, bound) of act(v + bias) + residual computed in FP32 from a sum
    that is within dv of v.  The activations' slopes are at most 1.13 (GELU
    has the largest).  Their FP32 evaluation: a handful of operations and one
    library function of at most 4 units in the last place, each relative to
    the activation's value or to v: 16 of 2^-24 (|v| + |act|); GELU's tanh
    form takes exp of a polynomial in v, off by 2^-22 |t| relative, and |t|
    times the result is at most 12 where the result is not negligible or
    saturated: another 48 of 2^-24 (|v| + |act|) covers it.  GELU's normal
    tail comes from a fit within 4.3e-8 and exp(-v^2 / 2) with the exponent
    rounded, off by 2^-23 v^2 / 2 relative, and v^2 / 2 times the tail is at
    most 0.2: less than the tanh form's.  BF16 adds one rounding of the
    result."""
    s = v + bias
    dv = dv + F32 * np.abs(s)
    a = act_f64(s, act)
    da = 1.13 * dv + (0 if act in ("none", "relu") else 64 * F32) * (np.abs(s) + np.abs(a))
    y = a + residual
    dy = da + F32 * np.abs(y) + F32 * da
    if bf16:
        dy = dy + HALF_ULP * (np.abs(y) + dy)
    return y, dy + 1e-30


SMALLEST_NORMAL = 2.0 ** -126


def act_tail(v, name):
    """act_f64 in forms that keep their relative accuracy for negative v,
    where 1 + tanh would cancel."""
    v = np.asarray(v, dtype=np.float64)
    if name != "gelu_tanh":
        return act_f64(v, name)
    t = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-t))


def activation_bound(v, name):
    """Largest error of an FP32 activation of an exact v, relative to the
    activation itself; below the smallest normal number nothing is promised.
    u = 2^-24 is one FP32 rounding; a unit in the last place is at most 2 u.

    SiLU, (v or v e) / (1 + e) with e = exp(-|v|): e 2 units (4 u), v e 1 u,
    1 + e 1 u and half of e's error, the quotient 2 units (4 u): 12 u.
    GELU's tanh form, the same with t, which is off by 7 u relative (three
    products, a sum, two rounded constants and their product), so e by
    another 7 u |t|, and the divisor by half of that.
    GELU, v Phi(v) with Phi(-a) = exp(-a^2 / 2) t P(t) / 2: t 7 u (divisor 3 u,
    quotient 4 u), and t P(t) changes by at most 2.3 times as much; P 9
    roundings of terms whose magnitudes add up to 2.2 times P, and the fit's
    1 u; the products 4 u; the fast exponential of x = -v^2 / 2 is off by
    2 + 1.173 |x| units, and the rounding of x gives another |x| u."""
    v = np.asarray(v, dtype=np.float64)
    y = np.abs(act_tail(v, name))
    if name == "gelu":
        rel = 48 + 1.7 * v * v
    elif name == "gelu_tanh":
        rel = 13 + 11 * np.abs(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    else:
        rel = np.full_like(v, 13.0 if name == "silu" else 0.0)
    return np.minimum(rel * F32, 1.0) * y + SMALLEST_NORMAL


def product(w, x):
    """x W^T in float64 and sum |w x| (BF16 bit patterns in)."""
    wf, xf = O.bf16_to_f64(w), O.bf16_to_f64(x)
    return xf @ wf.T, np.abs(xf) @ np.abs(wf).T


def grouped_ref(ws, x, rows, offsets, biases=None, act="none", residual=None, bf16=True):
    """[(slot range, value, bound)] expert by expert."""
    out = []
    for e, w in enumerate(ws):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b <= a:
            continue
        v, ab = product(w, x[rows[a:b]])
        bias = 0.0 if biases is None else O.bf16_to_f64(biases[e])[None, :]
        res = 0.0 if residual is None else O.bf16_to_f64(residual[a:b])
        out.append((a, b) + epilogue_bound(v, sum_bound(ab, w.shape[1]), bias, act, res, bf16))
    return out


def swiglu_ref(gs, us, x, rows, offsets):
    """SiLU(g) u with |dg|, |du| from the sums: |d| <= 1.1 |dg| |u| +
    |silu(g)| |du| + 1.1 |dg| |du|, and the FP32 evaluation and rounding."""
    out = []
    for e, (wg, wu) in enumerate(zip(gs, us)):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b <= a:
            continue
        K = wg.shape[1]
        g, ag = product(wg, x[rows[a:b]])
        u, au = product(wu, x[rows[a:b]])
        dg, du = sum_bound(ag, K), sum_bound(au, K)
        s = O.silu(g)
        y = s * u
        d = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du
        d = d + 16 * F32 * (np.abs(g) + np.abs(s)) * np.abs(u)
        out.append((a, b, y, d + HALF_ULP * (np.abs(y) + d) + 1e-30))
    return out


def check_slots(got, refs):
    """got: float64 [n, rows]; refs as above.  The worst excess over the bound."""
    worst = -math.inf
    for a, b, y, d in refs:
        worst = max(worst, float(np.max(np.abs(got[a:b] - y) - d)))
    return worst <= 0, worst


def route_ref(logits, k, renormalize=True):
    """Token by token: (weights, experts, slots, rows, offsets), float64."""
    T, E = logits.shape
    weights, experts = np.zeros((T, k)), np.full((T, k), -1, np.int32)
    groups = [[] for _ in range(E)]
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        l = [(-math.inf if math.isnan(v) else min(v, big)) for v in logits[t].astype(np.float64)]
        order = sorted((e for e in range(E) if l[e] > -math.inf), key=lambda e: (-l[e], e))[:k]
        if not order:
            continue
        p = {e: math.exp(l[e] - l[order[0]]) for e in range(E) if l[e] > -math.inf}
        whole = sum(p[e] for e in order) if renormalize else sum(p.values())
        for j, e in enumerate(order):
            weights[t, j], experts[t, j] = p[e] / whole, e
            groups[e].append((t, j))
    slots, rows, offsets = np.full((T, k), -1, np.int32), [], [0]
    for g in groups:
        for t, j in g:
            slots[t, j] = len(rows)
            rows.append(t)
        offsets.append(len(rows))
    return weights, experts, slots, np.array(rows, np.int32), np.array(offsets, np.int32)


def expert_weights(E, rows, cols, seed, rate=1e-3, scale=200.0):
    return [synth.weight_matrix(rows, cols, 0.02, rate, scale, seed + e) for e in range(E)]
