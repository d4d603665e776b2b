"""fp64 oracle of the expert router and of the combine step.

TEST INFRASTRUCTURE (see the package docstring). Both are the plain
definitions, one token at a time.
"""

import math

import numpy as np

from . import bf16
from .fused import rms_norm


def route(logits, k, bias=None, scoring="softmax", n_groups=1, top_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """(ids [T, K], weights [T, K]) of float64 logits [T, E].

    A logit that is NaN or -inf, or a bias that is, leaves its expert out;
    +inf counts as the largest fp32. Missing slots have id -1, weight 0.
    """
    big = float(np.finfo(np.float32).max)
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        x = [min(float(v), big) for v in logits[t]]
        there = [e for e in range(E) if x[e] > -math.inf]  # NaN compares false
        if scoring == "softmax":
            top = max((x[e] for e in there), default=0.0)
            ex = {e: math.exp(max(x[e] - top, -800.0)) for e in there}
            total = math.fsum(ex.values())
            s = {e: ex[e] / total for e in there}
        else:
            s = {e: _sigmoid(x[e]) for e in there}
        if bias is not None:
            b = [min(float(v), big) for v in bias]
            there = [e for e in there if b[e] > -math.inf]
            value = {e: s[e] + b[e] for e in there}
        else:
            value = s
        order = value if bias is not None else {e: x[e] for e in there}
        if top_groups < n_groups:
            size = E // n_groups
            sums = {}
            for g in range(n_groups):
                best = sorted((value[e] for e in there if e // size == g), reverse=True)
                if best:
                    if group_top == 1 and bias is None:  # a score's order is its logit's
                        sums[g] = max(x[e] for e in there if e // size == g)
                    else:
                        sums[g] = sum(best[:group_top])
            kept = sorted(sums, key=lambda g: (-sums[g], g))[:top_groups]
            there = [e for e in there if e // size in kept]
        chosen = sorted(there, key=lambda e: (-order[e], e))[:k]
        if not chosen:
            continue
        w = [s[e] for e in chosen]
        if renormalize:
            # the scores' ratio, from their logarithms where they underflow
            if scoring == "softmax":
                m = max(x[e] for e in chosen)
                w = [math.exp(max(x[e] - m, -800.0)) for e in chosen]
            else:
                logs = [_log_sigmoid(x[e]) for e in chosen]
                m = max(logs)
                w = [math.exp(max(v - m, -800.0)) for v in logs]
            total = math.fsum(w)
            w = [v / total for v in w]
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [v * scale for v in w]
    return ids, weights


def _sigmoid(x):
    return 1.0 / (1.0 + math.exp(-x)) if x > -700.0 else math.exp(max(x, -745.0))


def _log_sigmoid(x):
    return -math.log1p(math.exp(-x)) if x > -700.0 else x


def combine(experts, rows, weights, partials, residual, gamma, eps):
    """(z64, y64, absum) of the combine step; bf16 tensors as uint16 bits.

    absum is the sum of the absolute values of z's terms, for error bounds. A
    row index outside the expert rows adds nothing.
    """
    z = bf16.decode(residual).astype(np.float64)
    absum = np.abs(z)
    for p in partials:
        v = bf16.decode(p)
        z, absum = z + v, absum + np.abs(v)
    x = bf16.decode(experts)
    for t in range(z.shape[0]):
        for j in range(rows.shape[1]):
            r = int(rows[t, j])
            if 0 <= r < x.shape[0]:
                v = float(weights[t, j]) * x[r]
                z[t] = z[t] + v
                absum[t] = absum[t] + np.abs(v)
    return z, rms_norm(z, bf16.decode(gamma), eps), absum
