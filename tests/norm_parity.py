"""Checks of the combine and 8-bit norm steps against the fp64 oracle.

Error bounds, from the arithmetic (u = 2^-24, fp32's half step):
  * z is a sum of n terms in fp32: |z32 - z64| <= n u absum, absum the sum of
    the terms' absolute values (a product's rounding is inside the fma).
  * the residual is z32 rounded once to bf16: half a bf16 step more.
  * y = (z r) gamma: z's error carried through r |gamma|, and a relative error
    of (H / 256 + 32) u: each thread adds H / 256 squares in turn and 13 more
    partial sums, which r halves; rsqrtf is within 2 ulp, its argument and the
    two products within 4 u.
  * bf16 output: half a step more. e4m3 output: half an e4m3 step at y / s,
    times s, with the division's and the scale's roundings (4 u, relative)
    inside the relative error above.
"""

import numpy as np

from oracle import bf16, quant8

U = 2.0 ** -24


def bits16(t):
    import torch
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def half_ulp(x):
    return 0.5 * bf16.ulp(x)


def y_error(z64, y64, absum, n_terms, gamma_bits, eps):
    """Bound of |y32 - y64| per element."""
    h = z64.shape[1]
    r = 1.0 / np.sqrt(np.mean(z64 * z64, axis=1, keepdims=True) + eps)
    carried = r * np.abs(bf16.decode(gamma_bits))[None, :] * (n_terms * U * absum)
    # an error of z also moves r: by at most its largest relative part
    moved = np.abs(y64) * (np.linalg.norm(n_terms * U * absum, axis=1, keepdims=True) /
                           np.maximum(np.linalg.norm(z64, axis=1, keepdims=True), 1e-300))
    return carried + moved + (h / 256 + 32) * U * np.abs(y64)


def check_residual(z64, absum, n_terms, residual):
    got = bf16.decode(bits16(residual))
    slack = n_terms * U * absum
    assert np.all(np.abs(got - z64) <= half_ulp(np.abs(z64) + slack) + slack)


def check_bf16(y64, y_err, out):
    got = bf16.decode(bits16(out))
    bad = ~(np.abs(got - y64) <= half_ulp(np.abs(y64) + y_err) + y_err)
    assert not bad.any(), "%d of %d outputs off" % (bad.sum(), bad.size)


def check_q8(y64, y_err, out, scales, group):
    """Codes and scales of an e4m3 output against y64 within y_err."""
    import torch
    t, h = y64.shape
    g = group or h
    e8m0 = scales.dtype is not torch.float32
    kind = "e8m0" if e8m0 else "f32"
    stored = quant8.decode_scales(scales.cpu().view(torch.uint8).numpy() if e8m0
                                  else scales.cpu().numpy(), kind)
    amax = quant8.group_max(y64, group)
    err = y_err.reshape(t, h // g, g).max(axis=2)
    lo = quant8.scale(np.maximum(amax - err, 0.0), kind) * (1 - 4 * U)
    hi = quant8.scale(amax + err, kind) * (1 + 4 * U)
    assert np.all((stored >= lo) & (stored <= hi)), "scales off"
    q = quant8.decode(out.cpu().view(torch.uint8).numpy())
    s = np.repeat(stored, g, axis=1)
    tol = s * quant8.half_step((np.abs(y64) + y_err) / s) + y_err
    bad = ~(np.abs(q * s - y64) <= tol)
    assert not bad.any(), "%d of %d codes off" % (bad.sum(), bad.size)
