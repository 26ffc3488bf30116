"""Decayed linear attention and the 8-bit state pool in 64 bits on the CPU, from
their definitions, and the error bounds that the kernels are held to.

Bounds. Every output is a sum of products; `mag` is the same sum with every
factor replaced by its magnitude, so a relative error eps of each term moves the
output by at most eps * mag. With u the half step of the type (bf16 2^-8... as
finfo(t).eps / 2) the terms of o carry one rounding of an operand to the 16-bit
type (the decayed score of a token of the same block, or the state that enters
the block: never both), o one more of its own, and the fp32 arithmetic at most
(2 T + dk + 64) roundings of 2^-24 (T updates of two operations, the products'
sums). The state carries the fp32 part alone: its operands are split so that
nothing above 2^-24 is dropped.
"""
import numpy as np
import torch

F32 = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def linear_prefill(q, k, v, g, state_in, cu, scale=None):
    """(o, S, mag_o, mag_S): g [T, Hv] or [Hv]. Rows of o outside the sequences stay NaN."""
    q, k, v, g = f64(q), f64(k), f64(v), f64(g)
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1:]
    head = np.arange(Hv) // (Hv // Hqk)
    scale = dk ** -0.5 if scale is None else scale
    if g.ndim == 1:
        g = np.broadcast_to(g, (T, Hv))
    cu = [int(c) for c in cu]
    N = len(cu) - 1
    S = np.zeros((N, Hv, dv, dk)) if state_in is None else f64(state_in).copy()
    A = np.abs(S)
    o, mag = np.full((T, Hv, dv), np.nan), np.zeros((T, Hv, dv))
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            a = np.exp(g[t])[:, None, None]
            kt, qt, vt = k[t, head], q[t, head] * scale, v[t]
            # a reset (alpha = 0) forgets even an infinite or NaN past
            S[n] = np.where(a == 0, 0, a * S[n]) + vt[:, :, None] * kt[:, None, :]
            A[n] = np.where(a == 0, 0, a * A[n]) + np.abs(vt[:, :, None] * kt[:, None, :])
            o[t] = np.einsum("hij,hj->hi", S[n], qt)
            mag[t] = np.einsum("hij,hj->hi", A[n], np.abs(qt))
    return o, S, mag, A


def steps(cu):
    return max([int(b) - int(a) for a, b in zip(cu[:-1], cu[1:])] + [1])


def check_o(o, ref, mag, T, dk, what="o"):
    u = torch.finfo(o.dtype).eps / 2
    tiny = torch.finfo(o.dtype).tiny * u * 2 if o.dtype == torch.float16 else 0.0   # half a step below the normal range
    bound = u * np.abs(ref) + ((u if o.dtype != torch.float32 else 0.0) + (2 * T + dk + 64) * F32) * mag * (1 + u) + tiny
    _within(f64(o), ref, bound, what)


def check_state(s, ref, mag, T, what="state", extra=0.0):
    u = torch.finfo(s.dtype).eps / 2 if s.dtype != torch.float32 else 0.0
    _within(f64(s), ref, u * np.abs(ref) + ((2 * T + 64) * F32 * (1 + u) + extra) * mag + 1e-37, what)


def _within(x, ref, bound, what):
    assert x.shape == ref.shape
    bad = ~(np.abs(x - ref) <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(np.abs(x - ref) / (bound + 1e-300), nan=1e300), 0)), x.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, worst at {at}: "
                             f"{x[at]!r} against {ref[at]!r}, bound {bound[at]:.3e}")


# ------------------------------------------------------------- state pool ---
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def quantise(x, dtype):
    """(values that the codes stand for, exponent bytes) of x [..., dk]."""
    x = f64(x)
    group = min(32, x.shape[-1])
    y = x.reshape(*x.shape[:-1], -1, group)
    amax = np.abs(y).max(-1)
    bad = ~np.isfinite(y).all(-1)
    m, e = np.frexp(np.where(bad, 0, amax) / QMAX[dtype])      # amax / QMAX = m 2^e, m in [1/2, 1): 2^e is enough, 2^(e-1) if m = 1/2
    e = np.where(m == 0.5, e - 1, e)
    e = np.where(m == 0, -127, np.maximum(e, -127))
    z = np.where(bad[..., None], 0, y) / np.exp2(e.astype(np.float64))[..., None]
    step = np.exp2(np.maximum(np.frexp(z)[1] - 4, -9).astype(np.float64)) if dtype == torch.float8_e4m3fn else 1.0
    val = np.round(z / step) * step * np.exp2(e.astype(np.float64))[..., None]     # numpy rounds ties to even
    val = np.where(bad[..., None], np.nan, val)
    return val.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)
