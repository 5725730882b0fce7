"""The attention operators' definition in fp64 numpy, one token and head at a time, and the
error bounds their tests use.  Shares no code with the library.

Bounds.  With p_j the softmax weights of a row and A = sum_j p_j |v_j| (per element), the
kernels' result o differs from the exact one by at most

    A * (r_P + 2 e_s + (n + 16) u) + |o| (r_out + 16 u),      u = 2^-24

* r_P: the weights are rounded to bf16 before the product with v in the bf16 mode (half a
  step, 2^-8 relative), and 7.5e-5 relative is left for the way they are formed, in the
  numerator and in the sum (twice); neither in fp32;
* e_s: a score is a sum of D products in fp32, each term and each partial sum rounded:
  |ds| <= (D + 3) u scale sum_d |q_d k_d|, which moves a weight by the factor e^ds, and the
  row's sum by no more: 2 e_s in all (the scores' products are exact: bf16 times bf16, or
  within the same count of roundings in fp32);
* (n + 16) u: the sums over n keys in fp32, in any order, and the exponentials (a few ulp);
* r_out: the output's own rounding (bf16 2^-8, fp32 2^-24); the gate adds a few ulp of o.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def attend_row(q, k, v, scale):
    """One row: q [D], k, v [n, D] fp64 -> (o [D], A [D], e_s); zeros for n == 0."""
    D = q.shape[0]
    n = k.shape[0]
    if n == 0:
        return np.zeros(D), np.zeros(D), 0.0
    s = scale * (k @ q)
    w = np.exp(s - s.max())
    p = w / w.sum()
    e_s = (D + 3) * U * abs(scale) * float((np.abs(k) @ np.abs(q)).max())
    return p @ v, p @ np.abs(v), e_s


def attention(q, k, v, past, scale, dtype, z=None):
    """q [n, HQ, D]; k, v [n + past, HKV, D] fp64: causal, the last query at the last key.
    Returns (o, bound), both [n, HQ, D]."""
    n, HQ, D = q.shape
    G = HQ // k.shape[1]
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    r_p = HALF_STEP["bf16"] + 2 * 7.5e-5 if dtype == "bf16" else 0.0
    for i in range(n):
        m = max(past + i + 1, 0)
        for h in range(HQ):
            x, A, e_s = attend_row(q[i, h], k[:m, h // G], v[:m, h // G], scale)
            g = 1.0
            if z is not None and m > 0:
                g = 1.0 / (1.0 + np.exp(-z[i, h]))
            o[i, h] = x * g
            bound[i, h] = g * A * (r_p + 2 * e_s + (m + 16) * U) + np.abs(x * g) * (HALF_STEP[dtype] + 16 * U)
    return o, bound


def rotate(x, pos, inv_freq, interleaved):
    """x [D] fp64 turned by pos * inv_freq (inv_freq fp64 values of the fp32 table)."""
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = pos * float(inv_freq[i])
        y[a] = x[a] * np.cos(t) - x[b] * np.sin(t)
        y[b] = x[b] * np.cos(t) + x[a] * np.sin(t)
    return y


def rotate_bound(x, y, inv_freq, interleaved, dtype):
    """Per element: the fp32 angle within [-pi, pi] is off by at most pi u, sine and cosine by
    2 ulp, the two products and the sum by u each: 8 u of the pair's absolute sum, and the
    output's rounding."""
    half = len(inv_freq)
    b = np.zeros(x.shape)
    for i in range(half):
        e = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        s = abs(x[e[0]]) + abs(x[e[1]])
        b[list(e)] = 8 * U * s
    b += np.abs(y) * HALF_STEP[dtype]
    b[2 * half:] = 0.0          # what is not rotated is copied
    return b
