"""Tolerances of the paged cache's GPU tests, derived from the kernels' roundings.

With u = eps / 2 of the output's type (one rounding) and e = 2^-24 (fp32):

attend  a logit is a d-term fp32 sum of exact products, times a rounded scale: off by at most
        D = (d + 4) e S, S = max_j sum_i |q_i k_ji| / sqrt(d).  A weight exp(s) / sum is off by a
        relative 2 D (numerator and sum) + 8 e (two exponentials of 2 ulp each way, one division)
        + (n + 64) e (the fp32 sums over n keys, joined); weights split into two 16-bit halves
        add 2^-16.  With A = sum_j p_j |v_j|:  |out - ref| <= u |ref| + (2 D + (2 n + 136) e + 2^-16) A.
        An f16 output below 2^-14 rounds in steps of 2^-24: + 2^-25.  f16 halves of a weight round
        in steps of 2^-24 of the largest weight: + n 2^-25 max |v| for f16.
write   cos and sin of a table product are within 4 e, two products and a sum add 3 e:
        |y - ref| <= u |ref| + 7 e (|x1| + |x2|); values are rounded once.
k_mean  against the stored keys: u |ref| + page e mean|k|.
"""
import numpy as np

E32 = 2.0 ** -24


def attend_tolerance(u, d, f16, ref, size, big, v):
    """ref, size [G][d], big: as oracle.pages.attend_one returns them; v [n][d] the values."""
    n = len(v)
    tol = u * np.abs(ref) + (2 * (d + 4) * E32 * big + (2 * n + 136) * E32 + 2.0 ** -16) * size
    if f16:
        tol = tol + 2.0 ** -25 * (1 + n * np.abs(v).max() if n else 1)
    return tol
