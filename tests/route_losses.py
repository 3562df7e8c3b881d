"""Bounds on the router's two losses (test infrastructure), each against its own
value.

Balance: a sum of positive terms counts_e prob_sum_e, of which prob_sum carries
the error of a probability (2^-17 relative, which covers its own additions) and
the sums in 64 bits none; the result is rounded once: 2^-16.
z: the mean of lse^2; lse is off by 2^-17 of its value and 2^-20, and at most 70
fp32 additions in a row (2^-17.8) sum the squares: (2^-16 + 2^-17) z + 2^-19
sqrt(z)."""
import numpy as np


def losses_off(got, want):
    """The losses (balance, z) that are not within their bounds, by name."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = [2.0 ** -16 * want[0], (2.0 ** -16 + 2.0 ** -17) * want[1] + 2.0 ** -19 * np.sqrt(want[1])]
    return [n for n, g, w, t in zip(("balance", "z"), got, want, tol) if not abs(g - w) <= t]
