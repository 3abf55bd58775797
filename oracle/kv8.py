"""CPU reference (numpy, fp64) of the 8-bit KV cache: what a sub-block of 16 tokens holds after
a write, and which tokens an eviction keeps.  (The window's attention over held values is
kv4.attention's.)

x' = clamp(x, -65504, 65504) with NaN -> -65504; e = least exponent in -15..8 with
max |x'| <= 448 * 2^e over the call's rows of the sub-block, at least the old one where the
sub-block's first token is not among them; a value is held as the e4m3 number nearest to
x' / 2^e (ties to even) times 2^e.
"""
import numpy as np

from .kv4 import saturate

SUB = 16
MIN_EXP, MAX_EXP = -15, 8


def needed_exp(a):
    for e in range(MIN_EXP, MAX_EXP):
        if a <= 448.0 * 2.0 ** e:
            return e
    return MAX_EXP


def e4m3(y):
    """Nearest e4m3 number (ties to even) of |y| <= 448: steps of 2^(k - 3) in [2^k, 2^(k + 1)), 2^-9 below 2^-6."""
    y = np.asarray(y, np.float64)
    _, x = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))   # 2^(x - 1) <= |y| < 2^x
    step = np.ldexp(1.0, x - 1 - 3)
    return np.rint(y / step) * step                     # rint: ties to even


class HeldSeq:
    """K or V of one kv head of one sequence: y [tokens, hd] held values, e [tokens / 16]
    (`e`: what the memory says before any write; it counts where a sub-block's first token is
    not the first that is written)."""

    def __init__(self, tokens, hd, e=0):
        self.y = np.zeros((tokens, hd))
        self.e = np.full(tokens // SUB, e)

    def write(self, start, x):
        """Rows x at positions start, start + 1, ...: those below 0 or past the end have no cell."""
        x = saturate(x)
        for s in range(len(self.e)):
            lo, hi = max(start, s * SUB), min(start + len(x), (s + 1) * SUB)
            if lo >= hi:
                continue
            rows = x[lo - start:hi - start]
            e = needed_exp(np.abs(rows).max())
            if lo > s * SUB:
                e = max(e, self.e[s])
            self.e[s] = e
            blk = slice(s * SUB, (s + 1) * SUB)
            old = e4m3(np.clip(self.y[blk] / 2.0 ** e, -448, 448)) * 2.0 ** e
            self.y[blk] = old
            self.y[lo:hi] = e4m3(rows / 2.0 ** e) * 2.0 ** e


def held(x):
    """What one write from token 0 on holds of x [tokens, hd]."""
    c = HeldSeq((len(x) + SUB - 1) // SUB * SUB, x.shape[1])
    c.write(0, x)
    return c.y[:len(x)]


def keep_tokens(weight, n, keep, recent):
    """Positions that stay of n tokens with weights weight[:n]: the last `recent`, the others by
    weight (the earlier of equal ones; NaN lowest)."""
    m = min(n, keep)
    r = min(recent, m)
    w = np.asarray(weight[:n - r], np.float64)
    w = np.where(np.isnan(w), -np.inf, w)
    nan_last = np.isnan(np.asarray(weight[:n - r], np.float64))
    order = np.lexsort((np.arange(n - r), nan_last, -w))     # last key first: weight, then NaN behind -inf, then position
    return np.concatenate([np.sort(order[:m - r]), np.arange(n - r, n)]).astype(np.int64)
