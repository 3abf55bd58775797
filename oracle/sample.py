"""CPU reference (numpy, fp64 exponentials and whole-number masses) of sampling from logits.

R_v = floor(2^40 exp((l_v - max l) / T)); ranked by logit (ties: the lower index) the kept
tokens are the shortest of: the first top_k; the shortest prefix whose R reach ceil(top_p * the
top-k's sum); those with R_v >= min_p 2^40.  The token is the first whose running sum of kept R
exceeds floor(floor(2^24 u) Z / 2^24).
"""
import math

import numpy as np


def clean(l):
    l = np.asarray(l, np.float64)
    return np.where(np.isnan(l), -np.inf, l)


def masses(l, temperature):
    """Whole-number masses as float64 (exact: at most 2^40)."""
    l = clean(l)
    top = l.max()
    if top == np.inf:
        return np.where(l == np.inf, 2.0 ** 40, 0.0)
    with np.errstate(over="ignore"):
        return np.floor(np.exp((l - top) / float(temperature)) * 2.0 ** 40)


def valid(u, temperature, top_k=0, top_p=1.0, min_p=0.0):
    t_ok = temperature == 0 or (np.float32(1e-6) <= temperature <= np.float32(1e30))
    return bool(t_ok and top_k >= 0 and 0 < top_p <= 1 and 0 <= min_p <= 1 and (temperature == 0 or 0 <= u < 1))


def kept_masses(l, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(masses of kept tokens, zeros elsewhere, as Python-exact float64; how near the decisions
    were: the least relative distance of a prefix sum from top_p's target)."""
    R = masses(l, temperature)
    V = len(R)
    order = np.lexsort((np.arange(V), -clean(l)))
    ranked = R[order].astype(np.uint64)
    cum = np.cumsum(ranked)
    n, near = V, 1.0
    if 1 <= top_k < V:
        n = top_k
    if top_p < 1:
        tau = max(1, math.ceil(float(np.float32(top_p)) * float(cum[n - 1])))
        near = float(np.abs(cum[:n].astype(np.float64) - tau).min() / tau)
        n = min(n, int((cum < np.uint64(tau)).sum()) + 1)
    n = min(n, int((ranked.astype(np.float64) >= float(np.float32(min_p)) * 2.0 ** 40).sum()))
    keep = np.zeros(V)
    keep[order[:n]] = R[order[:n]]
    return keep, near


def draw(keep, u):
    """(token, relative distance of the target from the nearest edge of the token's step)."""
    cum = np.cumsum(keep.astype(np.uint64))
    Z = int(cum[-1])
    t = (int(np.floor(np.float64(np.float32(u)) * 2 ** 24)) * Z) >> 24
    v = int(np.searchsorted(cum, np.uint64(t), side="right"))
    lo = int(cum[v - 1]) if v else 0
    return v, min((t - lo) if v else Z, int(cum[v]) - t) / Z


def sample(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, q [V], how near the decisions were to another outcome)."""
    V = len(l)
    if not valid(u, temperature, top_k, top_p, min_p) or clean(l).max() == -np.inf:
        return -1, np.zeros(V), 1.0
    if temperature == 0:
        v = int(np.argmax(clean(l)))
        return v, np.eye(1, V, v)[0], 1.0
    keep, near = kept_masses(l, temperature, top_k, top_p, min_p)
    v, edge = draw(keep, u)
    return v, keep / keep.sum(), min(near, edge)
