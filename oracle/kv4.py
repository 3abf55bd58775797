"""CPU reference (numpy, fp64) of the 4-bit KV cache: what it holds of a vector, and the
verify window's attention over held values.

Per vector x (one token's K or V of one kv head): x' = clamp(x, -65504, 65504) with NaN
-> -65504, m = fp16 rounded down of min x', s = fp16 rounded up of (max x' - m) / 15,
c = floor((x' - m) / s + 1/2) (0 where s = 0); it stands for s * c + m.  The differences
with m are fp32 numbers.
"""
import numpy as np

HALF_MAX = 65504.0


def saturate(x):
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -HALF_MAX, np.clip(x, -HALF_MAX, HALF_MAX))


def half_down(x):
    h = np.clip(x, -HALF_MAX, HALF_MAX).astype(np.float16)
    return np.where(h.astype(np.float64) > x, np.nextafter(h, np.float16(-HALF_MAX)), h).astype(np.float64)


def half_up(x):
    return -half_down(-x)


def quantise(x):
    """x [..., hd] -> (codes, s, m); s and m [..., 1]."""
    x = saturate(x)
    m = half_down(x.min(-1, keepdims=True))
    d = (x - m).astype(np.float32).astype(np.float64)
    s = half_up(d.max(-1, keepdims=True) / 15.0)
    q = np.divide(d, s, out=np.zeros_like(x), where=s > 0)
    return np.clip(np.floor(q + 0.5), 0, 15), s, m


def held(x):
    c, s, m = quantise(x)
    return c * s + m


def window_mask(n_rows, parent=None):
    """[n_rows, n_rows] bool: window rows that each row sees (itself and its ancestors)."""
    see = np.zeros((n_rows, n_rows), bool)
    for j in range(n_rows):
        i = j
        while i >= 0:
            see[j, i] = True
            i = parent[i] if parent is not None else i - 1
    return see


def attention(q, k, v, n_cached, parent=None, scale=None, key_ok=None):
    """q [n, Hq, hd]; k, v [n_cached + n, Hkv, hd] held values; key_ok [keys]: tokens with a cell.
    Returns (out [n, Hq, hd], weights list [Hkv] of [grp, n, keys] probabilities)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, Hq, hd = q.shape
    Hkv = k.shape[1]
    grp = Hq // Hkv
    scale = hd ** -0.5 if scale is None else scale
    see = np.concatenate([np.ones((n, n_cached), bool), window_mask(n, parent)], 1)
    if key_ok is not None:
        see &= key_ok[None, :]
    out = np.zeros((n, Hq, hd))
    probs = []
    for h in range(Hkv):
        sc = np.einsum("ngd,kd->gnk", q[:, h * grp:(h + 1) * grp], k[:, h]) * scale
        sc = np.where(see[None], sc, -np.inf)
        top = sc.max(-1, keepdims=True)
        w = np.exp(sc - np.where(np.isfinite(top), top, 0.0))
        tot = w.sum(-1, keepdims=True)
        p = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
        probs.append(p)
        out[:, h * grp:(h + 1) * grp] = np.einsum("gnk,kd->ngd", p, v[:, h])
    return out, probs
