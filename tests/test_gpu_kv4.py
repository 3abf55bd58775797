"""4-bit KV cache on the GPU against the fp64 oracle: write, read back, attention over it.

Tolerances, derived:
 - a read is s * c + m in fp32, rounded to the caller's type: half a step of that type
   (2^-11 of the value for fp16, 2^-8 for bf16, 2^-25 near zero), 2^-23 for the fp32 sum;
 - attention: half a step of the output; weights P s rounded to fp16 (2^-11 of each, or 2^-25 of
   the largest scale once P s is subnormal) times |c - 7.5| <= 7.5; and the scores' fp32 error e
   (2^-22 of the sum of the magnitudes of their terms, and 2^-21 for exp2 and the running sums),
   which moves each weight by a relative 2 e at most, on both sides of the quotient."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu

STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def spec_():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    return spec


def np64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A pool whose unwritten bytes are 0xff (NaN parameters) and page tables over shuffled pages."""

    def __init__(self, lens, Hkv, hd, seed=0, spare=3, first_page=0):
        spec = spec_()
        rng = np.random.default_rng(seed)
        need = [(n + 63) // 64 for n in lens]
        pages = rng.permutation(sum(need) + spare) + first_page
        self.width = max(max(need), 1) + 1
        tab = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            tab[b, :n] = pages[at:at + n]
            at += n
        self.lens, self.Hkv, self.hd = lens, Hkv, hd
        self.table = torch.from_numpy(tab).cuda()
        self.pool = spec.spec_kv4_pool(sum(need) + spare + first_page, Hkv, hd)
        self.pool[first_page:] = 0xff

    def fill(self, seed, dtype=torch.float16):
        """Write every position of every sequence; returns the oracle's held k, v per sequence."""
        spec = spec_()
        off = np.concatenate([[0], np.cumsum(self.lens)])
        g = torch.Generator().manual_seed(seed)
        kv = []
        for _ in range(2):
            x = torch.randn(int(off[-1]), self.Hkv, self.hd, generator=g)
            x = x * torch.exp(0.7 * torch.randn(self.Hkv, self.hd, generator=g)) + 0.5 * torch.randn(self.Hkv, self.hd, generator=g)
            kv.append(x.to(dtype))
        start = torch.zeros(len(self.lens), dtype=torch.int32, device="cuda")
        spec.spec_kv4_write(kv[0].cuda(), kv[1].cuda(), start, self.table, self.pool,
                            row_off=torch.tensor(off, dtype=torch.int32, device="cuda"))
        held = [O.quantise(np64(x)) for x in kv]
        return [(tuple((c * s + m)[off[b]:off[b + 1]] for c, s, m in held), held[1][1][off[b]:off[b + 1]])
                for b in range(len(self.lens))]


def rows_ref(q, held, n_cached, parent=None, scale=None, key_ok=None, dtype=torch.float16):
    """Oracle output of one sequence's window and the derived bound of its error."""
    (k, v), vs = held
    out, probs = O.attention(q, k, v, n_cached, parent, scale, key_ok)
    n, Hq, hd = q.shape
    Hkv = k.shape[1]
    grp = Hq // Hkv
    sc = abs(hd ** -0.5 if scale is None else scale)
    tol = STEP[dtype] * np.abs(out) + 2.0 ** -25
    for h in range(Hkv):
        p, s = probs[h], vs[:, h, 0]                         # [grp, n, keys], [keys]
        live = p.max(-1, initial=0) > 0
        top = np.where(live, p.max(-1, initial=0), 1)        # 1 / l in units of the largest weight
        rnd = 7.5 * (2.0 ** -11 * (p @ s) + 2.0 ** -25 * 2 * s.max(initial=0) * (p > 0).sum(-1) * top)
        mag = np.einsum("ngd,kd->gnk", np.abs(q[:, h * grp:(h + 1) * grp]), np.abs(k[:, h]) + 16 * np.abs(k[:, h]).max(-1, initial=0, keepdims=True))
        e = 2.0 ** -22 * sc * np.where(p > 0, mag, 0).max(-1, initial=0) + 2.0 ** -21
        dev = np.einsum("gnk,kd->gnd", p, np.abs(v[:, h])) + np.abs(np.einsum("gnk,kd->gnd", p, v[:, h]))
        err = rnd[..., None] + 2 * e[..., None] * dev
        tol[:, h * grp:(h + 1) * grp] += np.moveaxis(err, 0, 1)
    return out, tol


def check(got, ref, tol):
    got = np64(got)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / tol).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.3g} of the derived bound"


# ------------------------------------------------------------------ write and read back
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd,Hkv", [(64, 1), (64, 3), (128, 8), (128, 1)])
@pytest.mark.parametrize("B,n,first", [(1, 1, 0), (2, 1, 63), (3, 5, 61), (2, 64, 0), (2, 131, 17), (1, 700, 33)])
def test_write_then_read_is_what_the_oracle_holds(dtype, hd, Hkv, B, n, first):
    spec = spec_()
    c = Cache([first + n] * B, Hkv, hd, seed=n)
    g = torch.Generator().manual_seed(n + hd)
    gain = torch.exp(2 * torch.randn(B, n, Hkv, 1, generator=g))
    k, v = ((torch.randn(B, n, Hkv, hd, generator=g) * gain).to(dtype) for _ in range(2))
    start = torch.full((B,), first, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k.cuda(), v.cuda(), start, c.table, c.pool)
    got = spec.spec_kv4_read(c.pool, start, c.table, n, dtype=dtype)
    for x, y in zip((k, v), got):
        ref = O.held(np64(x))
        y = np64(y)
        tol = STEP[dtype] * np.abs(ref) + 2.0 ** -25 + 2.0 ** -23 * np.abs(ref)
        assert (np.abs(y - ref) <= tol).all()
    # the other type reads the same cells
    other = torch.bfloat16 if dtype == torch.float16 else torch.float16
    for a, b in zip(got, spec.spec_kv4_read(c.pool, start, c.table, n, dtype=other)):
        assert (np.abs(np64(a) - np64(b)) <= 2.0 ** -7 * np.abs(np64(a)) + 2.0 ** -24).all()


def test_special_values():
    spec = spec_()
    hd = 64
    x = torch.zeros(1, 9, 1, hd)
    x[0, 1] = 3.25                                        # no spread
    x[0, 2, 0, 5] = float("inf")
    x[0, 3, 0, 7] = float("-inf")
    x[0, 4, 0, 9] = float("nan")
    x[0, 5] = torch.linspace(-65504, 65504, hd)
    x[0, 6] = torch.linspace(0, 6e-8 * 5, hd)             # fp16 subnormals
    x[0, 7] = torch.arange(hd) % 16 + 0.0                 # whole codes
    x[0, 8] = (torch.arange(hd) % 31) * 0.5               # halves: go up
    for dtype in (torch.float16, torch.bfloat16):
        y = x.to(dtype)
        c = Cache([9], 1, hd)
        start = torch.zeros(1, dtype=torch.int32, device="cuda")
        spec.spec_kv4_write(y.cuda(), y.cuda(), start, c.table, c.pool)
        for got in spec.spec_kv4_read(c.pool, start, c.table, 9, dtype=dtype):
            ref = O.held(np64(y))
            if dtype == torch.float16:
                ref = np.minimum(ref, 65504)              # s is rounded up: 15 s + m may pass fp16's largest
            assert (np.abs(np64(got) - ref) <= (STEP[dtype] + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25).all()
    # values beyond fp16 saturate (infinities times 0 are NaN: those tokens hold -65504 too)
    y = (x * 0 + 1e30).to(torch.bfloat16)
    spec.spec_kv4_write(y.cuda(), y.cuda(), start, c.table, c.pool)
    got, ref = np64(spec.spec_kv4_read(c.pool, start, c.table, 9, dtype=torch.float16)[0]), O.held(np64(y))
    assert (np.abs(got - np.minimum(ref, 65504)) <= 2.0 ** -11 * np.abs(ref)).all() and (got[0, 0] == 65504).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_quotients_next_to_a_half(hd):
    """Quotients above, at and below 7.5 by down to 2^-22 of themselves: each code is the formula's,
    as are those of a million values of one row's scale (about one in a million lies as near)."""
    spec = spec_()
    near = [2.0 ** -e for e in range(8, 22)]
    x = np.zeros((2, 64))
    x[:, 0], x[:, 1] = -7.5, 7.5                           # m = -7.5, s = 1
    x[0, 2:2 + len(near)] = near
    x[1, 2:2 + len(near)] = [-d for d in near]
    rng = np.random.default_rng(1)
    more = np.concatenate([rng.normal(size=(8192, 62)) * 2.0 ** rng.integers(-20, 3, size=(8192, 62)),
                           np.tile([[-7.5, 7.5]], (8192, 1))], 1).clip(-7.5, 7.5)
    x = torch.from_numpy(np.concatenate([x, more])).half()
    x = x.repeat(1, hd // 64).view(1, -1, 1, hd)
    c = Cache([x.shape[1]], 1, hd)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(x.cuda(), x.cuda(), z, c.table, c.pool)
    ref = torch.from_numpy(O.held(np64(x))).half()         # whole steps from -7.5 on: exact
    assert ref[0, 0, 0, 2:2 + len(near)].eq(0.5).all() and ref[0, 1, 0, 2:2 + len(near)].eq(-0.5).all()
    for got in spec.spec_kv4_read(c.pool, z, c.table, x.shape[1]):
        assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd", [64, 128])
def test_many_rows_with_a_few_that_need_saturating(dtype, hd):
    """More rows than warps hold at once, at odd positions, in two sequences: every value as the oracle
    holds it, also beside rows with infinities, NaN, values past fp16 (bf16) and no spread."""
    spec = spec_()
    Hkv, lens, first = 8, [2603, 3000], [3, 62]
    assert sum(lens) * Hkv > 152 * 64 * 256 // hd
    c = Cache([n + f for n, f in zip(lens, first)], Hkv, hd, seed=hd)
    g = torch.Generator().manual_seed(hd)
    k, v = (torch.randn(sum(lens), Hkv, hd, generator=g) * torch.exp(torch.randn(sum(lens), Hkv, 1, generator=g)) for _ in range(2))
    k[17, 3, 5], k[18, 3], v[700, 0, 0], v[701, 7, 63], k[2602, 1, 9] = float("nan"), 2.5, float("inf"), float("-inf"), 1e30
    k, v = k.to(dtype), v.to(dtype)
    start = torch.tensor(first, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k.cuda(), v.cuda(), start, c.table, c.pool, row_off=off)
    for x, y in zip((k, v), spec.spec_kv4_read(c.pool, start, c.table, sum(lens), row_off=off, dtype=dtype)):
        ref = O.held(np64(x))
        if dtype == torch.float16:
            ref = np.minimum(ref, O.HALF_MAX)              # what a read gives at most
        assert (np.abs(np64(y) - ref) <= STEP[dtype] * np.abs(ref) + 2.0 ** -25 + 2.0 ** -23 * np.abs(ref)).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_write_touches_its_cells_only(hd):
    """Neighbours in the page, other pages and other heads keep their bytes; a token at a time gives
    the bytes of one call."""
    spec = spec_()
    c = Cache([200, 90], 2, hd, seed=3)
    c.fill(1)
    before = c.pool.clone()
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(2, 3, 2, hd, generator=g).half().cuda() for _ in range(2))
    start = torch.tensor([126, 7], dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k, v, start, c.table, c.pool)
    whole = c.pool.clone()
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    ref = spec.spec_kv4_read(before, z, c.table, 200)
    now = spec.spec_kv4_read(whole, z, c.table, 200)
    for a, b in zip(ref, now):
        keep = torch.ones(2, 200, dtype=torch.bool, device="cuda")
        keep[0, 126:129] = False
        keep[1, 7:10] = False
        keep[1, 90:] = False                              # never written: NaN parameters
        assert torch.equal(a[keep], b[keep])
        assert not torch.equal(a[0, 126:129], b[0, 126:129])
    assert int((before != whole).sum()) <= 2 * 3 * 2 * (hd + 8)
    c.pool.copy_(before)
    for j in (2, 0, 1):
        spec.spec_kv4_write(k[:, j:j + 1], v[:, j:j + 1], start + j, c.table, c.pool)
    assert torch.equal(c.pool, whole)


def test_rows_without_a_cell_and_rows_of_no_sequence():
    spec = spec_()
    c = Cache([70, 70], 2, 64)
    c.fill(2)
    before = c.pool.clone()
    tab = c.table.clone()
    tab[0, 1] = -1
    tab[1, 1] = c.pool.shape[0]                           # outside the pool
    k = torch.randn(9, 2, 64).half().cuda()
    start = torch.tensor([62, 190], dtype=torch.int32, device="cuda")      # the second starts near the table's end
    off = torch.tensor([1, 5, 8], dtype=torch.int32, device="cuda")        # rows 0 and 8 belong to nobody
    spec.spec_kv4_write(k, k, start, tab, c.pool, row_off=off)
    after = spec.spec_kv4_read(c.pool, torch.tensor([62, 62], dtype=torch.int32, device="cuda"), c.table, 2)[0]
    assert int((before != c.pool).sum()) <= 2 * 2 * 72      # rows 1 and 2 alone had a cell
    assert (np.abs(np64(after[0]) - O.held(np64(k[1:3]))) <= 2.0 ** -10 * np.abs(np64(after[0])) + 2.0 ** -24).all()
    outs = tuple(torch.full((9, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    spec.spec_kv4_read(c.pool, start, tab, 9, row_off=off, outs=outs)
    for o in outs:
        assert (o[0] == 7).all() and (o[8] == 7).all() and (o[3:8] == 0).all() and torch.equal(o[1:3], after[0])
    start = torch.tensor([-2, 0], dtype=torch.int32, device="cuda")         # positions before the first token
    got = spec.spec_kv4_read(c.pool, start, c.table, 3)[0]
    assert (got[0, :2] == 0).all() and (got[0, 2] != 0).any()


def test_strided_rows_of_a_fused_projection():
    spec = spec_()
    c = Cache([80, 80], 2, 128)
    c.pool.zero_()
    qkv = torch.randn(2, 6, 4 + 2 + 2, 128, device="cuda").half()
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    start = torch.tensor([60, 3], dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k, v, start, c.table, c.pool)
    a = c.pool.clone()
    spec.spec_kv4_write(k.contiguous(), v.contiguous(), start, c.table, c.pool)
    assert torch.equal(a, c.pool)
    assert torch.equal(spec.spec_kv4_attention(q, c.pool, start, c.table),
                       spec.spec_kv4_attention(q.contiguous(), c.pool, start, c.table))


# ------------------------------------------------------------------------- attention
CASES = [
    # hd, Hkv, grp, W, cached lengths
    (128, 2, 4, 1, [0]), (128, 1, 1, 1, [1]), (128, 2, 4, 1, [1023]), (64, 2, 2, 1, [64, 63, 65, 0, 1]),
    (128, 2, 4, 2, [127, 128]), (128, 2, 4, 5, [1024, 3]), (64, 4, 1, 7, [0, 5, 500]), (128, 1, 4, 8, [640, 61]),
    (128, 2, 4, 15, [300, 64]), (128, 1, 4, 16, [2000, 48, 0]), (64, 1, 8, 8, [333]), (64, 3, 5, 3, [100, 1000]),
    (128, 1, 3, 6, [77, 512]), (128, 1, 6, 7, [200]), (64, 2, 7, 9, [190, 2]), (64, 1, 16, 4, [129]),
    (128, 1, 64, 1, [66]), (128, 8, 4, 4, [4097]), (64, 2, 4, 3, [9000]),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hd,Hkv,grp,W,lens", CASES)
@pytest.mark.parametrize("tree", [False, True])
def test_attention_matches_oracle(dtype, hd, Hkv, grp, W, lens, tree):
    if tree and W < 3:
        pytest.skip("a tree needs three rows to differ from a chain")
    spec = spec_()
    parent = [-1] + [(j - 1) // 2 for j in range(1, W)] if tree else None
    c = Cache([n + W for n in lens], Hkv, hd, seed=W)
    held = c.fill(sum(lens) + W)
    q = (2 * torch.randn(len(lens), W, Hkv * grp, hd, generator=torch.Generator().manual_seed(W))).to(dtype)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for hint in (0, max(lens)):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, c.table, parent=parent, max_kv_len=hint)
        for b, n in enumerate(lens):
            check(got[b], *rows_ref(np64(q[b]), held[b], n, parent, dtype=dtype))
    assert torch.equal(got, spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, c.table, parent=parent, max_kv_len=hint))


@pytest.mark.parametrize("hd,grp", [(64, 1), (128, 4)])
def test_ragged_windows_and_untouched_rows(hd, grp):
    spec = spec_()
    W, Hkv = 8, 2
    rows, lens = [3, 0, 8, 1, 5], [65, 12, 0, 1023, 60]
    c = Cache([n + r for n, r in zip(lens, rows)], Hkv, hd)
    held = c.fill(4)
    off = np.concatenate([[2], 2 + np.cumsum(rows)])
    q = torch.randn(int(off[-1]) + 3, Hkv * grp, hd).half()
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table,
                            row_off=torch.tensor(off, dtype=torch.int32, device="cuda"), max_width=W, out=out)
    for b, n in enumerate(lens):
        check(out[off[b]:off[b + 1]], *rows_ref(np64(q[off[b]:off[b + 1]]), held[b], n))
    assert (out[:2] == 9).all() and (out[off[-1]:] == 9).all()
    # a sequence with more rows than max_width: the rest stay as they were
    out.fill_(9)
    spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table,
                            row_off=torch.tensor(off, dtype=torch.int32, device="cuda"), max_width=4, out=out)
    assert (out[off[2] + 4:off[3]] == 9).all()
    check(out[off[2]:off[2] + 4], *rows_ref(np64(q[off[2]:off[2] + 4]), tuple([(held[2][0][0][:4], held[2][0][1][:4]), held[2][1][:4]]), 0))
    # offsets that run past the rows given, or backwards, stay inside the tensors
    wild = torch.tensor([0, 1 << 20, -5, 4, 3, 1 << 30], dtype=torch.int32, device="cuda")
    spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table, row_off=wild)
    torch.cuda.synchronize()


def test_missing_pages_are_masked_and_an_empty_row_is_zero():
    spec = spec_()
    c = Cache([200, 40], 2, 128)
    held = c.fill(6)
    tab = c.table.clone()
    tab[0, 1] = -1
    tab[1, 0] = c.pool.shape[0] + 5
    q = torch.randn(2, 2, 4, 128).half()
    kv_len = torch.tensor([198, 38], dtype=torch.int32, device="cuda")
    got = spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, tab)
    ok = np.ones(200, bool)
    ok[64:128] = False
    check(got[0], *rows_ref(np64(q[0]), held[0], 198, key_ok=ok))
    assert (got[1] == 0).all()
    # lengths outside the page table stay inside it
    for wild in ([-7, 1 << 30], [1 << 20, 38]):
        spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor(wild, dtype=torch.int32, device="cuda"), c.table)
    torch.cuda.synchronize()


@pytest.mark.parametrize("k_gain,v_gain,q_gain", [(1, 1e-6, 1), (1, 2e4, 1), (2e3, 1, 1e-4), (1e-4, 1, 2e3), (30, 1, 8), (1, 1, 0)])
def test_magnitudes(k_gain, v_gain, q_gain):
    """Tiny and huge scales, near one-hot and uniform weights."""
    spec = spec_()
    n, W, hd = 700, 3, 128
    c = Cache([n + W], 1, hd)
    g = torch.Generator().manual_seed(3)
    k = (k_gain * torch.randn(1, n + W, 1, hd, generator=g)).half()
    v = (v_gain * torch.randn(1, n + W, 1, hd, generator=g) * torch.exp(torch.randn(1, n + W, 1, 1, generator=g))).clamp(-6e4, 6e4).half()
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv4_write(k.cuda(), v.cuda(), z, c.table, c.pool)
    q = (q_gain * torch.randn(1, W, 4, hd, generator=g)).half()
    got = spec.spec_kv4_attention(q.cuda(), c.pool, z + n, c.table)
    held = ((O.held(np64(k[0])), O.held(np64(v[0]))), O.quantise(np64(v[0]))[1])
    check(got[0], *rows_ref(np64(q[0]), held, n))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.02, 3.0])
def test_scale(scale):
    spec = spec_()
    c = Cache([150], 2, 64)
    held = c.fill(8)
    q = torch.randn(1, 4, 4, 64).half()
    got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor([146], dtype=torch.int32, device="cuda"), c.table, scale=scale)
    check(got[0], *rows_ref(np64(q[0]), held[0], 146, scale=scale))


def test_tiny_queries_under_a_large_scale():
    """Scores of order one from queries of order 1e-13: such rows are not zeros."""
    spec = spec_()
    c = Cache([150], 2, 128)
    held = c.fill(18)
    q = (1e-13 * torch.randn(1, 2, 4, 128, generator=torch.Generator().manual_seed(1))).bfloat16()
    got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor([148], dtype=torch.int32, device="cuda"), c.table, scale=2.0 ** 40)
    check(got[0], *rows_ref(np64(q[0]), held[0], 148, scale=2.0 ** 40, dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_queries_that_are_not_numbers_are_saturated(dtype):
    """Each such element outweighs the rest of its row, so the row's weight sits on one token."""
    spec = spec_()
    c = Cache([90], 1, 64)
    held = c.fill(19)
    q = torch.randn(1, 4, 1, 64, generator=torch.Generator().manual_seed(2)).to(dtype)
    for j, x in enumerate(("inf", "-inf", "nan")):
        q[0, j, 0, 3 * j] = float(x)
    got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor([86], dtype=torch.int32, device="cuda"), c.table)
    check(got[0], *rows_ref(O.saturate(np64(q[0])), held[0], 86, dtype=dtype))


@pytest.mark.parametrize("lens,W,grp", [([20000], 1, 4), ([9000, 20000, 5], 4, 4), ([12000], 12, 4)])
def test_a_length_bound_that_is_too_small(lens, W, grp):
    """max_kv_len sets the launch shape only: all pages are attended to whatever it says."""
    spec = spec_()
    Hkv, hd = 2, 128
    c = Cache([n + W for n in lens], Hkv, hd, seed=W)
    held = c.fill(20)
    q = torch.randn(len(lens), W, Hkv * grp, hd, generator=torch.Generator().manual_seed(W)).half()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for hint in (1, 64, 300, 700, 2000, 6000):
        got = spec.spec_kv4_attention(q.cuda(), c.pool, kv_len, c.table, max_kv_len=hint)
        for b, n in enumerate(lens):
            check(got[b], *rows_ref(np64(q[b]), held[b], n))


def test_out_may_be_q():
    spec = spec_()
    for lens in ([200, 3], [30000, 64]):
        c = Cache([n + 4 for n in lens], 2, 128)
        c.fill(21)
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q = torch.randn(2, 4, 8, 128).half().cuda()
        want = spec.spec_kv4_attention(q, c.pool, kv_len, c.table)
        assert spec.spec_kv4_attention(q, c.pool, kv_len, c.table, out=q) is q
        assert torch.equal(q, want)


def test_calls_at_once_on_streams_and_in_graphs():
    """Eager calls on two streams and replays of two graphs, in flight together, over caches whose
    sequences are shared by many CTAs: each gives the bits it gives alone."""
    spec = spec_()
    cases = []
    for lens, W in (([9000, 30000], 2), ([20000], 5)):
        c = Cache([n + W for n in lens], 2, 128, seed=W)
        c.fill(22 + W)
        q = torch.randn(len(lens), W, 8, 128, generator=torch.Generator().manual_seed(W)).half().cuda()
        cases.append((q, c.pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table))
    want = [spec.spec_kv4_attention(*a) for a in cases]
    torch.cuda.synchronize()
    graphs, outs = [], [torch.empty_like(a[0]) for a in cases]
    for a, o in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            spec.spec_kv4_attention(*a, out=o)
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append((i, spec.spec_kv4_attention(*cases[i])))
            with torch.cuda.stream(streams[2 + i]):
                graphs[i].replay()
                got.append((i, outs[i].clone()))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)


def test_one_sequence_per_page_order_and_shared_pages():
    """Two sequences over the same pages (a shared prefix) see the same tokens."""
    spec = spec_()
    c = Cache([192], 2, 128)
    c.fill(9)
    tab = c.table.repeat(2, 1).contiguous()
    q = torch.randn(1, 1, 8, 128).half().cuda().repeat(2, 1, 1, 1)
    got = spec.spec_kv4_attention(q, c.pool, torch.tensor([191, 191], dtype=torch.int32, device="cuda"), tab)
    assert torch.equal(got[0], got[1])


def test_cells_past_four_gigabytes():
    spec = spec_()
    first = 62500                                          # 62500 pages of 8 x 8704 bytes: 4.35 GB
    c = Cache([130], 8, 128, first_page=first)
    assert first * 8 * 8704 > 2 ** 32
    held = c.fill(10)
    q = torch.randn(1, 2, 8, 128).half()
    got = spec.spec_kv4_attention(q.cuda(), c.pool, torch.tensor([128], dtype=torch.int32, device="cuda"), c.table)
    check(got[0], *rows_ref(np64(q[0]), held[0], 128))
    k = spec.spec_kv4_read(c.pool, torch.zeros(1, dtype=torch.int32, device="cuda"), c.table, 130)[0]
    assert (np.abs(np64(k[0]) - held[0][0][0]) <= 2.0 ** -10 * np.abs(held[0][0][0]) + 2.0 ** -24).all()


def test_a_round_of_write_and_attend_on_a_side_stream_and_in_a_graph():
    """The serving loop: the window's K/V are written, the window attends, lengths advance; the same
    calls on a side stream and replayed from a captured graph give the same bits."""
    spec = spec_()
    B, W, Hkv, grp, hd = 3, 4, 2, 4, 128
    lens = torch.tensor([100, 0, 63], dtype=torch.int32)
    rounds = [tuple(torch.randn(B, W, h, hd, generator=torch.Generator().manual_seed(10 * i + h)).half().cuda() for h in (Hkv * grp, Hkv, Hkv + 1))
              for i in range(3)]
    base = Cache([120, 20, 80], Hkv, hd, seed=2)
    base.fill(11)

    def one(pool, kv_len, q, k, v, out=None):
        spec.spec_kv4_write(k, v, kv_len, base.table, pool)
        return spec.spec_kv4_attention(q, pool, kv_len, base.table, out=out)

    pool, kv_len, want = base.pool.clone(), lens.cuda(), []
    for q, k, v in rounds:
        want.append(one(pool, kv_len, q, k, v[:, :, :Hkv].contiguous()))
        kv_len = kv_len + W
    torch.cuda.synchronize()

    side, got = torch.cuda.Stream(), []
    pool2 = base.pool.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv_len = lens.cuda()
        for q, k, v in rounds:
            got.append(one(pool2, kv_len, q, k, v[:, :, :Hkv].contiguous()))
            kv_len = kv_len + W
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(pool, pool2)

    pool3, kv_len = base.pool.clone(), lens.cuda()
    q0, k0, v0 = (torch.zeros_like(t) for t in (rounds[0][0], rounds[0][1], rounds[0][1]))
    out = torch.empty_like(q0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one(pool3, kv_len, q0, k0, v0, out=out)
        kv_len += W
    for i, (q, k, v) in enumerate(rounds):
        q0.copy_(q), k0.copy_(k), v0.copy_(v[:, :, :Hkv])
        graph.replay()
        assert torch.equal(out, want[i])
    assert torch.equal(pool3, pool)
