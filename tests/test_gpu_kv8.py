"""8-bit KV cache on the GPU against the fp64 oracle: writes (bit for bit), reads, attention with
accumulated weights, eviction, and a drafter's run of them together."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O4
from oracle import kv8 as O
from oracle import sample as OS
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a step of a rounding, relative


@pytest.fixture(scope="module")
def spec():
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    spec.load_library()
    return spec


def rounded(y, dt):
    """fp64 to the type, once, as a read does."""
    if dt == "fp16":
        y = np.clip(y, -65504, 65504)
    return torch.from_numpy(np.ascontiguousarray(y)).to(DT[dt]).double().numpy()


class Cache:
    """A GPU pool with garbage (all bytes 0xff: NaN codes) in it, page tables in random order, and
    the oracle's view of every (sequence, head)."""

    def __init__(self, spec, B, H, hd, max_pages, seed=0, absent=(), spare=0):
        self.spec, self.B, self.H, self.hd, self.max_pages = spec, B, H, hd, max_pages
        self.rng = np.random.default_rng(seed)
        n = B * max_pages + 3 + spare
        self.pool = spec.spec_kv8_pool(n, H, hd)
        self.pool.fill_(255)
        perm = self.rng.permutation(n)
        table = perm[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.spare = perm[B * max_pages:]
        for b, p in absent:
            table[b, p] = -1 if (b + p) % 2 else n + 5
        self.table_np = table
        self.table = torch.from_numpy(table).cuda()
        T = max_pages * 64
        self.k = [[O.HeldSeq(T, hd, -1) for _ in range(H)] for _ in range(B)]    # the byte 0xff is -1
        self.v = [[O.HeldSeq(T, hd, -1) for _ in range(H)] for _ in range(B)]
        self.here = np.repeat((table >= 0) & (table < n), 64, 1)

    def values(self, n, gain=1.0, dt="fp16"):
        x = self.rng.normal(size=(n, self.H, self.hd)) * np.exp(0.5 * self.rng.normal(size=(1, self.H, self.hd))) * gain
        return torch.from_numpy(x).to(DT[dt])

    def write(self, start, ks, vs, ragged=True, pad=0):
        """ks, vs: per sequence [n_b, H, hd] CPU tensors."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        if ragged:
            off = np.concatenate([[0], np.cumsum([len(k) for k in ks])])
            k, v, row_off = torch.cat(ks).cuda(), torch.cat(vs).cuda(), i32(off.tolist())
        else:
            k, v, row_off = torch.stack(ks).cuda(), torch.stack(vs).cuda(), None
        if pad:  # rows inside a wider projection's output
            wide = torch.full(k.shape[:-2] + (2 * self.H * self.hd + pad,), float("nan"), dtype=k.dtype, device="cuda")
            a, b = wide[..., :self.H * self.hd], wide[..., self.H * self.hd + pad:]
            a.copy_(k.flatten(-2)), b.copy_(v.flatten(-2))
            k, v = a.unflatten(-1, (self.H, self.hd)), b.unflatten(-1, (self.H, self.hd))
        self.spec.spec_kv8_write(k, v, i32(list(start)), self.table, self.pool, row_off=row_off)
        for b in range(self.B):
            for h in range(self.H):
                self.k[b][h].write(int(start[b]), ks[b][:, h].double().numpy())
                self.v[b][h].write(int(start[b]), vs[b][:, h].double().numpy())

    def held(self, b, n):
        """K, V [n, H, hd] of the first n positions, zeros where there is no cell."""
        out = []
        for c in (self.k, self.v):
            y = np.stack([c[b][h].y[:n] for h in range(self.H)], 1)
            out.append(np.where(self.here[b, :n, None, None], y, 0.0))
        return out

    def check_read(self, start, counts, dt, ragged=True):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        off = np.concatenate([[0], np.cumsum(counts)])
        row_off = i32(off.tolist()) if ragged else None
        k, v = self.spec.spec_kv8_read(self.pool, i32(list(start)), self.table, int(off[-1]) if ragged else counts[0], row_off=row_off, dtype=DT[dt])
        k, v = (x.reshape(-1, self.H, self.hd).double().cpu().numpy() for x in (k, v))
        for b in range(self.B):
            ref = self.held(b, self.max_pages * 64)
            for got, r in ((k, ref[0]), (v, ref[1])):
                for j in range(counts[b]):
                    pos = start[b] + j
                    want = r[pos] if 0 <= pos < len(r) else np.zeros_like(r[0])
                    assert np.array_equal(got[off[b] + j], rounded(want, dt)), (b, pos)


# --------------------------------------------------------------------------- write and read
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("hd,H,B", [(64, 3, 5), (128, 2, 3), (128, 1, 1), (64, 8, 40)])
def test_writes_in_any_split_bit_for_bit(spec, hd, H, B, dt):
    c = Cache(spec, B, H, hd, 3, seed=hd + B)
    at = [int(x) for x in c.rng.integers(0, 20, B)]
    c.write([0] * B, [c.values(a, dt=dt) for a in at], [c.values(a, dt=dt) for a in at])
    for step in range(4):
        n = [int(x) for x in c.rng.integers(0, (40, 1, 7, 18)[step] + 1, B)]
        gain = (1.0, 30.0, 0.01, 900.0)[step]            # exponents rise, and do not fall
        c.write(at, [c.values(x, gain, dt) for x in n], [c.values(x, gain, dt) for x in n], pad=8 if step == 2 else 0)
        at = [a + x for a, x in zip(at, n)]
    c.check_read([0] * B, at, dt)
    c.check_read([max(0, a - 5) for a in at], [min(a, 5) for a in at], "fp16")
    if min(at) >= 3:
        c.check_read([a - 3 for a in at], [3] * B, dt, ragged=False)


@pytest.mark.parametrize("hd", [64, 128])
def test_bytes_of_a_block(spec, hd):
    """Where each code lies, which pools that a caller lays out have to hold to."""
    codes = torch.randint(0, 256, (2, 64, 2, hd), generator=torch.Generator().manual_seed(hd), dtype=torch.uint8)
    codes[(codes & 127) == 127] = 1                         # no NaN
    codes[:, ::16] = 126                                    # 448: exponent 0 in every sub-block
    k, v = codes.view(torch.float8_e4m3fn).half()
    pool = spec.spec_kv8_pool(2, 2, hd)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    spec.spec_kv8_write(k[None].cuda(), v[None].cuda(), z, z.view(1, 1) + 1, pool)
    want = torch.zeros(2, 4, 32 * hd + 16, dtype=torch.uint8)
    for t in range(64):
        u, (c, i) = t % 16, (t % 8 // 2, t % 16 // 8 * 2 + t % 2)
        for d in range(hd):
            j, g, n = d // 16, d // (hd // 8), d % (hd // 8)
            at_k = u * hd + ((j ^ (4 * (u % 2))) if hd == 128 else j) * 16 + d % 16
            at_v = 16 * hd + n // 4 * 512 + (4 * g + c) * 16 + n % 4 * 4 + i
            want[:, t // 16, at_k], want[:, t // 16, at_v] = codes[0, t, :, d], codes[1, t, :, d]
    assert torch.equal(pool[1].cpu().view(2, 4, -1), want) and (pool[0] == 0).all()


def test_uniform_rows_overwrite_and_start_anew(spec):
    c = Cache(spec, 2, 2, 128, 2)
    c.write([0, 0], [c.values(60, 50.0)] * 2, [c.values(60, 50.0)] * 2, ragged=False)
    c.write([16, 20], [c.values(9)] * 2, [c.values(9)] * 2, ragged=False)   # a sub-block anew, and within one
    c.check_read([16, 0], [9, 60], "fp16")


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_extreme_values(spec, dt):
    c = Cache(spec, 1, 1, 64, 1)
    fin = torch.finfo(DT[dt])
    vals = [0.0, -0.0, float("nan"), float("inf"), -float("inf"), fin.max, -fin.max, fin.tiny, fin.smallest_normal, 65504.0, 65536.0,
            2.0 ** -24, 2.0 ** -25, 448.0, 464.0, 57344.0, 57345.0, 1e-5, 3.0]
    for lo in range(0, 64, 16):
        x = torch.zeros(16, 1, 64, dtype=DT[dt])
        pick = vals if lo == 0 else [v for v in vals if v == v and abs(v) < (1.0, 500.0, 1e30)[lo // 16 - 1]]
        x.view(-1)[:len(pick)] = torch.tensor(pick, dtype=torch.float64).to(DT[dt])
        c.write([lo], [x], [x.flip(0)])
    c.check_read([0], [64], "fp16")
    c.check_read([0], [64], "bf16")


def test_positions_without_a_cell(spec):
    c = Cache(spec, 3, 2, 64, 2, absent=[(1, 0), (2, 1)])
    c.write([-20, 0, 50], [c.values(30), c.values(128), c.values(100)], [c.values(30), c.values(128), c.values(100)])
    c.check_read([-20, 0, 50], [30, 128, 100], "fp16")
    assert int((c.pool.view(-1, 8256)[:, 32 * 64 + 2:32 * 64 + 16] == 255).all(1).sum()) > 0    # pages of nobody stay as they were


def test_rows_of_no_sequence(spec):
    c = Cache(spec, 2, 1, 64, 1)
    k = c.values(20)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    spec.spec_kv8_write(k.cuda(), k.cuda(), i32([0, 0]), c.table, c.pool, row_off=i32([3, 7, 15]))
    outs = tuple(torch.full((20, 1, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    spec.spec_kv8_read(c.pool, i32([0, 0]), c.table, 20, row_off=i32([3, 7, 15]), outs=outs)
    got = outs[0].cpu()
    assert (got[:3] == 7).all() and (got[15:] == 7).all()
    for lo, hi in ((3, 7), (7, 15)):
        assert np.array_equal(got[lo:hi, 0].double().numpy(), rounded(O.held(k[lo:hi, 0].double().numpy()), "fp16"))


def test_many_sequences_of_one_row(spec):
    B = 3000
    pool = spec.spec_kv8_pool(B, 1, 64)
    table = torch.arange(B, dtype=torch.int32, device="cuda").flip(0).view(B, 1).contiguous()
    start = torch.arange(B, dtype=torch.int32, device="cuda") % 64
    x = torch.randn(B, 1, 1, 64, device="cuda", dtype=torch.float16)
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    spec.spec_kv8_write(x.view(B, 1, 64), x.view(B, 1, 64), start, table, pool, row_off=off)
    a, _ = spec.spec_kv8_read(pool, start, table, 1)
    b, v = spec.spec_kv8_read(pool, start, table, B, row_off=off)
    assert torch.equal(a.view(B, 64), b.view(B, 64)) and torch.equal(b, v)
    # fresh exponents or the pool's zeros' (0): within half a step of either
    assert ((a - x).abs() <= (x.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)).all()


# --------------------------------------------------------------------------- attention
def attention_tolerance(q, k, v, scale, hd, dt):
    """Bound on |out - exact| per row and head.  Scores: fp32 sums of hd exact products, each addition
    within 2^-23 of the largest partial sum (sum of |q k|), and a rounding of the product with the
    scale and of the exp2 (2^-22).  A weight's relative error is twice (numerator and denominator) the score's, plus fp16's half step;
    the sum over tokens weighs |v| <= max|v|.  Then the output's own rounding."""
    mag = np.einsum("nhd,khd->nhk", np.abs(q), np.abs(k)).max() * abs(scale)
    eps = 2 * ((hd + 2) * 2.0 ** -23 * mag + 2.0 ** -22) + 2 * 2.0 ** -11
    vmax = np.abs(v).max()
    return vmax * (eps + HALF[dt])


def run_attention(spec, c, lens, rows, grp, dt="fp16", parent=None, scale=None, ragged=True, weight_len=None, qgain=1.0, qpad=0,
                  max_kv_len=0, width=None, check=True):
    """Attention over c, whose windows are written, against the oracle; returns (out, weight)."""
    Hq, hd = c.H * grp, c.hd
    total = sum(rows)
    q = torch.from_numpy(c.rng.normal(size=(total, Hq, hd)) * qgain).to(DT[dt])
    qg = q.cuda()
    if qpad:
        wide = torch.full((total, Hq * hd + qpad), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, :Hq * hd] = qg.flatten(1)
        qg = wide[:, :Hq * hd].unflatten(1, (Hq, hd))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    off = np.concatenate([[0], np.cumsum(rows)])
    W = width or max(max(rows), 1)
    weight = before = None
    if weight_len:
        weight = torch.rand(c.B, c.H, weight_len, device="cuda")
        before = weight.double().cpu().numpy()
    kw = dict(parent=parent, scale=scale, max_kv_len=max_kv_len, weight=weight)
    if ragged:
        out = spec.spec_kv8_attention(qg, c.pool, i32(lens), c.table, row_off=i32(off.tolist()), max_width=W, **kw)
    else:
        out = spec.spec_kv8_attention(qg.view(c.B, -1, Hq, hd), c.pool, i32(lens), c.table, **kw).view(total, Hq, hd)
    got = out.double().cpu().numpy()
    sc = hd ** -0.5 if scale is None else scale
    wref = before.copy() if weight_len else None
    weps = 0.0
    for b in range(c.B):
        n, L = rows[b], lens[b]
        if not check or n == 0:
            continue
        keys = min(max(L + n, 0), c.max_pages * 64)
        k, v = c.held(b, keys)
        qb = q[off[b]:off[b + 1]].double().numpy()
        qb = np.clip(qb, -65504, 65504)
        first = max(0, -L)                       # window rows before position 0 have no cell
        see = np.zeros((n, keys), bool)
        mask = O4.window_mask(n, parent)
        for j in range(n):
            see[j, :min(max(L, 0), keys)] = True
            for i in range(n):
                if 0 <= L + i < keys and i >= first:
                    see[j, L + i] = mask[j, i]
        see &= c.here[b, :keys]
        ref = np.zeros((n, Hq, hd))
        for h in range(c.H):
            s = np.einsum("ngd,kd->ngk", qb[:, h * grp:(h + 1) * grp], k[:, h]) * sc
            s = np.where(see[:, None], s, -np.inf)
            top = s.max(-1, keepdims=True) if keys else np.full((n, grp, 1), -np.inf)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            tot = p.sum(-1, keepdims=True)
            p = np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)
            ref[:, h * grp:(h + 1) * grp] = np.einsum("ngk,kd->ngd", p, v[:, h])
            if weight_len:
                m = min(keys, weight_len)
                wref[b, h, :m] += p.sum((0, 1))[:m]
        if keys:
            tol = attention_tolerance(qb, np.repeat(k, grp, 1), v, sc, hd, dt)
            if dt == "fp16":
                ref = np.clip(ref, -65504, 65504)
            err = np.abs(got[off[b]:off[b + 1]] - ref).max()
            assert err <= tol, (b, err, tol)
            mag = np.einsum("nhd,khd->nhk", np.abs(qb), np.abs(np.repeat(k, grp, 1))).max() * abs(sc)
            weps = max(weps, 2 * ((hd + 2) * 2.0 ** -23 * mag + 2.0 ** -21))
        else:
            assert (got[off[b]:off[b + 1]] == 0).all()
    if weight_len and check:
        wg = weight.double().cpu().numpy()
        # a share's relative error is the weights'; the running sum rounds once more in fp32
        assert (np.abs(wg - wref) <= (wref - before) * weps + wref * 2.0 ** -23).all()
    return out, weight


def filled(spec, lens, rows, H, hd, max_pages, seed=0, dt="fp16", **kw):
    c = Cache(spec, len(lens), H, hd, max_pages, seed=seed, **kw)
    n = [max(0, a) + b for a, b in zip(lens, rows)]
    c.write([0] * len(lens), [c.values(x, dt=dt) for x in n], [c.values(x, dt=dt) for x in n])
    return c


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("hd,H,grp,W", [(128, 2, 4, 1), (128, 1, 4, 5), (64, 2, 1, 3), (128, 2, 7, 4), (64, 1, 8, 8), (128, 1, 4, 16),
                                        (64, 3, 5, 7), (128, 1, 3, 11), (64, 2, 4, 10)])
def test_attention_shapes(spec, hd, H, grp, W, dt):
    lens = [0, 1, 31, 32, 63, 64, 65, 200, 777]
    rows = [W, 1, W, max(1, W - 1), W, 0, W, (W + 1) // 2, W]
    c = filled(spec, lens, rows, H, hd, 14, seed=W, dt=dt)
    run_attention(spec, c, lens, rows, grp, dt, width=W, weight_len=14 * 64)


@pytest.mark.parametrize("W,parent", [(7, [-1, 0, 0, 1, 1, 2, 2]), (15, [-1] + [(j - 1) // 2 for j in range(1, 15)]), (4, [-1, 0, 0, 0])])
@pytest.mark.parametrize("hd", [64, 128])
def test_trees(spec, W, parent, hd):
    lens, rows = [5, 120, 0], [W] * 3
    c = filled(spec, lens, rows, 2, hd, 3)
    run_attention(spec, c, lens, rows, 4, parent=parent, ragged=False, weight_len=150)


@pytest.mark.parametrize("W,grp", [(1, 4), (4, 4), (16, 4)])
def test_long_caches_are_cut_and_merged(spec, W, grp):
    lens, rows = [9000, 130, 5000], [W] * 3
    c = filled(spec, lens, rows, 1, 128, 150)
    a, w = run_attention(spec, c, lens, rows, grp, weight_len=150 * 64)
    for hint in (1, 100, 1 << 20):                          # a launch shape that does not fit the lengths
        c.rng = np.random.default_rng(5)
        x, _ = run_attention(spec, c, lens, rows, grp, max_kv_len=hint)
        c.rng = np.random.default_rng(5)
        y, _ = run_attention(spec, c, lens, rows, grp, max_kv_len=hint, check=False)
        assert torch.equal(x, y)                            # one order of the sums


@pytest.mark.parametrize("B,H,pages", [(3, 8, 150), (5, 4, 83), (19, 2, 158), (1, 24, 100)])
def test_clusters_of_middling_lengths_need_no_workspace(spec, B, H, pages):
    """20 to 38 groups of 5 to 10 thousand tokens: one cluster each on some GPUs, pieces on others."""
    lens, rows = [pages * 64 - 1] + [300 * b + 5 for b in range(1, B)], [1] * B
    c = filled(spec, lens, rows, H, 64, pages, seed=B)
    run_attention(spec, c, lens, rows, 2)
    run_attention(spec, c, lens, rows, 1, weight_len=pages * 64)


def test_longest_cache(spec):
    lens, rows = [65520], [3]
    c = filled(spec, lens, rows, 1, 64, 1024)
    run_attention(spec, c, lens, rows, 2, weight_len=65523)


def test_many_sequences(spec):
    rng = np.random.default_rng(3)
    B = 70
    lens = [int(x) for x in rng.integers(0, 150, B)]
    rows = [int(x) for x in rng.integers(0, 4, B)]
    c = filled(spec, lens, rows, 2, 64, 3)
    run_attention(spec, c, lens, rows, 4, width=3, qpad=8, weight_len=100)     # weights of the first 100 positions alone


@pytest.mark.parametrize("grp", [1, 4])
def test_windows_before_zero_past_the_table_and_absent_pages(spec, grp):
    lens, rows = [-3, 126, 60, 0], [5, 5, 4, 2]
    c = filled(spec, lens, rows, 1, 64, 2, absent=[(2, 0), (3, 0)])
    run_attention(spec, c, lens, rows, grp, weight_len=128)


def test_pool_past_4_gb(spec):
    """The cells of the last pages of a pool whose byte offsets pass 32 bits."""
    H, hd, n = 8, 128, 33000
    pool = spec.spec_kv8_pool(n, H, hd)
    assert pool.numel() > 2 ** 32
    c = Cache(spec, 1, H, hd, 3, spare=2)
    c.table = torch.tensor([[n - 1, 3, n - 2]], dtype=torch.int32, device="cuda")
    pool[[n - 1, 3, n - 2]] = 255
    c.pool, c.here[:], c.spare = pool, True, np.array([n - 3, n - 4])
    c.write([0], [c.values(170)], [c.values(170)])
    c.check_read([0], [170], "fp16")
    run_attention(spec, c, [168], [2], 2, weight_len=170)
    w = torch.rand(1, H, 170, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dst = i32([[n - 3, n - 4]])
    _, kept, _ = spec.spec_kv8_evict(pool, w, i32([170]), c.table, dst, 100, 10)
    k, _ = spec.spec_kv8_read(pool, i32([0]), dst, 100)
    hk, _ = c.held(0, 170)
    for h in range(H):
        stay = O.keep_tokens(w[0, h].cpu().numpy(), 170, 100, 10)
        assert kept[0, h].tolist() == stay.tolist()
        assert np.array_equal(k[0, :, h].double().cpu().numpy(), rounded(O.held(hk[stay, h]), "fp16"))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(spec, scale):
    lens, rows = [100, 40], [3, 3]
    c = filled(spec, lens, rows, 1, 128, 2)
    run_attention(spec, c, lens, rows, 4, scale=scale)


def test_tiny_and_huge_queries(spec):
    lens, rows = [100], [4]
    c = filled(spec, lens, rows, 1, 64, 2)
    run_attention(spec, c, lens, rows, 2, "bf16", qgain=1e-30, scale=1e10)
    run_attention(spec, c, lens, rows, 2, "bf16", qgain=1e-30, scale=2.0 ** 40)
    run_attention(spec, c, lens, rows, 2, "fp16", qgain=3e4, scale=1e-6)


def test_scores_past_2_to_24_put_all_weight_on_the_largest(spec):
    c = Cache(spec, 1, 1, 64, 4)
    k, v = c.values(200), c.values(200)
    k[37] = 60000.0
    v[37] = torch.arange(64).view(1, 64).to(torch.float16) / 16
    v[48:64] *= 2000                                              # a sub-block of large values without weight
    c.write([0], [k], [v])
    q = torch.full((1, 1, 4, 64), 60000.0, dtype=torch.float16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for scale in (1.0, 2.0 ** 20, 2.0 ** 40):
        out = spec.spec_kv8_attention(q, c.pool, i32([199]), c.table, scale=scale)
        want = rounded(c.held(0, 38)[1][37], "fp16")
        assert np.array_equal(out[0, 0].double().cpu().numpy(), np.repeat(want, 4, 0))


@pytest.mark.parametrize("big", [1, 130])
def test_exponents_of_tokens_without_weight_cost_nothing(spec, big):
    """V of a sub-block 2^15 times the others': its tokens' scores are 60 below, so the result is that of the
    others alone, to their own rounding."""
    c = Cache(spec, 1, 1, 128, 3)
    k, v = c.values(160, 0.05), c.values(160, 0.01)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.float16, device="cuda")
    q[..., 0] = 8.0
    k[:, 0, 0] = 0.0
    s = big // 16 * 16
    k[s:s + 16, 0, 0] = -100.0
    v[s:s + 16] = v[s:s + 16].sign() * 300.0
    c.write([0], [k], [v])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = spec.spec_kv8_attention(q, c.pool, i32([159]), c.table, scale=1.0).double().cpu().numpy()[0, 0]
    kk, vv = c.held(0, 160)
    sc = (q[0, 0].double().cpu().numpy() @ kk[:, 0].T)
    p = np.exp(sc - sc.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref = p @ vv[:, 0]
    rest = np.abs(np.delete(vv[:, 0], np.s_[s:s + 16], 0)).max()
    assert np.abs(out - ref).max() <= rest * 2.0 ** -8


def test_out_may_be_q_and_results_repeat(spec):
    lens, rows = [300, 77], [4, 4]
    c = filled(spec, lens, rows, 2, 128, 6)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, 4, 8, 128, device="cuda", dtype=torch.float16)
    ref = spec.spec_kv8_attention(q, c.pool, i32(lens), c.table)
    out = q.clone()
    assert spec.spec_kv8_attention(out, c.pool, i32(lens), c.table, out=out) is out
    assert torch.equal(out, ref)


# --------------------------------------------------------------------------- eviction
def run_evict(spec, c, lens, weight, keep, recent):
    dst_pages = (keep + 63) // 64
    dst = torch.from_numpy(c.spare[:c.B * dst_pages].reshape(c.B, dst_pages).astype(np.int32)).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool0 = c.pool.clone()
    new_len, kept, wout = spec.spec_kv8_evict(c.pool, weight, i32(lens), c.table, dst, keep, recent)
    src = torch.from_numpy(np.setdiff1d(np.arange(len(c.pool)), dst.cpu().numpy().ravel())).cuda()
    assert torch.equal(c.pool[src], pool0[src])
    k, v = spec.spec_kv8_read(c.pool, torch.zeros(c.B, dtype=torch.int32, device="cuda"), dst, keep)
    w = weight.cpu().numpy()
    for b in range(c.B):
        n = max(0, min(lens[b], w.shape[2], c.max_pages * 64))
        m = min(n, keep)
        assert int(new_len[b]) == m
        hk, hv = c.held(b, n)
        for h in range(c.H):
            stay = O.keep_tokens(w[b, h], n, keep, recent)
            assert kept[b, h].tolist() == stay.tolist() + [-1] * (keep - m), (b, h)
            assert np.array_equal(wout[b, h, :m].cpu().numpy(), w[b, h][stay], equal_nan=True) and (wout[b, h, m:] == 0).all()
            for got, src_ in ((k, hk), (v, hv)):
                if m:
                    assert np.array_equal(got[b, :m, h].double().cpu().numpy(), rounded(O.held(src_[stay, h]), "fp16"))
    return new_len, dst, wout


@pytest.mark.parametrize("hd,H", [(64, 3), (128, 2)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (50, 0), (64, 64), (100, 7), (300, 10)])
def test_evict(spec, hd, H, keep, recent):
    lens = [0, 1, 50, 64, 130, 299]
    c = filled(spec, lens, [0] * 6, H, hd, 5, spare=6 * 5)
    c.write([200] * 6, [c.values(40 if n > 240 else 0, 1000.0) for n in lens], [c.values(40 if n > 240 else 0, 1e-3) for n in lens])
    w = torch.from_numpy(c.rng.random((6, H, 300)).astype(np.float32) ** 8).cuda()
    run_evict(spec, c, lens, w, keep, recent)


def test_evict_ties_nan_and_signed_zeros(spec):
    lens = [200, 200, 200, 200]
    c = filled(spec, lens, [0] * 4, 1, 64, 4, spare=40)
    w = torch.zeros(4, 1, 256)
    w[0] = 1.0
    w[1, 0, ::3] = float("nan")
    w[1, 0, 5] = -float("inf")
    w[2, 0, ::2] = -0.0
    w[3] = -torch.rand(256)
    w[3, 0, 100] = float("inf")
    for keep, recent in ((70, 0), (70, 20), (195, 3)):
        run_evict(spec, c, lens, w.cuda(), keep, recent)


def test_evict_absent_pages_short_weights_and_missing_destinations(spec):
    lens = [250, 120]
    c = filled(spec, lens, [0, 0], 2, 64, 4, absent=[(0, 1)], spare=20)
    w = torch.rand(2, 2, 150, device="cuda")
    run_evict(spec, c, lens, w, 90, 30)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    before = c.pool.clone()
    dst = torch.tensor([[-1, len(c.pool)], [len(c.pool) + 7, -5]], dtype=torch.int32, device="cuda")
    new_len, kept, _ = spec.spec_kv8_evict(c.pool, w, i32(lens), c.table, dst, 90, 30)
    assert torch.equal(c.pool, before) and new_len.tolist() == [90, 90] and (kept >= 0).all()


@pytest.mark.parametrize("n", [48 * 1024, 48 * 1024 + 1, 65520])
def test_evict_long(spec, n):
    """The threshold from weights in shared memory, and from longer ones read again."""
    c = Cache(spec, 1, 1, 64, 1024, spare=200)
    c.pool.zero_()
    w = torch.rand(1, 1, n, device="cuda")
    w[0, 0, :500] = w[0, 0, 600]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dst = torch.from_numpy(c.spare[:160].astype(np.int32)).view(1, 160).cuda()
    for keep, recent in ((10000, 128), (int((w > w[0, 0, 600]).sum()) + 250, 0)):
        _, kept, wout = spec.spec_kv8_evict(c.pool, w, i32([n]), c.table, dst[:, :max(160, 1)], min(keep, 10240), recent)
        want = O.keep_tokens(w[0, 0].cpu().numpy(), n, min(keep, 10240), recent)
        assert kept[0, 0].tolist() == want.tolist()
        assert torch.equal(wout[0, 0, :len(want)], w[0, 0][torch.from_numpy(want).cuda()])


# --------------------------------------------------------------------------- streams, graphs, devices
def test_captured_and_replayed_beside_eager_calls(spec):
    lens, rows = [500, 90], [2, 2]
    c = filled(spec, lens, rows, 2, 128, 9, spare=10)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, 2, 8, 128, device="cuda", dtype=torch.float16)
    k = torch.randn(2, 2, 2, 128, device="cuda", dtype=torch.float16)
    L, dst = i32(lens), torch.from_numpy(c.spare[:4].reshape(2, 2).astype(np.int32)).cuda()
    w0 = torch.zeros(2, 2, 576, device="cuda")
    logits, u = torch.randn(4, 5000, device="cuda"), torch.rand(4, device="cuda")

    def step(w):
        spec.spec_kv8_write(k, k, L, c.table, c.pool)
        o = spec.spec_kv8_attention(q, c.pool, L, c.table, weight=w)
        e = spec.spec_kv8_evict(c.pool, w, L, c.table, dst, 100, 10)
        r = spec.spec_kv8_read(c.pool, torch.zeros_like(L), dst, 90)
        return (o,) + e + r + spec.spec_sample(logits, u, 0.8, top_k=50, top_p=0.9, return_probs=True)

    w1 = w0.clone()
    ref = step(w1)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        w = w0.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = step(w)
        graphs.append((g, w, out))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, w, out in graphs:
            w.copy_(w0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ref, out)) and torch.equal(w, w1)


def test_calls_at_once_on_two_streams(spec):
    lens, rows = [4000, 900], [1, 1]
    c = filled(spec, lens, rows, 2, 128, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    L = i32(lens)
    qs = [torch.randn(2, 1, 8, 128, device="cuda", dtype=torch.float16) for _ in range(2)]
    ref = [spec.spec_kv8_attention(q, c.pool, L, c.table) for q in qs]
    logits, u = torch.randn(3, 100000, device="cuda"), torch.rand(3, device="cuda")
    tok = spec.spec_sample(logits, u, top_p=0.9)[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((spec.spec_kv8_attention(qs[i], c.pool, L, c.table), spec.spec_sample(logits, u, top_p=0.9)[0]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, ref[i]) and torch.equal(t, tok) for o, t in got[i])


# --------------------------------------------------------------------------- together
def test_a_drafters_steps(spec):
    """Prompt in, decode steps with weights kept, eviction, more steps on the smaller cache, draft tokens with
    their q, and the acceptance of them."""
    c = Cache(spec, 2, 2, 64, 6, spare=8)
    H, hd, grp = 2, 64, 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [250, 133]
    c.write([0, 0], [c.values(n) for n in lens], [c.values(n) for n in lens])
    weight = torch.zeros(2, H, 384, device="cuda")
    wref = np.zeros((2, H, 384))
    for _ in range(3):
        c.write(lens, [c.values(1)] * 2, [c.values(1)] * 2, ragged=False)
        q = torch.from_numpy(c.rng.normal(size=(2, 1, H * grp, hd))).to(torch.float16)
        out = spec.spec_kv8_attention(q.cuda(), c.pool, i32(lens), c.table, weight=weight)
        for b in range(2):
            k, v = c.held(b, lens[b] + 1)
            ref, probs = O4.attention(q[b].double().numpy(), k, v, lens[b])
            assert np.abs(out[b].double().cpu().numpy() - ref).max() <= np.abs(v).max() * 2.0 ** -8
            for h in range(H):
                wref[b, h, :lens[b] + 1] += probs[h].sum((0, 1))
        lens = [n + 1 for n in lens]
    assert np.abs(weight.double().cpu().numpy() - wref).max() <= 1e-4
    new_len, dst, weight2 = run_evict(spec, c, lens, weight, 100, 20)
    # the smaller cache goes on in its new pages
    small = Cache(spec, 2, H, hd, 2)
    small.pool, small.table, small.here[:] = c.pool, dst, True
    for b in range(2):
        k, v = c.held(b, lens[b])
        for h in range(H):
            stay = O.keep_tokens(weight[b, h].cpu().numpy(), lens[b], 100, 20)
            small.k[b][h].write(0, k[stay, h]), small.v[b][h].write(0, v[stay, h])
    lens = new_len.tolist()
    small.write(lens, [small.values(3)] * 2, [small.values(3)] * 2, ragged=False)
    run_attention(spec, small, lens, [3, 3], grp, ragged=False)
    # drafts from logits, and their acceptance against a target near the draft
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(2, 4, 1000, generator=g) * 3
    u = torch.rand(2, 4, generator=g)
    x, qd = spec.spec_sample(logits.cuda(), u.cuda(), 0.9, top_k=[40, 0], top_p=[1.0, 0.9], rows_per_setting=4, return_probs=True)
    for b in range(2):
        for j in range(4):
            t, qr, near = OS.sample(logits[b, j].numpy(), u[b, j].item(), np.float32(0.9), (40, 0)[b], (1.0, np.float32(0.9))[b])
            assert near > 1e-9 and int(x[b, j]) == t
            assert np.abs(qd[b, j].double().cpu().numpy() - qr).max() <= 2.0 ** -22
    acc, com, bon = spec.spec_accept_probs(torch.cat([qd, qd[:, :1]], 1), qd, x, torch.rand(2, 5, device="cuda"))
    assert acc.tolist() == [4, 4] and torch.equal(com[:, :4], x)       # p = q accepts everything
