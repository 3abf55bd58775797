"""The model with its KV cache in 4 bits, against the oracle decoder over the same cells.

The GPU's K and V differ from the oracle's by the activations' rounding before they are quantised, so a value
next to a border may take the neighbouring code, a step of 1/15 of its vector's range.  So the oracle attends
to the cells that the GPU wrote, and each of them is compared with the oracle's own K or V: within half a step
and the decoder's stated 1e-2 of the maximum.  Logits over the same cells are within that 1e-2."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from oracle.decoder import OracleDecoder, weights_to_numpy
from speculative_decoding_verify_step_gb300 import synth
from tests._gpu import need_gpu, rel_err, top2_gap

pytestmark = pytest.mark.gpu


class Held(np.ndarray):
    """A KV store that keeps what the 4-bit cache holds of every vector written to it; with `given`, the
    cells [layer][(page, offset)] of a window, those, and the distances to the vectors written."""

    given = None

    def __setitem__(self, at, value):
        if self.given is None or len(at) != 4 or not isinstance(at[0], int):
            super().__setitem__(at, O.held(value))
            return
        layer, page, _, off = at
        cell = self.given[layer][(page, off)]
        step = (value.max(-1, keepdims=True) - value.min(-1, keepdims=True)) / 15
        assert (np.abs(cell - value) <= 0.51 * step + 1e-2 * np.abs(value).max()).all()
        super().__setitem__(at, cell)


class Kv4Oracle(OracleDecoder):
    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.kv.k, self.kv.v = self.kv.k.view(Held), self.kv.v.view(Held)

    def forward_over_cells_of(self, m, ids, tok, parent=None):
        """forward(), the window's cells being those that model m wrote."""
        W = tok.shape[1]
        k, v = [{} for _ in range(self.dims.n_layers)], [{} for _ in range(self.dims.n_layers)]
        for s in ids:
            n = self.kv.length[s]
            self.kv.ensure(s, n + W)
            for layer in range(self.dims.n_layers):
                for store, x in zip((k, v), m.read_kv(layer, s, n, W)):
                    for j in range(W):
                        store[layer][self.kv.slot(s, n + j)] = x[j].double().numpy()
        self.kv.k.given, self.kv.v.given = k, v
        try:
            return self.forward(ids, tok, parent)
        finally:
            self.kv.k.given = self.kv.v.given = None


DIMS = synth.TINY
WIDE = synth.Dims(n_layers=2, d_model=512, n_heads=8, n_kv_heads=2, head_dim=128, ffn_dim=512, vocab=512)


def models(dims, seed=1, **kw):
    need_gpu()
    from speculative_decoding_verify_step_gb300 import spec
    w = synth.make_weights(dims, seed=seed, gain_jitter=0.1)
    m = spec.SpecModel(dims, kv_format="int4", **kw)
    m.load_weights((k, v.cuda()) for k, v in w.items())
    orc = Kv4Oracle(dims, weights_to_numpy(w), **{k: kw[k] for k in ("max_batch", "max_seq_len", "num_pages")})
    return m, orc


@pytest.fixture(scope="module", params=["tiny", "wide"])
def pair(request):
    m, orc = models(DIMS if request.param == "tiny" else WIDE, max_batch=3, max_width=16, max_seq_len=1024, num_pages=60)
    yield m, orc
    m.close()


def start(m, orc, lens, seed=0):
    """Sequences with given caches on both sides."""
    d = m.dims
    rng = np.random.default_rng(seed)
    m.seq_reset(list(range(m.cfg.max_batch)))
    orc.reset(range(m.cfg.max_batch))
    for s, n in enumerate(lens):
        k, v = (torch.from_numpy(rng.normal(size=(d.n_layers, n, d.n_kv_heads, d.head_dim)) * 0.5).half() for _ in range(2))
        m.kv_write(s, k, v)
        orc.load_cache(s, k.double().numpy(), v.double().numpy())


def gpu_logits(m, ids, tok, parent=None):
    out = m.score(ids, torch.as_tensor(tok), parent=parent).cpu().double().numpy()
    m.sync_status()
    return out


def held_rows(orc, layer, s, t0, n):
    rows = [orc.kv.slot(s, t) for t in range(t0, t0 + n)]
    return tuple(np.asarray([np.asarray(x[layer, pg, :, off]) for pg, off in rows]) for x in (orc.kv.k, orc.kv.v))


@pytest.mark.parametrize("lens,W,tree", [([0, 1, 63], 1, False), ([64, 130, 7], 3, False), ([700, 0, 333], 8, False),
                                         ([65, 129, 500], 15, True), ([126, 62, 3], 16, False)])
def test_window_logits_and_cells_match_the_oracle(pair, lens, W, tree):
    m, orc = pair
    if W * (m.dims.n_heads // m.dims.n_kv_heads) > 64:
        W = 16
    start(m, orc, lens, seed=W)
    parent = [-1] + [(j - 1) // 2 for j in range(1, W)] if tree else None
    tok = np.random.default_rng(W).integers(0, m.dims.vocab, (3, W))
    got = gpu_logits(m, [0, 1, 2], tok, parent)
    ref = orc.forward_over_cells_of(m, [0, 1, 2], tok, None if parent is None else np.array(parent))
    assert rel_err(got, ref) < 1e-2


def test_kv_write_read_and_fill_hold_the_quantised_values(pair):
    m, orc = pair
    start(m, orc, [300, 65, 1], seed=5)
    for s, n in enumerate([300, 65, 1]):
        for layer in range(m.dims.n_layers):
            for x, y in zip(m.read_kv(layer, s, 0, n), held_rows(orc, layer, s, 0, n)):
                assert (np.abs(x.double().numpy() - y) <= 2.0 ** -10 * np.abs(y) + 2.0 ** -24).all()
    lens, pages = m.kv_state([0, 1, 2])
    assert lens == [300, 65, 1] and [sum(p >= 0 for p in row) for row in pages] == [5, 2, 1]
    # the pseudo-random fill is the fp16 cache's, quantised
    from speculative_decoding_verify_step_gb300 import spec
    f = spec.SpecModel(m.dims, max_batch=3, max_width=16, max_seq_len=1024, num_pages=60)
    for x in (m, f):
        x.seq_reset([0, 1, 2])
        x.kv_fill_random([1, 0], [70, 5], seed=9, scale=0.5)
    for layer in range(m.dims.n_layers):
        for a, b in zip(m.read_kv(layer, 1, 0, 70), f.read_kv(layer, 1, 0, 70)):
            b = O.held(b.double().numpy())
            assert (np.abs(a.double().numpy() - b) <= 2.0 ** -10 * np.abs(b) + 2.0 ** -24).all()
    f.close()


def test_verify_rounds_accept_what_decode_steps_produce(pair, margins):
    """A token's cell does not depend on the window it was written in: with the decode steps' own tokens as
    drafts, greedy rounds accept them wherever the logits' margin is clear."""
    m, orc = pair
    start(m, orc, [100, 64, 0], seed=7)
    tok = torch.tensor([3, 5, 7], dtype=torch.int32, device="cuda")
    seqs, gaps = [tok.cpu().numpy()], []
    for _ in range(12):
        tok = m.decode_step([0, 1, 2], tok)
        gaps.append(top2_gap(m.debug_logits(3).cpu().numpy()))
        seqs.append(tok.cpu().numpy())
    m.sync_status()
    seqs, gaps = np.array(seqs), np.array(gaps)
    cells = [m.read_kv(1, s, 0, n + 12) for s, n in enumerate([100, 64, 0])]
    start(m, orc, [100, 64, 0], seed=7)
    at, near, compared = 0, 0, 0
    while at + 4 <= 12:
        acc, com, _ = m.verify_step([0, 1, 2], torch.as_tensor(seqs[at:at + 4].T.copy()))
        m.sync_status()
        for b in range(3):
            clear = (gaps[at:at + 4, b] > 1e-2).all()
            near += not clear
            if clear:
                compared += 1
                assert int(acc[b]) == 3 and com[b].cpu().tolist() == seqs[at + 1:at + 5, b].tolist()
        if not (acc == 3).all():
            break
        at += 4
    margins(compared, near)
    assert compared > 0
    if at == 12:
        for s, n in enumerate([100, 64, 0]):
            for a, b in zip(cells[s], m.read_kv(1, s, 0, n + 12)):
                a, b = a.double().numpy(), b.double().numpy()
                assert (np.abs(a - b) > 0.02 * np.abs(a).max()).mean() < 0.05


def test_tree_commit_moves_the_accepted_cells(pair):
    m, orc = pair
    parent = [-1, 0, 0, 1, 1, 2, 2]
    moved = 0
    for seed in range(6):
        start(m, orc, [120, 62, 9], seed=20 + seed)
        rng = np.random.default_rng(seed)
        # children of the root: the target's own choice and another token, then again below it
        tok = np.zeros((3, 7), np.int64)
        tok[:, 0] = rng.integers(0, m.dims.vocab, 3)
        first = gpu_logits(m, [0, 1, 2], tok[:, :1])[:, 0].argmax(-1)
        tok[:, 1], tok[:, 2] = (first + 1) % m.dims.vocab, first
        nxt = gpu_logits(m, [0, 1, 2], tok[:, [0, 2]])[:, 1].argmax(-1)
        tok[:, 3], tok[:, 4], tok[:, 5], tok[:, 6] = nxt, first, (nxt + 1) % m.dims.vocab, nxt
        gpu_logits(m, [0, 1, 2], tok, parent)
        before = [[m.read_kv(layer, s, n, 7) for layer in range(m.dims.n_layers)] for s, n in enumerate([120, 62, 9])]
        acc, com, bon = m.verify_tree_step([0, 1, 2], torch.as_tensor(tok), parent)
        m.sync_status()
        lens, _ = m.kv_state([0, 1, 2])
        for s, n in enumerate([120, 62, 9]):
            node, path = 0, []
            for t in com[s].cpu().tolist()[:int(acc[s])]:
                node = next(c for c in range(7) if parent[c] == node and tok[s, c] == t)
                path.append(node)
            assert lens[s] == n + 1 + len(path)
            for layer in range(m.dims.n_layers):
                now = m.read_kv(layer, s, n, 1 + len(path))
                for a, b in zip(now, before[s][layer]):
                    assert torch.equal(a, b[[0] + path])
            moved += sum(d != c for d, c in enumerate(path, 1))
    assert moved > 0


def test_sampled_ragged_and_full_rounds_run_and_agree(pair):
    """Sampled rounds: ragged compact and cap-accept give one decision on one state; temperature, top-k and
    top-p rounds commit."""
    m, orc = pair
    V, W = m.dims.vocab, 5
    rng = np.random.default_rng(3)
    tok = rng.integers(0, V, (3, W))
    q = torch.softmax(torch.from_numpy(rng.normal(size=(3, W - 1, V))).float(), -1).cuda()
    u = torch.from_numpy(rng.random((3, W))).float().cuda()
    vl = [5, 2, 3]
    res = []
    from speculative_decoding_verify_step_gb300 import spec
    for mode in (spec.RAGGED_CAP_ACCEPT, spec.RAGGED_COMPACT):
        start(m, orc, [200, 31, 64], seed=4)
        t = torch.as_tensor(tok) if mode == spec.RAGGED_CAP_ACCEPT else torch.cat([torch.as_tensor(tok[b, :vl[b]]) for b in range(3)])
        acc, com, bon = m.verify_ragged([0, 1, 2], t, vl, mode, q=q, u=u, temperature=1.0, gamma=W - 1)
        m.sync_status()
        res.append((acc.tolist(), m.kv_state([0, 1, 2])[0]))
    assert res[0] == res[1]
    start(m, orc, [200, 31, 64], seed=4)
    acc, com, bon = m.verify_step([0, 1, 2], torch.as_tensor(tok), q=q, u=u, temperature=0.8, top_k=[20, 0, 5], top_p=[0.9, 1.0, 0.5])
    m.sync_status()
    assert m.kv_state([0, 1, 2])[0] == [n + 1 + int(a) for n, a in zip([200, 31, 64], acc)]


def test_prefill_matches_the_oracle(pair):
    m, orc = pair
    m.seq_reset([0, 1, 2])
    orc.reset([0, 1, 2])
    prompts = synth.prompts(3, 90, m.dims.vocab, seed=2)
    lens = [90, 17, 66]
    m.prefill([0, 1, 2], prompts.cuda(), lens)
    for s, n in enumerate(lens):
        if n > 1:
            orc.forward_over_cells_of(m, [s], prompts[s:s + 1, :n - 1].numpy())
            orc.kv.truncate(s, n - 1)
    tok = np.array([[int(prompts[b, n - 1]), 1, 2] for b, n in enumerate(lens)])
    got = gpu_logits(m, [0, 1, 2], tok)
    assert rel_err(got, orc.forward_over_cells_of(m, [0, 1, 2], tok)) < 1e-2


def test_long_caches_split_over_many_ctas():
    m, orc = models(synth.Dims(n_layers=1, d_model=256, n_heads=8, n_kv_heads=2, head_dim=128, ffn_dim=256, vocab=256),
                    max_batch=4, max_width=5, max_seq_len=8192, num_pages=330)
    lens = [5000, 64, 7001, 0]
    start(m, orc, lens, seed=1)
    tok = np.random.default_rng(0).integers(0, 256, (4, 5))
    got = gpu_logits(m, [0, 1, 2, 3], tok)
    assert rel_err(got, orc.forward_over_cells_of(m, [0, 1, 2, 3], tok)) < 1e-2
    m.close()


def test_capacity_and_repeated_ids_leave_the_cache_alone():
    from speculative_decoding_verify_step_gb300 import spec
    m, orc = models(DIMS, max_batch=2, max_width=4, max_seq_len=256, num_pages=3)
    start(m, orc, [64, 120], seed=1)
    before = [m.read_kv(0, s, 0, n) for s, n in enumerate([64, 120])]
    tok = torch.ones(2, 4, dtype=torch.int32)
    m.verify_step([0, 1], tok)                           # sequence 0 needs a page, none is left
    with pytest.raises(spec.SpecError) as e:
        m.sync_status()
    assert e.value.status == 4 and m.kv_state([0])[0] == [64]
    m.verify_step([1, 1], tok)
    with pytest.raises(spec.SpecError) as e:
        m.sync_status()
    assert e.value.status == 1
    for s, n in enumerate([64, 120]):
        for a, b in zip(before[s], m.read_kv(0, s, 0, n)):
            assert torch.equal(a, b)
    m.close()
