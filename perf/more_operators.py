"""Measured cases of what a drafter's own decode step needs beside the verify round: an 8-bit
paged KV cache (written, attended over, cut down by accumulated attention weight) and the
sampler that turns draft logits into a token and the distribution q it was drawn from.

The cache.  A page holds 64 tokens; per kv head it is four sub-blocks of 16 tokens.  A
sub-block has one power-of-two scale 2^e for K and one for V (-15 <= e <= 8) and holds each
value x as the e4m3 number nearest to clamp(x, -65504, 65504) / 2^e (ties to even).  Writing the first
token of a sub-block sets e to the least exponent whose 448 * 2^e reaches the largest of the
call's values there; a later write into it only raises e, and what the sub-block held is then
rounded to the coarser grid.  Sub-block bytes: 16 * hd K codes, 16 * hd V codes, then 16 bytes
whose first two are e of K and e of V (signed).  `_k_place` and `_v_place` give a code's byte.

Attention.  Row j of sequence b's window (tokens kv_len .. kv_len + n_b - 1 of its page table)
attends to every cached token and to the window rows that are its ancestors (chain: 0..j); query
head h reads kv head h // (Hq / Hkv); softmax scale 1/sqrt(head_dim).  With `weight`
[B, Hkv, T], weight[b, h, t] grows by what the window's rows and the heads of kv head h give
token t.

Eviction.  Of each (sequence, kv head)'s n tokens min(keep, n) stay: the `recent` last ones and
those of the largest weight (ties: the earlier token).  They move, in order, to the first cells
of other pages, as if written there; their weights move along.

Sampling.  With x_v = (l_v - max l) / temperature, R_v = floor(2^40 e^x_v).  Ranked by logit (ties: the
lower index), the kept tokens are the shortest prefix of: the top_k first; the first whose R
reach top_p of the top-k's sum; those with R_v >= min_p 2^40.  q_v = R_v / Z, Z the kept sum; the
token is the first whose running kept sum (by index) exceeds floor(floor(2^24 u) Z / 2^24).
"""
import math

import numpy as np
import torch

own = False

PAGE, SUB = 64, 16


def listed():
    big = dict(hq=32, hkv=8, hd=128)    # the 8B decoder shape
    tiny = dict(hq=4, hkv=4, hd=64)     # the 2-layer decoder's heads
    att = dict(kind="attention", dtype="fp16", tree=False, ragged=False, weight=False)
    smp = dict(kind="sample", dtype="fp32", temperature=0.7, top_k=0, top_p=1.0, min_p=0.0, mixed=False, probs=False)
    return [
        # one token of one sequence: the smallest decode step
        dict(att, name="decode_1x1024", b=1, len_min=1024, len_max=1024, w=1, **big),
        # the long-context batch: the cache is most of the step's bytes
        dict(att, name="verify_8x32768_w4", b=8, len_min=32768, len_max=32768, w=4, **big),
        # a full serving batch of mixed lengths
        dict(att, name="verify_64x512-2048_w5", b=64, len_min=512, len_max=2048, w=5, **big),
        # small heads, bf16, odd lengths from an empty cache on, windows of 1..7 rows
        dict(att, name="ragged_bf16_16x0-5003", b=16, len_min=0, len_max=5003, w=7, **tiny) | {"dtype": "bf16", "ragged": True},
        # decode steps that also keep each token's attention weight, for eviction
        dict(att, name="weights_8x16384", b=8, len_min=16384, len_max=16384, w=1, **big) | {"weight": True},
        # the write of one verify window of 16 sequences into caches under way, read back
        dict(kind="write", name="write_16x5", dtype="fp16", b=16, len_min=100, len_max=1777, w=5, ragged=False, **big),
        # prompts written at once (the cache of a prefill computed elsewhere), read back
        dict(kind="write", name="write_8x8192", dtype="fp16", b=8, len_min=0, len_max=0, w=8192, ragged=False, **big),
        # two short contexts cut down to an odd length
        dict(kind="evict", name="evict_2x411-1777_to_601", dtype="bf16", b=2, len_min=411, len_max=1777, keep=601, recent=64, **tiny),
        # a drafter's long contexts cut down to 2048 tokens
        dict(kind="evict", name="evict_8x32768_to_2048", dtype="fp16", b=8, len_min=32768, len_max=32768, keep=2048, recent=256, **big),
        # one draft token from the 8B vocabulary, nucleus sampling
        dict(smp, name="sample_1x128256_topp", rows=1, v=128256, top_p=0.95),
        # a batch of draft tokens with the rows q that the verify round asks for
        dict(smp, name="sample_64x128256_q", rows=64, v=128256, top_k=50, top_p=0.95, probs=True),
        # bf16 logits, an odd vocabulary, every sequence with settings of its own
        dict(smp, name="sample_bf16_256x50257", dtype="bf16", rows=256, v=50257, temperature=1.0, top_k=200, top_p=0.9, min_p=0.02, mixed=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attention", "attention", "attention", "write", "evict", "sample", "sample"])
    if kind == "sample":
        v = log(300, 200000)
        rows = log(1, max(1, min(1024, 64 * 128256 // v)))
        return dict(kind=kind, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), rows=rows, v=v, temperature=rng.choice([1.0, 0.7, 1.3]),
                    top_k=rng.choice([0, 0, log(1, 1000)]), top_p=rng.choice([1.0, 0.95, 0.8]), min_p=rng.choice([0.0, 0.0, 0.05]),
                    mixed=rng.random() < 0.4, probs=rng.random() < 0.5)
    hd, hkv, grp = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
    case = dict(kind=kind, dtype=rng.choice(["fp16", "fp16", "bf16"]), hd=hd, hkv=hkv)
    most = 8 * 32768 * 8 * 128          # cached values of one tensor in the largest listed case
    if kind == "attention":
        w = rng.randint(1, min(16, 64 // grp))
        b = log(1, 64)
        hi = log(1, max(1, min(65520, most // (4 * b * hkv * hd))))
        lo = rng.choice([hi, int(hi * rng.random())])
        return dict(case, b=b, len_min=lo, len_max=hi, w=w, hq=hkv * grp, tree=w > 2 and rng.random() < 0.4, ragged=rng.random() < 0.4, weight=rng.random() < 0.3)
    if kind == "evict":
        b = log(1, 16)
        hi = log(16, max(16, min(65520, most // (4 * b * hkv * hd))))
        keep = log(1, hi)
        return dict(case, b=b, len_min=rng.choice([hi, int(hi * rng.random())]), len_max=hi, keep=keep, recent=rng.randint(0, keep), hq=hkv)
    n = log(1, 8192)
    b = log(1, max(1, min(64, most // (4 * n * hkv * hd))))
    hi = rng.randint(0, 2000)
    return dict(case, b=b, len_min=rng.choice([hi, 0]), len_max=hi, w=n, ragged=rng.random() < 0.4, hq=hkv)


# ------------------------------------------------------------------ what a case stands for
def _lens(c):
    """Cached tokens of each sequence, spread evenly from len_min to len_max."""
    b = c["b"]
    return [c["len_min"] + (c["len_max"] - c["len_min"]) * i // max(1, b - 1) if b > 1 else c["len_max"] for i in range(b)]


def _rows(c):
    """Rows of each sequence: w, or between 1 and w where the batch is ragged."""
    if c["kind"] == "evict":
        return [0] * c["b"]
    return [1 + (7 * i + c["w"] - 1) % c["w"] if c["ragged"] else c["w"] for i in range(c["b"])]


def _parents(c):
    return [-1] + [(j - 1) // 2 for j in range(1, c["w"])] if c.get("tree") else None


def _dtype(c):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[c["dtype"]]


def work(case):
    c = case
    if c["kind"] == "sample":
        n = c["rows"] * c["v"]
        return {"bytes": n * ((4 if c["dtype"] == "fp32" else 2) + (4 if c["probs"] else 0)) + 8 * c["rows"], "flops": 8 * n}
    lens, rows, hd = _lens(c), _rows(c), c["hd"]
    cell = 2 * hd + 0.125               # K, V and their sub-block's share of the exponents
    if c["kind"] == "attention":
        keys = sum(n + r for n, r in zip(lens, rows))
        par, depth, vis = _parents(c), [0], 0
        for j in range(1, c["w"]):
            depth.append(depth[par[j] if par else j - 1] + 1)
        for n, r in zip(lens, rows):
            vis += sum(n + depth[j] + 1 for j in range(r))
        return {"bytes": keys * c["hkv"] * (cell + (8 if c["weight"] else 0)) + 4 * sum(rows) * c["hq"] * hd, "flops": 4 * vis * c["hq"] * hd}
    if c["kind"] == "write":
        n = sum(rows) * c["hkv"]
        return {"bytes": n * (4 * hd + cell + 4 * hd), "flops": 2 * n * hd * 4}
    kept = sum(min(n, c["keep"]) for n in lens) * c["hkv"]
    full = c["b"] * c["hkv"] * c["len_max"]
    return {"bytes": sum(lens) * c["hkv"] * 4 + full * 4 + kept * (2 * cell + 4 * hd) + c["b"] * c["hkv"] * c["keep"] * 4, "flops": 4 * kept * hd}


# ---------------------------------------------------------------------------- the inputs
def _k_place(t, d, hd):
    """Byte of K's code for token t of a sub-block, dim d: 16-byte chunks of a token, those of odd tokens with
    halves exchanged at head_dim 128."""
    j = d // 16
    return t * hd + ((j ^ (4 * (t % 2)) if hd == 128 else j) * 16) + d % 16


def _v_place(t, d, hd):
    """Byte of V's code: a word holds one dim of tokens 2c, 2c + 1, 2c + 8, 2c + 9."""
    per = hd // 8
    g, i, c, byte = d // per, d % per, t % 8 // 2, t // 8 * 2 + t % 2
    return 16 * hd + i // 4 * 512 + (g * 4 + c) * 16 + i % 4 * 4 + byte


def _places(hd, dev):
    """[16 * hd] bytes in a sub-block of every K code, and of every V code."""
    t = torch.arange(SUB, device=dev).unsqueeze(1)
    d = torch.arange(hd, device=dev).unsqueeze(0)
    return _k_place(t, d, hd).reshape(-1), _v_place(t, d, hd).reshape(-1)


def _clamped(x):
    return torch.nan_to_num(x.float(), nan=-65504.0).clamp(-65504.0, 65504.0)


def _exponent(a):
    """Least e in -15..8 with a <= 448 * 2^e, for a >= 0."""
    m, x = torch.frexp(a)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -15)).clamp(-15, 8)


def _codes(x, e):
    """x on the e4m3 grid of scale 2^e, as fp8."""
    return torch.ldexp(x, -e).to(torch.float8_e4m3fn)


def _pack(k, v):
    """Sub-blocks [n, 32 * hd + 16] bytes of k, v [n, 16, hd]."""
    n, _, hd = k.shape
    out = torch.zeros(n, 32 * hd + 16, dtype=torch.uint8, device=k.device)
    for i, (x, at) in enumerate(zip((k, v), _places(hd, k.device))):
        x = _clamped(x)
        e = _exponent(x.abs().amax((1, 2), keepdim=True))
        out[:, at] = _codes(x, e).view(torch.uint8).reshape(n, -1)
        out[:, 32 * hd + i] = e.view(-1).to(torch.int8).view(torch.uint8)
    return out


def _values(shape, gen, dtype):
    """Keys or values as attention layers make them: some channels far larger than others."""
    dev = gen.device
    x = torch.randn(shape, generator=gen, device=dev)
    gain = torch.exp(0.5 * torch.randn(shape[-2:], generator=gen, device=dev))
    return (x * gain + 0.3 * torch.randn(shape[-2:], generator=gen, device=dev)).to(dtype)


def _prepare_sample(c, gen):
    """Logits of a language model's kind: a broad body and a few dozen candidates above it."""
    dev, r, v = gen.device, c["rows"], c["v"]
    x = 2.0 * torch.randn(r, v, generator=gen, device=dev)
    few = min(40, v)
    at = torch.randint(0, v, (r, few), generator=gen, device=dev)
    x.scatter_add_(1, at, 8.0 - 3.0 * torch.log1p(torch.arange(few, device=dev, dtype=torch.float32)).expand(r, few))
    s = dict(case=c, logits=x.to(_dtype(c)), u=torch.rand(r, generator=gen, device=dev))

    def per_row(value, spread, off):
        """One setting for all rows, or with `mixed` one for each: `spread` about the value, off at times."""
        if not c["mixed"]:
            return torch.full((r,), value, device=dev)
        y = value * (1 + spread * (2 * torch.rand(r, generator=gen, device=dev) - 1))
        return torch.where(torch.rand(r, generator=gen, device=dev) < 0.2, torch.full_like(y, off), y)

    s["temperature"] = per_row(c["temperature"], 0.5, 1.0)
    s["top_k"] = per_row(float(c["top_k"]), 0.9, 0.0).to(torch.int32) if c["top_k"] else None
    s["top_p"] = per_row(c["top_p"], 0.05, 1.0) if c["top_p"] < 1 else None
    s["min_p"] = per_row(c["min_p"], 0.9, 0.0) if c["min_p"] > 0 else None
    return s


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if c["kind"] == "sample":
        return _prepare_sample(c, gen)
    hd, hkv, dt = c["hd"], c["hkv"], _dtype(c)
    lens, rows = _lens(c), _rows(c)
    need = [(n + r + PAGE - 1) // PAGE for n, r in zip(lens, rows)]
    more = [(min(n, c["keep"]) + PAGE - 1) // PAGE if c["kind"] == "evict" else 0 for n in lens]
    total, width = sum(need), max(need) + 1
    num_pages = total + sum(more) + 5
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)

    def table(counts, before, w):
        first = np.cumsum([before] + counts[:-1])
        at = torch.as_tensor(first, device=dev).unsqueeze(1) + torch.arange(w, device=dev)
        some = torch.arange(w, device=dev) < torch.as_tensor(counts, device=dev).unsqueeze(1)
        return torch.where(some, perm[at.clamp(max=num_pages - 1)], torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()

    pool = torch.zeros(num_pages, hkv, PAGE * 2 * hd + 64, dtype=torch.uint8, device=dev)
    s = dict(case=c, pool=pool, table=table(need, 0, width), start=torch.tensor(lens, dtype=torch.int32, device=dev), dtype=dt,
             parent=_parents(c), rows=rows, lens=lens)
    cum = np.concatenate([[0], np.cumsum(rows)])
    s["total"] = int(cum[-1])
    s["row_off"] = torch.as_tensor(cum, dtype=torch.int32, device=dev) if c.get("ragged") else None
    for p0 in range(0, num_pages, 512):             # the cache's contents, 512 pages at a time
        n = min(512, num_pages - p0)
        k, v = (_values((n * PAGE, hkv, hd), gen, torch.float16).view(n, PAGE // SUB, SUB, hkv, hd).permute(0, 3, 1, 2, 4).reshape(-1, SUB, hd) for _ in range(2))
        pool[p0:p0 + n] = _pack(k, v).view(n, hkv, -1)
    lead = (s["total"],) if c.get("ragged") else (c["b"], c.get("w", 0))
    if c["kind"] == "attention":
        s["q"] = _values(lead + (c["hq"], hd), gen, dt)
        s["weight"] = torch.rand(c["b"], hkv, width * PAGE, generator=gen, device=dev) if c["weight"] else None
        return s
    if c["kind"] == "write":
        s["k"], s["v"] = (_values(lead + (hkv, hd), gen, dt) for _ in range(2))
        back = [(n - n // SUB * SUB) + r for n, r in zip(lens, rows)]   # read from the sub-block's first token on
        s["back_start"] = s["start"] // SUB * SUB
    else:
        # weight falls off as a power of rank, most of it at the start and the end
        s["weight"] = torch.rand(c["b"], hkv, c["len_max"], generator=gen, device=dev).pow(8)
        s["dst"] = table(more, total, max(more))
        back = [min(n, c["keep"]) for n in lens]
        s["back_start"] = torch.zeros_like(s["start"])
    s["back"], s["back_total"] = back, sum(back)
    s["back_off"] = torch.as_tensor(np.concatenate([[0], np.cumsum(back)]), dtype=torch.int32, device=dev)
    return s


# -------------------------------------------------------------------------- the operators
def run(state):
    s, c = state, state["case"]
    if own:
        from speculative_decoding_verify_step_gb300 import spec
        if c["kind"] == "sample":
            tok, q = spec.spec_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                      return_probs=c["probs"])
            return (tok, q) if c["probs"] else tok
        if c["kind"] == "attention":
            out = spec.spec_kv8_attention(s["q"], s["pool"], s["start"], s["table"], row_off=s["row_off"], max_width=c["w"],
                                          parent=s["parent"], max_kv_len=c["len_max"], weight=s["weight"])
            return (out, s["weight"]) if c["weight"] else out
        if c["kind"] == "write":
            spec.spec_kv8_write(s["k"], s["v"], s["start"], s["table"], s["pool"], row_off=s["row_off"])
            return spec.spec_kv8_read(s["pool"], s["back_start"], s["table"], s["back_total"], row_off=s["back_off"], dtype=s["dtype"])
        new_len, kept, weight = spec.spec_kv8_evict(s["pool"], s["weight"], s["start"], s["table"], s["dst"], keep=c["keep"], recent=c["recent"])
        return (new_len, kept, weight) + spec.spec_kv8_read(s["pool"], s["back_start"], s["dst"], s["back_total"], row_off=s["back_off"], dtype=s["dtype"])
    return {"sample": _plain_sample, "attention": _plain_attention, "write": _plain_write, "evict": _plain_evict}[c["kind"]](s)


def _expand(sub, hd):
    """Sub-blocks [..., 32 * hd + 16] -> k, v [..., 16, hd] fp32 and their exponents [..., 1, 1]."""
    out, exps = [], []
    for i, at in enumerate(_places(hd, sub.device)):
        e = sub[..., 32 * hd + i].contiguous().view(torch.int8).to(torch.int32)[..., None, None]
        out.append(torch.ldexp(sub[..., at].view(torch.float8_e4m3fn).float().unflatten(-1, (SUB, hd)), e))
        exps.append(e)
    return out, exps


def _cached(s):
    """k, v [B, hkv, keys, hd] fp32 of every sequence's pages, and exponents [B, hkv, keys / 16]."""
    hd = s["case"]["hd"]
    pages = s["pool"][s["table"].clamp(min=0).long()].unflatten(-1, (PAGE // SUB, 32 * hd + 16))
    kv, exps = _expand(pages, hd)                                   # [B, pages, hkv, 4, 16, hd]
    kv = [x.transpose(1, 2).flatten(2, 4) for x in kv]
    return kv, [e.transpose(1, 2).flatten(2) for e in exps]


def _row_places(total, off, start, ragged, w):
    """Sequence and token position of every flat row."""
    flat = torch.arange(total, device=start.device)
    if ragged:
        o = off.long()
        seq = torch.searchsorted(o[1:].contiguous(), flat, right=True)
        row = flat - o[seq]
    else:
        seq, row = flat // w, flat % w
    return seq, start.long()[seq] + row


def _rounded(x, dtype):
    return (x.clamp(-65504.0, 65504.0) if dtype == torch.float16 else x).to(dtype)


def _plain_attention(s):
    c, dev = s["case"], s["pool"].device
    b, w, hkv, hd, grp = c["b"], c["w"], c["hkv"], c["hd"], c["hq"] // c["hkv"]
    seq, pos = _row_places(s["total"], s["row_off"], s["start"], c["ragged"], w)
    row = pos - s["start"].long()[seq]
    q = torch.zeros(b, w, c["hq"], hd, device=dev)
    q[seq, row] = s["q"].reshape(-1, c["hq"], hd).float()
    (k, v), _ = _cached(s)
    n = k.shape[2]
    q = q.view(b, w, hkv, grp, hd).permute(0, 2, 1, 3, 4).reshape(b, hkv, w * grp, hd)
    score = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(hd)
    key = torch.arange(n, device=dev) - s["start"].long().unsqueeze(1)      # window row of each key, or below 0
    anc = torch.zeros(w, w, dtype=torch.bool, device=dev)
    par = s["parent"] or list(range(-1, w - 1))
    anc[0, 0] = True
    for j in range(1, w):
        anc[j] = anc[par[j]]
        anc[j, j] = True
    see = (key < 0).unsqueeze(1) | (anc[:, key.clamp(0, w - 1)].transpose(0, 1) & ((key >= 0) & (key < w)).unsqueeze(1))
    see = see.unsqueeze(1).repeat_interleave(grp, 2)             # [B, 1, w * grp, keys]
    score = torch.where(see, score, torch.full((), -math.inf, device=dev))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    v = torch.where((key < w).view(b, 1, n, 1), v, torch.zeros((), device=dev))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total
    o = _rounded(o.view(b, hkv, w, grp, hd).permute(0, 2, 1, 3, 4).reshape(b, w, c["hq"], hd), s["dtype"])
    o = o[seq, row] if c["ragged"] else o
    if not c["weight"]:
        return o
    real = torch.zeros(b, w, device=dev)
    real[seq, row] = 1.0
    s["weight"] += (p / total * real.view(b, 1, w, 1).repeat_interleave(grp, 2)).sum(2)
    return o, s["weight"]


def _plain_write(s):
    c = s["case"]
    hkv, hd = c["hkv"], c["hd"]
    seq, pos = _row_places(s["back_total"], s["back_off"], s["back_start"], True, 0)
    nseq, npos = _row_places(s["total"], s["row_off"], s["start"], c["ragged"], c["w"])
    at = (s["back_off"].long()[nseq] + npos - s["back_start"].long()[nseq])          # output row of each written row
    old = pos < s["start"].long()[seq]
    first = torch.cat([torch.ones(1, dtype=torch.bool, device=pos.device), (seq[1:] != seq[:-1]) | (pos[1:] % SUB == 0)])
    blk = torch.cumsum(first.long(), 0) - 1                                          # sub-block of each output row
    nblk = s["back_total"] // SUB + c["b"] + 1
    lo = s["back_start"].long()
    page = s["table"].clamp(min=0).long().gather(1, (lo // PAGE).unsqueeze(1)).squeeze(1)
    subs = s["pool"].unflatten(-1, (PAGE // SUB, 32 * hd + 16))[page, :, lo % PAGE // SUB]
    (held, exps), out = _expand(subs, hd), []                                        # each sequence's first sub-block
    for x, h, e in zip((s["k"], s["v"]), held, exps):
        new = torch.zeros(len(pos), hkv, hd, device=pos.device)
        new[at] = _clamped(x.reshape(-1, hkv, hd))
        mine = h[seq, :, pos % SUB]                                                  # [rows, hkv, hd]
        most = torch.zeros(nblk, hkv, device=pos.device)
        most = most.scatter_reduce(0, blk.unsqueeze(1).expand(-1, hkv), new.abs().amax(-1), "amax")
        exp = _exponent(most)
        was = torch.where(old.unsqueeze(1), e.view(-1, hkv)[seq], torch.full((), -15, dtype=e.dtype, device=pos.device))
        exp = exp.scatter_reduce(0, blk.unsqueeze(1).expand(-1, hkv), was, "amax")[blk].unsqueeze(-1)
        y = torch.where(old.view(-1, 1, 1), mine, new)
        out.append(_rounded(torch.ldexp(_codes(y, exp).float(), exp), s["dtype"]))
    return tuple(out)


def _keep_order(weight, n, keep, recent):
    """Positions that stay of each (sequence, kv head), in order, -1 behind the last; weight [B, hkv, T], n [B]."""
    b, hkv, t = weight.shape
    pos = torch.arange(t, device=weight.device)
    n = n.long().view(b, 1, 1)
    key = torch.where(torch.isnan(weight), torch.full((), -math.inf, device=weight.device), weight)
    key = torch.where(pos >= n - recent, torch.full((), math.inf, device=weight.device), key)
    rank = torch.argsort(torch.where(pos < n, -key.double(), torch.full((), math.inf, dtype=torch.float64, device=weight.device)), dim=-1, stable=True)
    # tokens behind the end come last: a stable sort puts them behind a weight of -inf too
    first = rank[..., :min(keep, t)]
    first = torch.where(torch.arange(first.shape[-1], device=weight.device) < n, first, torch.full_like(first, t)).sort(-1).values
    kept = torch.full((b, hkv, keep), -1, dtype=torch.int32, device=weight.device)
    kept[..., :first.shape[-1]] = torch.where(first < t, first, torch.full_like(first, -1)).to(torch.int32)
    return kept


def _plain_evict(s):
    c = s["case"]
    hkv, hd, keep = c["hkv"], c["hd"], c["keep"]
    w = s["weight"]
    kept = _keep_order(w, s["start"], keep, c["recent"])
    some = kept >= 0
    new_len = torch.minimum(s["start"], torch.full_like(s["start"], keep))
    weight = torch.zeros_like(w)
    got = torch.where(some, torch.gather(w, 2, kept.clamp(min=0).long()), torch.zeros((), device=w.device))
    n = min(keep, w.shape[-1])
    weight[..., :n] = got[..., :n]
    out = []
    pad = -keep % SUB
    for x in _cached(s)[0]:
        y = torch.gather(x, 2, kept.clamp(min=0).long().unsqueeze(-1).expand(-1, -1, -1, hd))
        y = torch.where(some.unsqueeze(-1), _clamped(y), torch.zeros((), device=w.device))
        y = torch.nn.functional.pad(y, (0, 0, 0, pad)).unflatten(2, (-1, SUB))       # [B, hkv, blocks, 16, hd]
        e = _exponent(y.abs().amax((-2, -1), keepdim=True))
        y = _rounded(torch.ldexp(_codes(y, e).float(), e), s["dtype"]).flatten(2, 3).transpose(1, 2)
        seq, pos = _row_places(s["back_total"], s["back_off"], s["back_start"], True, 0)
        out.append(y[seq, pos])
    return (new_len, kept, weight) + tuple(out)


def _plain_sample(s):
    # 64 bits: a token's place in the running sum lies next to its neighbours' by as little as 2^-40
    l = s["logits"].double()
    rows, v = l.shape
    x = (l - l.amax(1, keepdim=True)) / s["temperature"].double().unsqueeze(1)
    mass = torch.floor(torch.exp(x) * 2.0 ** 40).long()
    order = torch.argsort(l, dim=1, descending=True, stable=True)
    ranked = mass.gather(1, order)
    run_sum = torch.cumsum(ranked, 1)
    k = torch.full((rows,), v, dtype=torch.int64, device=l.device)
    if s["top_k"] is not None:
        k = torch.where((s["top_k"] >= 1) & (s["top_k"] < v), s["top_k"].long(), k)
    n = k
    if s["top_p"] is not None:
        top = run_sum.gather(1, (k - 1).unsqueeze(1)).double()
        tau = torch.ceil(s["top_p"].double().unsqueeze(1) * top).long().clamp(min=1)
        n = torch.minimum(n, torch.where(s["top_p"] < 1, (run_sum < tau).sum(1) + 1, n))
    if s["min_p"] is not None:
        n = torch.minimum(n, (ranked.double() >= s["min_p"].double().unsqueeze(1) * 2.0 ** 40).sum(1))
    keep = torch.zeros(rows, v, dtype=torch.bool, device=l.device)
    keep.scatter_(1, order, torch.arange(v, device=l.device) < n.unsqueeze(1))
    z = run_sum.gather(1, (n - 1).unsqueeze(1))
    m = torch.floor(s["u"].double() * 2.0 ** 24).long().unsqueeze(1)
    t = m * (z >> 24) + ((m * (z & 0xffffff)) >> 24)
    tok = (torch.cumsum(torch.where(keep, mass, torch.zeros_like(mass)), 1) <= t).sum(1).to(torch.int32)
    if not s["case"]["probs"]:
        return tok
    return tok, torch.where(keep, mass.double() / z.double(), torch.zeros((), dtype=torch.float64, device=l.device)).float()


# ------------------------------------------------------------- the definition, in 64 bits
def _exact_subs(raw, hd):
    """Sub-blocks raw [n, 32 * hd + 16] -> k, v [n, 16, hd] fp64, from the layout's picture and e4m3's fields."""
    n = raw.shape[0]

    def value(code, e):
        code = code.to(torch.int64)
        ex, m = code >> 3 & 15, (code & 7).double()
        y = torch.where(ex > 0, (8 + m) * torch.exp2((ex - 10).double()), m * 2.0 ** -9)
        return torch.where(code >= 128, -y, y) * torch.exp2(e.double()).view(n, 1, 1)

    kb = raw[:, :16 * hd].reshape(n, 8, 2, hd)                       # token pairs
    if hd == 128:
        kb = torch.stack([kb[:, :, 0], torch.cat([kb[:, :, 1, 64:], kb[:, :, 1, :64]], -1)], 2)
    vb = raw[:, 16 * hd:32 * hd].reshape(n, hd // 32, 8, 4, 4, 2, 2)  # chunk, g, c, dim in chunk, half, token in pair
    vb = vb.permute(0, 5, 3, 6, 2, 1, 4)                              # half, c, token | g, chunk, dim
    e = raw[:, 32 * hd:32 * hd + 2].contiguous().view(torch.int8)
    return value(kb.reshape(n, 16, hd), e[:, 0]), value(vb.reshape(n, 16, hd), e[:, 1])


def _exact_cells(s, b, n):
    """K and V of the first n tokens of sequence b: [n, hkv, hd] fp64."""
    c = s["case"]
    hd, hkv = c["hd"], c["hkv"]
    pages = s["table"][b, :(n + PAGE - 1) // PAGE].long()
    out = _exact_subs(s["pool"][pages].reshape(-1, 32 * hd + 16), hd)
    return tuple(x.view(len(pages), hkv, PAGE, hd).permute(0, 2, 1, 3).reshape(-1, hkv, hd)[:n] for x in out)


def _exact_held(y, first=None):
    """What sub-blocks hold of y [tokens, hkv, hd], 16 to one; the exponents [hkv] of the first are at least `first`."""
    n = len(y)
    y = torch.cat([y, y.new_zeros((-n % SUB,) + y.shape[1:])]).unflatten(0, (-1, SUB))
    a = y.abs().amax((1, 3))
    e = torch.full_like(a, -15)
    if first is not None and n:
        e[0] = first.double()
    for k in range(-14, 9):
        e = torch.where((e <= k - 1) & (a > 448 * 2.0 ** (k - 1)), torch.full_like(e, k), e)
    unit = torch.exp2(e).view(-1, 1, y.shape[2], 1)
    scaled = y / unit
    step = torch.exp2(torch.floor(torch.log2(scaled.abs().clamp(min=2.0 ** -6) * (1 + 1e-15))) - 3)
    return (torch.round(scaled / step) * step * unit).flatten(0, 1)[:n]


def _exact_write(s):
    c, at, outs = s["case"], 0, []
    x = [s[n].reshape(-1, c["hkv"], c["hd"]) for n in "kv"]
    for b in range(c["b"]):
        n, r = s["lens"][b], s["rows"][b]
        lo = n // SUB * SUB
        sub = s["pool"][s["table"][b, lo // PAGE].long()].view(c["hkv"], 4, -1)[:, lo % PAGE // SUB]
        old = [y.transpose(0, 1)[:n - lo] for y in _exact_subs(sub, c["hd"])]
        exps = sub[:, 32 * c["hd"]:].contiguous().view(torch.int8)
        new = [torch.nan_to_num(y[at:at + r].double(), nan=-65504.0).clamp(-65504, 65504) for y in x]
        # tokens held already: their exponent counts, whatever their values
        outs.append([_exact_held(torch.cat([o, y]), exps[:, i] if n > lo else None) for i, (o, y) in enumerate(zip(old, new))])
        at += r
    return tuple(torch.cat([o[i] for o in outs]) for i in range(2))


def _exact_attention(s):
    c, outs, at = s["case"], [], 0
    grp = c["hq"] // c["hkv"]
    weight = s["weight"].double() if c["weight"] else None
    for b in range(c["b"]):
        n, r = s["lens"][b], s["rows"][b]
        k, v = _exact_cells(s, b, n + r)
        q = s["q"].reshape(-1, c["hq"], c["hd"])[at:at + r].double()
        at += r
        see = np.zeros((r, n + r), bool)
        see[:, :n] = True
        for j in range(r):
            i = j
            while i >= 0:
                see[j, n + i] = True
                i = s["parent"][i] if s["parent"] else i - 1
        see = torch.as_tensor(see, device=k.device).unsqueeze(1)
        o = torch.empty(r, c["hq"], c["hd"], dtype=torch.float64, device=k.device)
        for h in range(c["hkv"]):
            sc = (q[:, h * grp:(h + 1) * grp] @ k[:, h].T) * c["hd"] ** -0.5
            p = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
            o[:, h * grp:(h + 1) * grp] = p @ v[:, h]
            if weight is not None:
                weight[b, h, :n + r] += p.sum((0, 1))
        outs.append(o)
    o = torch.cat(outs)
    o = o if c["ragged"] else o.view(c["b"], c["w"], c["hq"], c["hd"])
    return (o, weight) if c["weight"] else o


def _exact_evict(s):
    c = s["case"]
    w = torch.zeros(s["weight"].shape, dtype=torch.float64, device=s["pool"].device)
    outs = []
    for b in range(c["b"]):
        n = s["lens"][b]
        m = min(n, c["keep"])
        kv = _exact_cells(s, b, n)
        heads = []
        for h in range(c["hkv"]):
            wt = s["weight"][b, h, :n].double()
            r = min(c["recent"], m)
            old = torch.sort(wt[:n - r], descending=True, stable=True).indices[:m - r]
            stay = torch.cat([torch.sort(old).values, torch.arange(n - r, n, device=w.device)])
            w[b, h, :m] = wt[stay]
            heads.append([x[stay, h:h + 1] for x in kv])
        for i in range(2):
            heads[0][i] = _exact_held(torch.cat([y[i] for y in heads], 1))
        outs.append(heads[0])
    return (None, None, w) + tuple(torch.cat([o[i] for o in outs]) for i in range(2))


def _exact_sample(s):
    if not s["case"]["probs"]:
        return None
    out = []
    for r in range(s["case"]["rows"]):
        l = s["logits"][r].double()
        p = torch.softmax(l / s["temperature"][r].double(), 0)
        srt, idx = torch.sort(l, descending=True, stable=True)
        ps = p[idx]
        n = len(l)
        if s["top_k"] is not None and 1 <= int(s["top_k"][r]) < n:
            n = int(s["top_k"][r])
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            c = torch.cumsum(ps[:n], 0)
            n = min(n, int((c < s["top_p"][r].double() * c[-1]).sum()) + 1)
        if s["min_p"] is not None:
            n = min(n, int((ps >= s["min_p"][r].double() * ps[0]).sum()))
        q = torch.zeros_like(p)
        q[idx[:n]] = ps[:n] / ps[:n].sum()
        out.append(q)
    return None, torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "attention": _exact_attention, "write": _exact_write, "evict": _exact_evict}[case["kind"]](s)
