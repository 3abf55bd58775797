"""Thin Python binding of the verify-round C ABI (include/spec_verify.h).

Argument marshalling only: every step of the round runs in the CUDA library.
Tensors are torch CUDA tensors (device memory and streams come from PyTorch);
the current torch stream is passed to every call.  Loading fails loudly when
the library has not been built -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Iterable, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_OK = 0
STATUS_NAMES = {0: "SPEC_OK", 1: "SPEC_ERR_INVALID_ARG", 2: "SPEC_ERR_UNSUPPORTED_DEVICE", 3: "SPEC_ERR_OOM",
                4: "SPEC_ERR_CAPACITY", 5: "SPEC_ERR_CUDA", 6: "SPEC_ERR_TIMEOUT", 7: "SPEC_ERR_UNSUPPORTED"}

WEIGHT_KIND = {"embed": 0, "lm_head": 1, "final_norm": 2, "attn_norm": 3, "wq": 4, "wk": 5, "wv": 6, "wo": 7,
               "ffn_norm": 8, "w_gate": 9, "w_up": 10, "w_down": 11}


class SpecError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class spec_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn_dim", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("page_size", ctypes.c_int32), ("max_batch", ctypes.c_int32), ("max_width", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


EXPORTS = ["spec_model_create", "spec_model_destroy", "spec_model_set_weight", "spec_seq_reset", "spec_prefill",
           "spec_decode_step", "spec_verify_step", "spec_verify_tree_step", "spec_score", "spec_accept_probs",
           "spec_accept_greedy", "spec_get_kv_state", "spec_read_kv", "spec_debug_logits", "spec_debug_wait_probe",
           "spec_kv_fill_random", "spec_sync_status", "spec_max_pages_per_seq", "spec_last_launch_count", "spec_last_error",
           "spec_set_profiling", "spec_read_profile", "spec_accept_greedy_noalloc", "spec_verify_ragged",
           "spec_adjust_probs", "spec_verify_tree_sampled", "spec_accept_tree_probs", "spec_kv_write",
           "spec_kv4_block_bytes", "spec_kv4_write", "spec_kv4_read", "spec_kv4_attention", "spec_kv4_attention_workspace",
           "spec_model_create_kv"]

RAGGED_CAP_ACCEPT, RAGGED_COMPACT = 1, 2

PROFILE_CLASSES = ["qkv", "o", "gate_up", "down", "lm_head", "attention"]

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it is missing: build it with __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build the CUDA library first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P, I32, I64, F32, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64
    sig = {
        "spec_model_create": (I32, [ctypes.POINTER(spec_config), ctypes.POINTER(P)]),
        "spec_model_create_kv": (I32, [ctypes.POINTER(spec_config), I32, ctypes.POINTER(P)]),
        "spec_model_destroy": (None, [P]),
        "spec_model_set_weight": (I32, [P, I32, I32, P, I64, P]),
        "spec_seq_reset": (I32, [P, I32, P, P]),
        "spec_prefill": (I32, [P, I32, P, P, I32, P, P]),
        "spec_decode_step": (I32, [P, I32, P, P, F32, P, P, P, P, P]),
        "spec_verify_step": (I32, [P, I32, I32, P, P, P, P, F32, P, P, P, P, P, P]),
        "spec_verify_tree_step": (I32, [P, I32, I32, P, P, P, P, P, P, P]),
        "spec_verify_ragged": (I32, [P, I32, I32, P, P, P, I32, I32, P, P, F32, P, P, P, P, P, P]),
        "spec_adjust_probs": (I32, [I32, I32, P, P, P, P, I32, P]),
        "spec_verify_tree_sampled": (I32, [P, I32, I32, P, P, P, P, P, F32, P, P, P, P, P, P]),
        "spec_accept_tree_probs": (I32, [I32, I32, I32, P, P, P, P, P, P, P, P, P]),
        "spec_score": (I32, [P, I32, I32, P, P, P, P, P]),
        "spec_accept_probs": (I32, [I32, I32, I32, P, P, P, P, P, P, P, P]),
        "spec_accept_greedy": (I32, [I32, I32, I32, P, P, P, P, P, P]),
        "spec_get_kv_state": (I32, [P, I32, P, P, P]),
        "spec_read_kv": (I32, [P, I32, I32, I32, I32, P, P]),
        "spec_debug_logits": (I32, [P, P, I64, P]),
        "spec_debug_wait_probe": (I32, [P, I64, P]),
        "spec_kv_fill_random": (I32, [P, I32, P, P, U64, F32, P]),
        "spec_kv_write": (I32, [P, I32, I32, P, P, P]),
        "spec_sync_status": (I32, [P, P]),
        "spec_max_pages_per_seq": (I32, [P]),
        "spec_last_launch_count": (I32, [P]),
        "spec_last_error": (ctypes.c_char_p, []),
        "spec_set_profiling": (I32, [P, I32]),
        "spec_accept_greedy_noalloc": (I32, [I32, I32, I32, P, P, P, P, P, P]),
        "spec_read_profile": (I32, [P, P, P, P]),
        "spec_kv4_block_bytes": (I64, [I32]),
        "spec_kv4_write": (I32, [I32, I32, I32, P, P, P, I32, I32, I32, I32, I32, P, P, I64, I64, P, P]),
        "spec_kv4_read": (I32, [I32, I32, I32, P, P, P, I32, I32, I32, I32, I32, P, P, P, P]),
        "spec_kv4_attention": (I32, [I32, I32, I32, P, P, P, I32, I32, I32, I32, I32, I32, P, I64, P, F32, I32, P, P,
                                     P, I64, P]),
        "spec_kv4_attention_workspace": (I64, [I32, I32, I32, I32, I32, I32, I32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != SPEC_OK:
        raise SpecError(status, _lib.spec_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    assert t.is_contiguous(), "tensors must be contiguous"
    return ctypes.c_void_p(t.data_ptr())


def _i32_host(xs: Sequence[int]):
    arr = (ctypes.c_int32 * len(xs))(*[int(x) for x in xs])
    return arr


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev_i32(t, device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        t = torch.as_tensor(t)
    return t.to(device=device, dtype=torch.int32).contiguous()


def _f32(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """q and u are fp32 on the C side: convert (no copy when already fp32 and contiguous)."""
    return None if t is None else t.to(dtype=torch.float32).contiguous()


def _opt_dev(t, device, dtype):
    """None stays None (setting off); a list, array or tensor becomes a device tensor."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        t = torch.as_tensor(t)
    return t.to(device=device, dtype=dtype).contiguous()


KV_FORMATS = {"fp16": 0, "int4": 1}


class SpecModel:
    """Owns one spec_model handle.  Method names follow the C ABI without the prefix.
    kv_format "int4" holds the KV cache in 4 bits (a scale and an offset per token and kv
    head): 3.6 to 3.8 times the cached tokens in the same memory."""

    def __init__(self, dims, *, max_batch: int, max_width: int, max_seq_len: int, num_pages: int,
                 kv_format: str = "fp16"):
        if kv_format not in KV_FORMATS:
            raise ValueError(f"kv_format must be one of {sorted(KV_FORMATS)}")
        lib = load_library()
        self.dims = dims
        cfg = spec_config(dims.n_layers, dims.d_model, dims.n_heads, dims.n_kv_heads, dims.head_dim, dims.ffn_dim,
                          dims.vocab, dims.rms_eps, dims.rope_theta, 64, max_batch, max_width, max_seq_len, num_pages)
        self.cfg = cfg
        h = ctypes.c_void_p()
        _check(lib.spec_model_create_kv(ctypes.byref(cfg), KV_FORMATS[kv_format], ctypes.byref(h)))
        self.handle = h
        self.kv_format = kv_format
        self.device = torch.device("cuda", torch.cuda.current_device())
        self.max_pages = lib.spec_max_pages_per_seq(h)

    def close(self):
        if getattr(self, "handle", None):
            _lib.spec_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- weights
    def set_weight(self, name: str, tensor: torch.Tensor):
        """name: synth-style ('embed', 'layers.3.wq', ...).  bf16 matrices / fp32 gains."""
        parts = name.split(".")
        layer, kind = (int(parts[1]), parts[2]) if parts[0] == "layers" else (0, parts[0])
        want = torch.float32 if kind.endswith("norm") else torch.bfloat16
        t = tensor.to(want).contiguous()
        _check(_lib.spec_model_set_weight(self.handle, WEIGHT_KIND[kind], layer, _ptr(t), t.numel(), _stream()))
        torch.cuda.current_stream().synchronize()  # `t` may be a temporary

    def load_weights(self, items: Iterable[Tuple[str, torch.Tensor]]):
        for name, t in items:
            self.set_weight(name, t)

    # -------------------------------------------------------------- sequences
    def seq_reset(self, seq_ids: Sequence[int]):
        ids = _i32_host(seq_ids)
        _check(_lib.spec_seq_reset(self.handle, len(seq_ids), ids, _stream()))

    def prefill(self, seq_ids, tokens: torch.Tensor, lens: Sequence[int]):
        sid = _dev_i32(seq_ids, self.device)
        tok = _dev_i32(tokens, self.device)
        _check(_lib.spec_prefill(self.handle, sid.numel(), _ptr(sid), _ptr(tok), tok.shape[1], _i32_host(lens),
                                 _stream()))
        torch.cuda.current_stream().synchronize()

    def decode_step(self, seq_ids, tok, temperature: float = 0.0, u=None, out=None, top_k=None, top_p=None):
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        B = sid.numel()
        out = torch.empty(B, dtype=torch.int32, device=self.device) if out is None else out
        kk, pp = _opt_dev(top_k, self.device, torch.int32), _opt_dev(top_p, self.device, torch.float32)
        u = _f32(u)
        _check(_lib.spec_decode_step(self.handle, B, _ptr(sid), _ptr(tk), float(temperature), _ptr(kk), _ptr(pp),
                                     _ptr(u), _ptr(out), _stream()))
        return out

    def verify_step(self, seq_ids, tok, q=None, u=None, temperature: float = 0.0, outs=None, top_k=None,
                    top_p=None):
        """tok [B, gamma+1] (pending + drafts).  Returns (accepted [B], committed [B, W], bonus [B]).
        top_k / top_p: per-sequence sampling adjustments of sampled rounds (None = off)."""
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        B, W = tk.shape
        if outs is None:
            outs = (torch.empty(B, dtype=torch.int32, device=self.device),
                    torch.empty(B, W, dtype=torch.int32, device=self.device),
                    torch.empty(B, dtype=torch.int32, device=self.device))
        acc, com, bon = outs
        kk, pp = _opt_dev(top_k, self.device, torch.int32), _opt_dev(top_p, self.device, torch.float32)
        q, u = _f32(q), _f32(u)
        _check(_lib.spec_verify_step(self.handle, B, W - 1, _ptr(sid), _ptr(tk), _ptr(q), _ptr(u),
                                     float(temperature), _ptr(kk), _ptr(pp), _ptr(acc), _ptr(com), _ptr(bon),
                                     _stream()))
        return acc, com, bon

    def verify_ragged(self, seq_ids, tok, verify_lens, mode: int, q=None, u=None, temperature: float = 0.0,
                      gamma: Optional[int] = None, outs=None, top_k=None, top_p=None):
        """mode RAGGED_CAP_ACCEPT: tok [B, gamma+1]; RAGGED_COMPACT: tok packed [sum(verify_lens)].
        verify_lens: per-sequence rows (list or tensor).  Returns (accepted, committed [B, gamma+1], bonus)."""
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        lens = _dev_i32(verify_lens, self.device)
        B = sid.numel()
        if gamma is None:
            gamma = tk.shape[1] - 1 if mode == RAGGED_CAP_ACCEPT else int(lens.max().item()) - 1
        total = int(tk.numel()) if mode == RAGGED_COMPACT else B * (gamma + 1)
        if outs is None:
            outs = (torch.empty(B, dtype=torch.int32, device=self.device),
                    torch.empty(B, gamma + 1, dtype=torch.int32, device=self.device),
                    torch.empty(B, dtype=torch.int32, device=self.device))
        acc, com, bon = outs
        kk, pp = _opt_dev(top_k, self.device, torch.int32), _opt_dev(top_p, self.device, torch.float32)
        q, u = _f32(q), _f32(u)
        _check(_lib.spec_verify_ragged(self.handle, B, gamma, _ptr(sid), _ptr(tk), _ptr(lens), total, mode, _ptr(q),
                                       _ptr(u), float(temperature), _ptr(kk), _ptr(pp), _ptr(acc), _ptr(com),
                                       _ptr(bon), _stream()))
        return acc, com, bon

    def verify_tree_step(self, seq_ids, tok, parent: Sequence[int], outs=None):
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        B, N = tk.shape
        if outs is None:
            outs = (torch.empty(B, dtype=torch.int32, device=self.device),
                    torch.empty(B, N, dtype=torch.int32, device=self.device),
                    torch.empty(B, dtype=torch.int32, device=self.device))
        acc, com, bon = outs
        _check(_lib.spec_verify_tree_step(self.handle, B, N, _ptr(sid), _ptr(tk), _i32_host(parent), _ptr(acc),
                                          _ptr(com), _ptr(bon), _stream()))
        return acc, com, bon

    def verify_tree_sampled(self, seq_ids, tok, parent: Sequence[int], u, q=None, temperature: float = 1.0,
                            outs=None, top_k=None, top_p=None):
        """Sampled tree round: u [B, N]; q [B, N, V] (children of node v drawn from q[:, v])
        or None (deterministic candidates).  Returns (accepted, committed [B, N], bonus)."""
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        B, N = tk.shape
        if outs is None:
            outs = (torch.empty(B, dtype=torch.int32, device=self.device),
                    torch.empty(B, N, dtype=torch.int32, device=self.device),
                    torch.empty(B, dtype=torch.int32, device=self.device))
        acc, com, bon = outs
        kk, pp = _opt_dev(top_k, self.device, torch.int32), _opt_dev(top_p, self.device, torch.float32)
        q, u = _f32(q), _f32(u)
        _check(_lib.spec_verify_tree_sampled(self.handle, B, N, _ptr(sid), _ptr(tk), _i32_host(parent), _ptr(q),
                                             _ptr(u), float(temperature), _ptr(kk), _ptr(pp), _ptr(acc), _ptr(com),
                                             _ptr(bon), _stream()))
        return acc, com, bon

    def score(self, seq_ids, tok, parent: Optional[Sequence[int]] = None, logits_out=None):
        sid = _dev_i32(seq_ids, self.device)
        tk = _dev_i32(tok, self.device)
        B, W = tk.shape
        if logits_out is None:
            logits_out = torch.empty(B, W, self.dims.vocab, dtype=torch.float32, device=self.device)
        _check(_lib.spec_score(self.handle, B, W, _ptr(sid), _ptr(tk), _i32_host(parent) if parent is not None
                               else None, _ptr(logits_out), _stream()))
        return logits_out

    def kv_write(self, seq_id: int, k: torch.Tensor, v: torch.Tensor):
        """Give sequence seq_id the cached K/V k, v: [n_layers, n_tokens, n_kv_heads,
        head_dim] (converted to fp16; quantised, if kv_format is "int4"); its length becomes
        n_tokens."""
        want = (self.dims.n_layers, k.shape[1], self.dims.n_kv_heads, self.dims.head_dim)
        if tuple(k.shape) != want or tuple(v.shape) != want:
            raise ValueError(f"k, v must be {want}")
        kk = k.to(device=self.device, dtype=torch.float16).contiguous()
        vv = v.to(device=self.device, dtype=torch.float16).contiguous()
        _check(_lib.spec_kv_write(self.handle, int(seq_id), int(k.shape[1]), _ptr(kk), _ptr(vv), _stream()))

    def kv_fill_random(self, seq_ids: Sequence[int], lens: Sequence[int], seed: int = 0, scale: float = 0.5):
        _check(_lib.spec_kv_fill_random(self.handle, len(seq_ids), _i32_host(seq_ids), _i32_host(lens), seed,
                                        scale, _stream()))

    # ------------------------------------------------------------------ state
    def kv_state(self, seq_ids: Sequence[int]):
        n = len(seq_ids)
        lens = (ctypes.c_int32 * n)()
        pt = (ctypes.c_int32 * (n * self.max_pages))()
        _check(_lib.spec_get_kv_state(self.handle, n, _i32_host(seq_ids), lens, pt))
        return list(lens), [list(pt[i * self.max_pages:(i + 1) * self.max_pages]) for i in range(n)]

    def read_kv(self, layer: int, seq_id: int, t0: int, n: int):
        Hkv, hd = self.dims.n_kv_heads, self.dims.head_dim
        k = torch.empty((n, Hkv, hd), dtype=torch.int16)
        v = torch.empty((n, Hkv, hd), dtype=torch.int16)
        _check(_lib.spec_read_kv(self.handle, layer, seq_id, t0, n, ctypes.c_void_p(k.data_ptr()),
                                 ctypes.c_void_p(v.data_ptr())))
        return k.view(torch.float16), v.view(torch.float16)

    def debug_wait_probe(self, budget_cycles: int) -> None:
        """Enqueue one bounded device wait that nothing completes; the next
        sync_status() raises SpecError with SPEC_ERR_TIMEOUT (6)."""
        _check(_lib.spec_debug_wait_probe(self.handle, int(budget_cycles), _stream()))

    def debug_logits(self, rows: int) -> torch.Tensor:
        """Logits of the last forward ([rows, vocab] fp32, device)."""
        out = torch.empty(rows, self.dims.vocab, dtype=torch.float32, device=self.device)
        _check(_lib.spec_debug_logits(self.handle, _ptr(out), out.numel(), _stream()))
        return out

    def sync_status(self):
        _check(_lib.spec_sync_status(self.handle, _stream()))

    def set_profiling(self, enable: bool):
        _check(_lib.spec_set_profiling(self.handle, 1 if enable else 0))

    def read_profile(self):
        """{class: (ms, launches, bytes)} accumulated since the last read."""
        ms = (ctypes.c_double * 6)()
        n = (ctypes.c_int64 * 6)()
        by = (ctypes.c_double * 6)()
        _check(_lib.spec_read_profile(self.handle, ms, n, by))
        return {c: (ms[i], n[i], by[i]) for i, c in enumerate(PROFILE_CLASSES)}

    def last_launch_count(self) -> int:
        return _lib.spec_last_launch_count(self.handle)


# --------------------------------------------------------- standalone acceptance
def spec_accept_probs(p: torch.Tensor, q: Optional[torch.Tensor], x: Optional[torch.Tensor], u: torch.Tensor):
    """p [B, W, V], q [B, W-1, V], x [B, W-1], u [B, W] (CUDA).  Returns (accepted, committed, bonus)."""
    lib = load_library()
    B, W, V = p.shape
    dev = p.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    com = torch.empty(B, W, dtype=torch.int32, device=dev)
    bon = torch.empty(B, dtype=torch.int32, device=dev)
    xx = None if x is None else _dev_i32(x, dev)
    pp = p.float().contiguous()
    qq = None if q is None else q.float().contiguous()
    uu = u.float().contiguous()
    _check(lib.spec_accept_probs(B, W - 1, V, _ptr(pp), _ptr(qq), _ptr(xx), _ptr(uu), _ptr(acc), _ptr(com),
                                 _ptr(bon), _stream()))
    torch.cuda.current_stream().synchronize()
    return acc, com, bon


def spec_adjust_probs(p: torch.Tensor, top_k=None, top_p=None, rows_per_setting: int = 1, out=None):
    """Top-k / top-p adjustment of probability rows p [..., V] (CUDA fp32); setting
    i covers rows i*rows_per_setting .. (i+1)*rows_per_setting - 1 of the flattened
    rows.  `out` may be p itself."""
    lib = load_library()
    V = p.shape[-1]
    pp = p.float().contiguous()
    rows = pp.numel() // V
    out = torch.empty_like(pp) if out is None else out
    kk, tp = _opt_dev(top_k, p.device, torch.int32), _opt_dev(top_p, p.device, torch.float32)
    _check(lib.spec_adjust_probs(rows, V, _ptr(pp), _ptr(out), _ptr(kk), _ptr(tp), rows_per_setting, _stream()))
    torch.cuda.current_stream().synchronize()
    return out


def spec_accept_tree_probs(p: torch.Tensor, q: Optional[torch.Tensor], tok, parent: Sequence[int], u: torch.Tensor):
    """p [B, N, V], q [B, N, V] or None, tok [B, N], u [B, N] (CUDA).  Returns (accepted, committed, bonus)."""
    lib = load_library()
    B, N, V = p.shape
    dev = p.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    com = torch.empty(B, N, dtype=torch.int32, device=dev)
    bon = torch.empty(B, dtype=torch.int32, device=dev)
    tk = _dev_i32(tok, dev)
    pp = p.float().contiguous()
    qq = None if q is None else q.float().contiguous()
    uu = u.float().contiguous()
    _check(lib.spec_accept_tree_probs(B, N, V, _ptr(pp), _ptr(qq), _ptr(tk), _i32_host(parent), _ptr(uu), _ptr(acc),
                                      _ptr(com), _ptr(bon), _stream()))
    torch.cuda.current_stream().synchronize()
    return acc, com, bon


def spec_accept_greedy_noalloc(logits: torch.Tensor, x: Optional[torch.Tensor], outs=None):
    """Greedy acceptance through the entry point that allocates nothing in the
    library (its scratch is a fixed device array, 4096 rows at most).  `outs`
    lets the caller pass preallocated (accepted, committed, bonus) tensors."""
    lib = load_library()
    B, W, V = logits.shape
    dev = logits.device
    if outs is None:
        outs = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, W, dtype=torch.int32, device=dev),
                torch.empty(B, dtype=torch.int32, device=dev))
    acc, com, bon = outs
    for t, shape, what in ((acc, (B,), "accepted"), (com, (B, W), "committed"), (bon, (B,), "bonus")):
        if t.dtype != torch.int32 or t.device != dev or tuple(t.shape) != shape:
            raise ValueError(f"{what} must be an int32 tensor of shape {shape} on {dev}")
    xx = None if x is None else _dev_i32(x, dev)
    lg = logits.float().contiguous()
    _check(lib.spec_accept_greedy_noalloc(B, W - 1, V, _ptr(lg), _ptr(xx), _ptr(acc), _ptr(com), _ptr(bon),
                                          _stream()))
    torch.cuda.current_stream().synchronize()
    return acc, com, bon


def spec_accept_greedy(logits: torch.Tensor, x: Optional[torch.Tensor]):
    lib = load_library()
    B, W, V = logits.shape
    dev = logits.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    com = torch.empty(B, W, dtype=torch.int32, device=dev)
    bon = torch.empty(B, dtype=torch.int32, device=dev)
    xx = None if x is None else _dev_i32(x, dev)
    lg = logits.float().contiguous()
    _check(lib.spec_accept_greedy(B, W - 1, V, _ptr(lg), _ptr(xx), _ptr(acc), _ptr(com), _ptr(bon), _stream()))
    torch.cuda.current_stream().synchronize()
    return acc, com, bon


# ------------------------------------------------------------- 4-bit paged KV cache
_KV4_DTYPE = {torch.float16: 0, torch.bfloat16: 1}


def spec_kv4_pool(num_pages: int, n_kv_heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """An empty 4-bit KV pool: uint8 [num_pages, n_kv_heads, 64 * head_dim + 512], pages of
    64 tokens."""
    block = load_library().spec_kv4_block_bytes(int(head_dim))
    if block == 0:
        raise ValueError("head_dim must be 64 or 128")
    return torch.zeros(num_pages, n_kv_heads, block, dtype=torch.uint8, device=device)


_KV4_HEAD_DIM = {4608: 64, 8704: 128}  # by the bytes of a (page, kv head) block
_KV4_WORKSPACE = {}  # bytes by device index and the arguments of spec_kv4_attention_workspace


def _kv4_geometry(pool: torch.Tensor, start: torch.Tensor, page_table: torch.Tensor, row_off):
    """Checked (num_pages, n_kv_heads, head_dim, B, max_pages) of a call's pool and tables."""
    ps, ts, i32 = pool.shape, page_table.shape, torch.int32
    hd = _KV4_HEAD_DIM.get(ps[-1]) if len(ps) == 3 else None
    if hd is None or pool.dtype is not torch.uint8 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 [num_pages, n_kv_heads, 64 * head_dim + 512] tensor "
                         "(spec_kv4_pool)")
    B = start.numel()
    if start.dtype is not i32 or start.dim() != 1 or not start.is_contiguous():
        raise ValueError("start / kv_len must be a contiguous int32 tensor of shape (B,)")
    if page_table.dtype is not i32 or len(ts) != 2 or ts[0] != B or not page_table.is_contiguous():
        raise ValueError(f"page_table must be a contiguous int32 tensor of shape ({B}, max_pages)")
    dev = pool.device
    same = start.device == dev and page_table.device == dev
    if row_off is not None:
        if row_off.dtype is not i32 or row_off.dim() != 1 or row_off.numel() != B + 1 or not row_off.is_contiguous():
            raise ValueError(f"row_off must be a contiguous int32 tensor of shape ({B + 1},)")
        same = same and row_off.device == dev
    if not same or not pool.is_cuda:
        raise ValueError("pool, start / kv_len, page_table and row_off must be on one CUDA device")
    return ps[0], ps[1], hd, B, ts[1]


def _kv4_rows(x: torch.Tensor, what: str, B: int, heads, hd: int, ragged: bool, dev):
    """(total_rows, rows_per_seq, row stride) of x: [B, n, heads, hd], or [rows, heads, hd] with row_off.
    The heads of a row are contiguous; rows may be strided, evenly over all of x."""
    if x.device != dev or x.dtype not in _KV4_DTYPE:
        raise ValueError(f"{what} must be fp16 or bf16 on {dev}")
    xs = x.shape
    lead = 1 if ragged else 2
    if len(xs) != lead + 2 or xs[-1] != hd or (heads is not None and xs[-2] != heads) or (not ragged and xs[0] != B):
        want = "[rows, heads, head_dim]" if ragged else "[B, n, heads, head_dim]"
        raise ValueError(f"{what} must be {want} with head_dim {hd}" + (f" and {heads} heads" if heads else "")
                         + ("" if ragged else f" and B {B}"))
    total, n = (xs[0], 0) if ragged else (xs[0] * xs[1], xs[1])
    if x.is_contiguous():
        return total, n, xs[-2] * hd
    st = x.stride()
    row = st[lead - 1] if xs[lead - 1] > 1 else (st[0] if lead == 2 and xs[0] > 1 else xs[-2] * hd)
    if total and (st[-1] != 1 or (st[-2] != hd and xs[-2] > 1) or (
            lead == 2 and xs[0] > 1 and xs[1] > 1 and st[0] != xs[1] * row)):
        raise ValueError(f"{what}: each row must be contiguous and the rows evenly spaced")
    return total, n, row


def _kv4_call(dev, fn, *args):
    """Call `fn` with the current stream of `dev` (made current for the call where it is not)."""
    i = dev.index
    if i == torch._C._cuda_getDevice():
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(i)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(i)))


def spec_kv4_write(k: torch.Tensor, v: torch.Tensor, start: torch.Tensor, page_table: torch.Tensor,
                   pool: torch.Tensor, row_off: Optional[torch.Tensor] = None) -> None:
    """Quantise K/V rows into the 4-bit cache: k, v [B, n, n_kv_heads, head_dim] at positions
    start[b] .. start[b] + n - 1 of page_table[b], or packed [rows, n_kv_heads, head_dim]
    with sequence b's rows row_off[b] .. row_off[b + 1] - 1.  fp16 or bf16."""
    lib = _lib or load_library()
    P, H, hd, B, width = _kv4_geometry(pool, start, page_table, row_off)
    dev, ragged = pool.device, row_off is not None
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and type")
    total, n, ks = _kv4_rows(k, "k", B, H, hd, ragged, dev)
    _, _, vs = _kv4_rows(v, "v", B, H, hd, ragged, dev)
    _kv4_call(dev, lib.spec_kv4_write, B, n, total, row_off.data_ptr() if ragged else None, start.data_ptr(),
              page_table.data_ptr(), width, P, H, hd, _KV4_DTYPE[k.dtype], k.data_ptr(), v.data_ptr(),
              ks, vs, pool.data_ptr())


def spec_kv4_read(pool: torch.Tensor, start: torch.Tensor, page_table: torch.Tensor, n: int,
                  row_off: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.float16, outs=None):
    """K and V of n tokens per sequence from position start[b] on, as fp16 or bf16
    [B, n, n_kv_heads, head_dim]; with row_off, n rows in all, [n, n_kv_heads, head_dim].
    Rows of no sequence are left unwritten.  `outs`: preallocated (k, v)."""
    lib = _lib or load_library()
    P, H, hd, B, width = _kv4_geometry(pool, start, page_table, row_off)
    dev, ragged = pool.device, row_off is not None
    n = int(n)
    if dtype not in _KV4_DTYPE:
        raise ValueError("dtype must be torch.float16 or torch.bfloat16")
    if n < 0:
        raise ValueError("n must not be negative")
    shape = (n, H, hd) if ragged else (B, n, H, hd)
    if outs is None:
        outs = (torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev))
    k, v = outs
    for t in (k, v):
        if t.dtype != dtype or t.device != dev or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"outs must be contiguous {dtype} tensors of shape {shape} on {dev}")
    _kv4_call(dev, lib.spec_kv4_read, B, 0 if ragged else n, n if ragged else B * n,
              row_off.data_ptr() if ragged else None, start.data_ptr(), page_table.data_ptr(), width, P,
              H, hd, _KV4_DTYPE[dtype], pool.data_ptr(), k.data_ptr(), v.data_ptr())
    return k, v


def spec_kv4_attention(q: torch.Tensor, pool: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor,
                       row_off: Optional[torch.Tensor] = None, max_width: Optional[int] = None,
                       parent: Optional[Sequence[int]] = None, scale: Optional[float] = None, max_kv_len: int = 0,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of verify windows over the 4-bit cache.  q [B, W, n_heads, head_dim], or packed
    [rows, n_heads, head_dim] with row_off and at most max_width rows per sequence (default:
    as many as a window may have).  Row j of sequence b sees positions < kv_len[b] and its
    ancestors in the window, whose K/V sit at kv_len[b] + 0, 1, ... (parent: tree, default the
    chain).  scale: default head_dim ** -0.5.  max_kv_len: an upper bound of kv_len if known
    (launch shape only).  Returns q's shape and type; rows of no window are left unwritten."""
    lib = _lib or load_library()
    P, H, hd, B, width = _kv4_geometry(pool, kv_len, page_table, row_off)
    dev, ragged = pool.device, row_off is not None
    total, W, qs = _kv4_rows(q, "q", B, None, hd, ragged, dev)
    Hq = q.shape[-2]
    if ragged:
        W = max_width if max_width is not None else max(1, min(16, 64 // max(1, Hq // H)))
        if not 1 <= W <= 16:
            raise ValueError(f"max_width {W} outside 1..16")
    elif max_width is not None and max_width < W:
        raise ValueError(f"q has {W} rows per sequence, more than max_width {max_width}")
    par = None
    if parent is not None:
        if len(parent) < W:
            raise ValueError(f"parent must have {W} entries")
        par = _i32_host(parent)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.dtype != q.dtype or out.device != dev or out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} tensor of shape {tuple(q.shape)} on {dev}")
    key = (dev.index, B, W, Hq, H, hd, width, max_kv_len)
    size = _KV4_WORKSPACE.get(key)
    if size is None:
        if len(_KV4_WORKSPACE) > 4096:
            _KV4_WORKSPACE.clear()
        with torch.cuda.device(dev):
            size = _KV4_WORKSPACE[key] = lib.spec_kv4_attention_workspace(*key[1:])
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    _kv4_call(dev, lib.spec_kv4_attention, B, W, total, row_off.data_ptr() if ragged else None, kv_len.data_ptr(),
              page_table.data_ptr(), width, P, Hq, H, hd, _KV4_DTYPE[q.dtype], q.data_ptr(), qs, par,
              hd ** -0.5 if scale is None else scale, max_kv_len, pool.data_ptr(), out.data_ptr(),
              None if ws is None else ws.data_ptr(), size)
    return out
