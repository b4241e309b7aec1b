"""GB300 (sm_103a) hot path of context-lookup speculative decoding.

A thin ctypes binding over ``libclk.so`` (C ABI in ``include/clk.h``).  Every
step of the path runs in the library's CUDA kernels; this module only checks
tensors and passes their device pointers and the current CUDA stream.  There
is no fallback: if the library is missing, importing the binding's functions
raises.

Per decode step (HyperQwen context-lookup article, "lookup 草稿的原理：三步走"):

    lookup_propose    Step 1: longest 4..12 suffix match, most recent, LZ77 copy
    sched_step        Step 3: long-block scheduler (enter after 2, sticky 3)
    fuse              Step 2: head / tail fusion rule
    verify_greedy     greedy verification: argmax rows + accepted prefix
    lookup_append     commit the emitted tokens (incremental index update)

plus the fused launches ``propose_fuse_sched`` and ``verify_append`` that the
``Step`` driver uses (two kernels per step).

Beside the step, the target's side of it: a paged K/V cache (``Cache`` and the
``cache_*`` calls), trees of drafted tokens (``tree_masks``, ``tree_accept``)
and the attention that reads both (``tree_attend``, ``prompt_attend``).  The
cache may be one of 8-bit values with scales (``ScaledPool``), and queries and
keys may be rotated by their positions on the way (``Rotary``,
``tree_rotate``, ``cache_append_rotary``).
"""
from __future__ import annotations

import ctypes
import os
from functools import lru_cache
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libclk.so")

OK, EINVAL, ECAPACITY, ECUDA, ENOTIMPL, ESTATE = 0, -1, -2, -3, -4, -5
BF16, F32, F16, E4M3 = 0, 1, 2, 3
SENT = -1
BLOCK = 16
MAX_BATCH = 8192
TREE_MAX = 64

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class ClkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "min_k", "max_k", "head", "tail", "head_replace_k", "head_agree_k", "head_agree_n", "tail_k",
        "enter_streak", "sticky", "near_full_slack")]

    @classmethod
    def default(cls, **kw) -> "Params":
        p = cls()
        lib().clk_params_default(ctypes.byref(p))
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    @property
    def long_len(self) -> int:
        return 1 + self.head + self.tail

    @property
    def short_len(self) -> int:
        return 1 + self.head


class Counters(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("steps", "hits", "long_steps", "drafted", "accepted", "emitted")] + \
               [("accept_hist", (ctypes.c_int64 * 16) * 2)]

    def as_dict(self):
        d = {n: getattr(self, n) for n in ("steps", "hits", "long_steps", "drafted", "accepted", "emitted")}
        d["accept_hist"] = [[self.accept_hist[i][j] for j in range(16)] for i in range(2)]
        return d


class SlotInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "mode", "streak", "miss", "has_prev", "cur_len", "n_indexed")]


class PoolDesc(ctypes.Structure):
    """clk_pool"""
    _fields_ = [("d_base", _P), ("dtype", _I32), ("planes", _I32), ("heads", _I32), ("dim", _I32),
                ("plane_stride", _I64), ("page_stride", _I64), ("head_stride", _I64), ("tok_stride", _I64)]


class AttnDesc(ctypes.Structure):
    """clk_attn"""
    _fields_ = [(n, _I32) for n in ("dtype", "q_heads", "kv_heads", "dim")] + [("scale", ctypes.c_float)] + \
               [(n, _P) for n in ("d_q", "d_k", "d_v", "d_out")] + \
               [(n, _I64) for n in ("q_req", "q_row", "q_head", "k_req", "k_row", "k_head", "v_req", "v_row", "v_head")]


class ScalesDesc(ctypes.Structure):
    """clk_scales"""
    _fields_ = [("d_base", _P), ("tokens", _I32), ("plane_stride", _I64), ("page_stride", _I64), ("head_stride", _I64),
                ("block_stride", _I64)]


class RotaryDesc(ctypes.Structure):
    """clk_rotary"""
    _fields_ = [("d_table", _P), ("positions", _I64), ("pairs", _I32), ("neighbours", _I32)]


class TurnDesc(ctypes.Structure):
    """clk_turn"""
    _fields_ = [(n, _I32) for n in ("dtype", "q_heads", "kv_heads", "dim")] + \
               [(n, _P) for n in ("d_q", "d_k", "d_q_out", "d_k_out")] + \
               [(n, _I64) for n in ("q_req", "q_row", "q_head", "k_req", "k_row", "k_head", "qo_req", "qo_row", "qo_head",
                                    "ko_req", "ko_row", "ko_head")]


# (name, restype, argtypes) of every exported entry point
_SIGS = [
    ("clk_params_default", None, [_P]),
    ("clk_params_check", ctypes.c_int, [_P]),
    ("clk_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("clk_lookup_workspace_bytes", ctypes.c_int, [_P, _I32, _I64, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_lookup_create", ctypes.c_int, [ctypes.POINTER(_P), _P, _I32, _I64, _I32, _P, ctypes.c_size_t]),
    ("clk_lookup_reset", ctypes.c_int, [_P, _P]),
    ("clk_lookup_set_alone", ctypes.c_int, [_P, _I32]),
    ("clk_lookup_init", ctypes.c_int, [_P, _P, _I32, _P, _P, _P]),
    ("clk_lookup_append", ctypes.c_int, [_P, _P, _I32, _P, _P, _P]),
    ("clk_lookup_propose", ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P]),
    ("clk_lookup_propose_scan", ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P, _P]),
    ("clk_sched_step", ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P]),
    ("clk_fuse", ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    ("clk_fuse_sched", ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("clk_propose_fuse_sched", ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("clk_verify_scratch_bytes", ctypes.c_int, [_I32, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_verify_scratch_init", ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    ("clk_verify_greedy", ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                         ctypes.c_size_t, _P]),
    ("clk_verify_greedy_static", ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    ("clk_verify_append", ctypes.c_int, [_P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                         _P]),
    ("clk_verify_sample_scratch_bytes", ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_verify_sample", ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                         ctypes.c_size_t, _P]),
    ("clk_verify_sample_exact_scratch_bytes", ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_verify_sample_exact", ctypes.c_int, [_P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                               ctypes.c_size_t, _P]),
    ("clk_verify_sample_append", ctypes.c_int, [_P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                                _P, _P, _P, ctypes.c_size_t, _P]),
    ("clk_verify_sample_exact_append", ctypes.c_int, [_P, _P, _P, _I32, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P,
                                                      _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("clk_status", ctypes.c_int, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32), _P]),
    ("clk_status_clear", ctypes.c_int, [_P, _P]),
    ("clk_read_counters", ctypes.c_int, [_P, _I32, _P, _P]),
    ("clk_read_slot_info", ctypes.c_int, [_P, _I32, _P, _P]),
    ("clk_lookup_read_history", ctypes.c_int, [_P, _I32, _P, _I64, ctypes.POINTER(_I64), _P]),
    ("clk_lookup_restore_state", ctypes.c_int, [_P, _I32, _P, _P, _P]),
    ("clk_lookup_destroy", None, [_P]),
    ("clk_cache_workspace_bytes", ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_cache_create", ctypes.c_int, [ctypes.POINTER(_P), _I32, _I32, _I32, _I32, _P, ctypes.c_size_t]),
    ("clk_cache_reset", ctypes.c_int, [_P, _P]),
    ("clk_cache_buffers", ctypes.c_int, [_P, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    ("clk_cache_grow", ctypes.c_int, [_P, _P, _I32, _P, _P]),
    ("clk_cache_append", ctypes.c_int, [_P, _P, _I32, _P, _I32, _I32, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P]),
    ("clk_cache_fork", ctypes.c_int, [_P, _P, _P, _I32, _P, _P]),
    ("clk_cache_free", ctypes.c_int, [_P, _P, _I32, _P]),
    ("clk_cache_compact", ctypes.c_int, [_P, _P, _P, _P]),
    ("clk_cache_status", ctypes.c_int, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32), _P]),
    ("clk_cache_status_clear", ctypes.c_int, [_P, _P]),
    ("clk_cache_destroy", None, [_P]),
    ("clk_tree_masks", ctypes.c_int, [_I32, _I32, _P, _P, _P, _P]),
    ("clk_tree_accept", ctypes.c_int, [_I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("clk_attend_scratch_bytes", ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(ctypes.c_size_t)]),
    ("clk_attend_status", ctypes.c_int, [_P, ctypes.POINTER(_I32), _P]),
    ("clk_tree_attend", ctypes.c_int, [_P, _P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("clk_prompt_attend", ctypes.c_int, [_P, _P, _I32, _I64, _P, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    ("clk_cache_fork_scaled", ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P]),
    ("clk_cache_compact_scaled", ctypes.c_int, [_P, _P, _P, _P, _P]),
    ("clk_tree_rotate", ctypes.c_int, [_P, _P, _I32, _P, _I32, _P, _P, _P, _P, _P]),
    ("clk_cache_append_rotary", ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P,
                                               _P, _P, _P]),
    ("clk_tree_attend_scaled", ctypes.c_int, [_P, _P, _I32, _P, _P, _I32, _P, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("clk_prompt_attend_scaled", ctypes.c_int, [_P, _P, _I32, _I64, _P, _P, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
]


@lru_cache(maxsize=None)
def lib() -> ctypes.CDLL:
    """The loaded libclk.so; raises if it has not been built."""
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    for name, res, args in _SIGS:
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


def status_string(code: int) -> str:
    return lib().clk_status_string(code).decode()


def _check(fn: str, rc: int):
    if rc != OK:
        raise ClkError(fn, rc)


def _stream(stream=None) -> int:
    # the raw handle of the current stream, without building a Stream object (0.2 us instead of 2.9 us a call)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t: Optional[torch.Tensor], dtype=torch.int32, shape=None, name="tensor") -> int:
    if t is None:
        return 0
    if t.is_cuda and t.dtype == dtype and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _logits_args(logits: torch.Tensor):
    # a CUDA tensor, or a pinned host tensor that the kernels read in place
    if not (logits.is_cuda or logits.is_pinned()) or logits.dim() != 3:
        raise ValueError("logits must be a CUDA tensor or a pinned host tensor [B, rows, V]")
    if logits.dtype == torch.bfloat16:
        dt = BF16
    elif logits.dtype == torch.float32:
        dt = F32
    else:
        raise ValueError("logits must be bfloat16 or float32")
    if logits.stride(2) != 1:
        raise ValueError("logits rows must be contiguous")
    return dt, logits.stride(1), logits.stride(0), logits.shape[2]


class Lookup:
    """Histories, k-gram index and scheduler state of up to `max_slots` requests.

    Owns its device workspace (a torch uint8 tensor) and the C handle."""

    def __init__(self, max_slots: int, max_hist: int, vocab: int = 0, params: Optional[Params] = None,
                 device="cuda", stream=None):
        self.params = params or Params.default()
        L = lib()
        nbytes = ctypes.c_size_t()
        _check("clk_lookup_workspace_bytes",
               L.clk_lookup_workspace_bytes(ctypes.byref(self.params), max_slots, max_hist, ctypes.byref(nbytes)))
        self.workspace_bytes = nbytes.value
        # 256-byte alignment: torch's caching allocator returns 512-byte aligned blocks.
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
        h = _P()
        _check("clk_lookup_create", L.clk_lookup_create(ctypes.byref(h), ctypes.byref(self.params), max_slots,
                                                        max_hist, vocab, self.workspace.data_ptr(),
                                                        self.workspace_bytes))
        self.handle = h
        self.max_slots, self.max_hist, self.vocab = max_slots, max_hist, vocab
        _check("clk_lookup_reset", L.clk_lookup_reset(self.handle, _stream(stream)))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                lib().clk_lookup_destroy(h)
            except Exception:
                pass
            self.handle = None

    def set_alone(self, alone: bool):
        """clk_lookup_set_alone: True when the fused verify calls are launched
        with nothing to overlap (timing only; results are the same)."""
        _check("clk_lookup_set_alone", lib().clk_lookup_set_alone(self.handle, 1 if alone else 0))

    # -- inspection (synchronising) -------------------------------------
    def status(self, stream=None):
        st, det = _I32(), _I32()
        _check("clk_status", lib().clk_status(self.handle, ctypes.byref(st), ctypes.byref(det), _stream(stream)))
        return st.value, det.value

    def status_clear(self, stream=None):
        _check("clk_status_clear", lib().clk_status_clear(self.handle, _stream(stream)))

    def counters(self, slot: int = -1, stream=None) -> dict:
        c = Counters()
        _check("clk_read_counters", lib().clk_read_counters(self.handle, slot, ctypes.byref(c), _stream(stream)))
        return c.as_dict()

    def slot_info(self, slot: int, stream=None) -> dict:
        s = SlotInfo()
        _check("clk_read_slot_info", lib().clk_read_slot_info(self.handle, slot, ctypes.byref(s), _stream(stream)))
        return {n: getattr(s, n) for n, _ in SlotInfo._fields_}

    def history(self, slot: int, stream=None):
        import numpy as np
        n = _I64()
        _check("clk_lookup_read_history",
               lib().clk_lookup_read_history(self.handle, slot, None, 0, ctypes.byref(n), _stream(stream)))
        out = np.empty(n.value, dtype=np.int32)
        _check("clk_lookup_read_history",
               lib().clk_lookup_read_history(self.handle, slot, out.ctypes.data, n.value, ctypes.byref(n),
                                             _stream(stream)))
        return out

    # -- checkpoint / resume ----------------------------------------------
    def snapshot(self, slot: int, stream=None) -> dict:
        """Everything needed to resume request `slot` elsewhere: its history,
        scheduler state and counters (host copies; synchronising)."""
        return {"history": self.history(slot, stream), "info": self.slot_info(slot, stream),
                "counters": self.counters(slot, stream)}

    def restore(self, slot: int, snap: dict, stream=None):
        """Resume a snapshot in `slot` of this lookup (same parameters): the
        history is ingested again (which rebuilds its index), then the
        scheduler state and counters are written back (synchronising)."""
        import numpy as np
        dev = self.workspace.device
        hist = np.ascontiguousarray(snap["history"], dtype=np.int32)
        s = torch.tensor([slot], dtype=torch.int32, device=dev)
        off = torch.tensor([0, hist.size], dtype=torch.int64, device=dev)
        lookup_init(self, s, torch.from_numpy(hist).to(dev), off, stream=stream)
        info = SlotInfo(**{n: int(snap["info"][n]) for n, _ in SlotInfo._fields_})
        c = Counters(**{n: int(snap["counters"][n]) for n in
                        ("steps", "hits", "long_steps", "drafted", "accepted", "emitted")})
        for i in range(2):
            for j in range(16):
                c.accept_hist[i][j] = int(snap["counters"]["accept_hist"][i][j])
        _check("clk_lookup_restore_state",
               lib().clk_lookup_restore_state(self.handle, slot, ctypes.byref(info), ctypes.byref(c),
                                              _stream(stream)))


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI without the clk_ prefix)
# ---------------------------------------------------------------------------
def lookup_init(h: Lookup, slots, prompt, prompt_off, stream=None):
    B = slots.numel()
    _check("clk_lookup_init", lib().clk_lookup_init(h.handle, _ptr(slots, name="slots"), B,
                                                    _ptr(prompt, name="prompt"),
                                                    _ptr(prompt_off, torch.int64, (B + 1,), "prompt_off"),
                                                    _stream(stream)))


def lookup_append(h: Lookup, slots, tok, count, stream=None):
    B = slots.numel()
    _check("clk_lookup_append", lib().clk_lookup_append(h.handle, _ptr(slots, name="slots"), B,
                                                        _ptr(tok, shape=(B, BLOCK), name="tok"),
                                                        _ptr(count, shape=(B,), name="count"), _stream(stream)))


def lookup_propose(h: Lookup, slots, draft, k, j, stream=None):
    B = slots.numel()
    _check("clk_lookup_propose", lib().clk_lookup_propose(h.handle, _ptr(slots, name="slots"), B,
                                                          _ptr(draft, shape=(B, BLOCK), name="draft"),
                                                          _ptr(k, shape=(B,), name="k"), _ptr(j, shape=(B,), name="j"),
                                                          _stream(stream)))


def lookup_propose_scan(h: Lookup, slots, draft, k, j, stream=None, ctas_per_request: int = 0):
    """The proposal by a full history scan (clk_lookup_propose_scan);
    ctas_per_request=1 is the pages' one-program-per-request form."""
    B = slots.numel()
    _check("clk_lookup_propose_scan",
           lib().clk_lookup_propose_scan(h.handle, _ptr(slots, name="slots"), B, int(ctas_per_request),
                                         _ptr(draft, shape=(B, BLOCK)), _ptr(k, shape=(B,)), _ptr(j, shape=(B,)),
                                         _stream(stream)))


def sched_step(h: Lookup, slots, k, prev_accept, prev_len, length, stream=None):
    B = slots.numel()
    _check("clk_sched_step", lib().clk_sched_step(h.handle, _ptr(slots, name="slots"), B, _ptr(k, shape=(B,)),
                                                  _ptr(prev_accept, shape=(B,)), _ptr(prev_len, shape=(B,)),
                                                  _ptr(length, shape=(B,)), _stream(stream)))


def fuse(params: Params, last_tok, draft, k, head, length, block, stream=None):
    B = last_tok.numel()
    _check("clk_fuse", lib().clk_fuse(ctypes.byref(params), B, _ptr(last_tok, shape=(B,)),
                                      _ptr(draft, shape=(B, BLOCK)), _ptr(k, shape=(B,)),
                                      _ptr(head, shape=(B, params.head)), _ptr(length, shape=(B,)),
                                      _ptr(block, shape=(B, BLOCK)), _stream(stream)))


def fuse_sched(h: Lookup, slots, draft, k, head, prev_accept, prev_len, length, block, stream=None):
    B = slots.numel()
    _check("clk_fuse_sched", lib().clk_fuse_sched(h.handle, _ptr(slots), B, _ptr(draft, shape=(B, BLOCK)),
                                                  _ptr(k, shape=(B,)), _ptr(head, shape=(B, h.params.head)),
                                                  _ptr(prev_accept, shape=(B,)), _ptr(prev_len, shape=(B,)),
                                                  _ptr(length, shape=(B,)), _ptr(block, shape=(B, BLOCK)),
                                                  _stream(stream)))


def propose_fuse_sched(h: Lookup, slots, head, prev_accept, prev_len, draft, k, j, length, block, stream=None):
    B = slots.numel()
    _check("clk_propose_fuse_sched",
           lib().clk_propose_fuse_sched(h.handle, _ptr(slots), B, _ptr(head, shape=(B, h.params.head)),
                                        _ptr(prev_accept, shape=(B,)), _ptr(prev_len, shape=(B,)),
                                        _ptr(draft, shape=(B, BLOCK)), _ptr(k, shape=(B,)), _ptr(j, shape=(B,)),
                                        _ptr(length, shape=(B,)), _ptr(block, shape=(B, BLOCK)), _stream(stream)))


def verify_scratch_bytes(B: int) -> int:
    n = ctypes.c_size_t()
    _check("clk_verify_scratch_bytes", lib().clk_verify_scratch_bytes(B, ctypes.byref(n)))
    return n.value


def verify_scratch(B: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed scratch buffer for verify_greedy with up to B requests."""
    t = torch.empty(verify_scratch_bytes(B), dtype=torch.uint8, device=device)
    _check("clk_verify_scratch_init", lib().clk_verify_scratch_init(t.data_ptr(), t.numel(), _stream(stream)))
    return t


def verify_greedy(logits, block, length, argmax, accept, emitted, out_tok, scratch, stream=None):
    dt, rs, qs, V = _logits_args(logits)
    B = block.shape[0]
    _check("clk_verify_greedy",
           lib().clk_verify_greedy(logits.data_ptr(), dt, rs, qs, V, B, _ptr(block, shape=(B, BLOCK)),
                                   _ptr(length, shape=(B,)), _ptr(argmax, shape=(B, BLOCK)),
                                   _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                   _ptr(out_tok, shape=(B, BLOCK)), _ptr(scratch, torch.uint8, name="scratch"),
                                   scratch.numel(), _stream(stream)))


def verify_greedy_static(logits, block, length, argmax, accept, emitted, out_tok, stream=None):
    """verify_greedy with the library's own fixed scratch (no buffer from the
    caller, nothing allocated); B <= 1024; calls must not overlap on the GPU."""
    dt, rs, qs, V = _logits_args(logits)
    B = block.shape[0]
    _check("clk_verify_greedy_static",
           lib().clk_verify_greedy_static(logits.data_ptr(), dt, rs, qs, V, B, _ptr(block, shape=(B, BLOCK)),
                                          _ptr(length, shape=(B,)), _ptr(argmax, shape=(B, BLOCK)),
                                          _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                          _ptr(out_tok, shape=(B, BLOCK)), _stream(stream)))


def verify_sample_scratch(logits_dtype, V: int, B: int, device="cuda", stream=None, halves: int = 1) -> torch.Tensor:
    """A zeroed scratch buffer for verify_sample with vocabulary V and up to
    B requests (logits_dtype: torch.bfloat16 or torch.float32).  halves=2:
    two halves (each the needed size rounded up to 256 bytes), which
    verify_sample_append alternates so that a call may start while the
    previous one finishes."""
    dt = BF16 if logits_dtype == torch.bfloat16 else F32
    n = ctypes.c_size_t()
    _check("clk_verify_sample_scratch_bytes", lib().clk_verify_sample_scratch_bytes(dt, V, B, ctypes.byref(n)))
    size = n.value if halves == 1 else 2 * ((n.value + 255) // 256 * 256)
    t = torch.empty(size, dtype=torch.uint8, device=device)
    _check("clk_verify_scratch_init", lib().clk_verify_scratch_init(t.data_ptr(), t.numel(), _stream(stream)))
    return t


def verify_sample(logits, block, length, inv_temp, uniform, accept, emitted, out_tok, scratch, stream=None):
    """Sampling verification with point-mass drafts (clk_verify_sample).
    inv_temp: float32 [B]; uniform: float32 [B, 16, 2]."""
    dt, rs, qs, V = _logits_args(logits)
    B = block.shape[0]
    _check("clk_verify_sample",
           lib().clk_verify_sample(logits.data_ptr(), dt, rs, qs, V, B, _ptr(block, shape=(B, BLOCK)),
                                   _ptr(length, shape=(B,)), _ptr(inv_temp, torch.float32, (B,), "inv_temp"),
                                   _ptr(uniform, torch.float32, (B, BLOCK, 2), "uniform"),
                                   _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                   _ptr(out_tok, shape=(B, BLOCK)), _ptr(scratch, torch.uint8, name="scratch"),
                                   scratch.numel(), _stream(stream)))


def verify_sample_exact_scratch(logits_dtype, V: int, B: int, device="cuda", stream=None,
                                halves: int = 1) -> torch.Tensor:
    """A zeroed scratch buffer for verify_sample_exact with vocabulary V and
    up to B requests; halves=2: two halves for the fused calls to alternate
    (as verify_sample_scratch)."""
    dt = BF16 if logits_dtype == torch.bfloat16 else F32
    n = ctypes.c_size_t()
    _check("clk_verify_sample_exact_scratch_bytes",
           lib().clk_verify_sample_exact_scratch_bytes(dt, V, B, ctypes.byref(n)))
    size = n.value if halves == 1 else 2 * ((n.value + 255) // 256 * 256)
    t = torch.empty(size, dtype=torch.uint8, device=device)
    _check("clk_verify_scratch_init", lib().clk_verify_scratch_init(t.data_ptr(), t.numel(), _stream(stream)))
    return t


def verify_sample_exact(logits, block, length, inv_temp, uniform, accept, emitted, out_tok, scratch, stream=None):
    """Sampling verification on the fixed-point weights
    (clk_verify_sample_exact): the rule of verify_sample with every decision
    an integer comparison."""
    dt, rs, qs, V = _logits_args(logits)
    B = block.shape[0]
    _check("clk_verify_sample_exact",
           lib().clk_verify_sample_exact(logits.data_ptr(), dt, rs, qs, V, B, _ptr(block, shape=(B, BLOCK)),
                                         _ptr(length, shape=(B,)), _ptr(inv_temp, torch.float32, (B,), "inv_temp"),
                                         _ptr(uniform, torch.float32, (B, BLOCK, 2), "uniform"),
                                         _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                         _ptr(out_tok, shape=(B, BLOCK)), _ptr(scratch, torch.uint8, name="scratch"),
                                         scratch.numel(), _stream(stream)))


def verify_sample_append(h: Lookup, slots, logits, block, length, inv_temp, uniform, accept, emitted, out_tok,
                         scratch, stream=None, length_hint=None):
    """Sampling verification fused with the token commit (clk_verify_sample_append);
    ``length_hint`` (int32 [B] or None) predicts the block lengths."""
    dt, rs, qs, V = _logits_args(logits)
    B = slots.numel()
    _check("clk_verify_sample_append",
           lib().clk_verify_sample_append(h.handle, _ptr(slots), logits.data_ptr(), dt, rs, qs, V, B,
                                          _ptr(block, shape=(B, BLOCK)), _ptr(length, shape=(B,)),
                                          _ptr(length_hint, shape=(B,), name="length_hint"),
                                          _ptr(inv_temp, torch.float32, (B,), "inv_temp"),
                                          _ptr(uniform, torch.float32, (B, BLOCK, 2), "uniform"),
                                          _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                          _ptr(out_tok, shape=(B, BLOCK)), _ptr(scratch, torch.uint8, name="scratch"),
                                          scratch.numel(), _stream(stream)))


def verify_sample_exact_append(h: Lookup, slots, logits, block, length, inv_temp, uniform, accept, emitted, out_tok,
                               scratch, stream=None, length_hint=None):
    """Exact sampling verification (fixed-point weights) fused with the
    token commit (clk_verify_sample_exact_append)."""
    dt, rs, qs, V = _logits_args(logits)
    B = slots.numel()
    _check("clk_verify_sample_exact_append",
           lib().clk_verify_sample_exact_append(h.handle, _ptr(slots), logits.data_ptr(), dt, rs, qs, V, B,
                                                _ptr(block, shape=(B, BLOCK)), _ptr(length, shape=(B,)),
                                                _ptr(length_hint, shape=(B,), name="length_hint"),
                                                _ptr(inv_temp, torch.float32, (B,), "inv_temp"),
                                                _ptr(uniform, torch.float32, (B, BLOCK, 2), "uniform"),
                                                _ptr(accept, shape=(B,)), _ptr(emitted, shape=(B,)),
                                                _ptr(out_tok, shape=(B, BLOCK)),
                                                _ptr(scratch, torch.uint8, name="scratch"), scratch.numel(),
                                                _stream(stream)))


def verify_append(h: Lookup, slots, logits, block, length, argmax, accept, emitted, out_tok, stream=None,
                  length_hint=None):
    dt, rs, qs, V = _logits_args(logits)
    B = slots.numel()
    _check("clk_verify_append",
           lib().clk_verify_append(h.handle, _ptr(slots), logits.data_ptr(), dt, rs, qs, V, B,
                                   _ptr(block, shape=(B, BLOCK)), _ptr(length, shape=(B,)),
                                   _ptr(length_hint, shape=(B,), name="length_hint"),
                                   _ptr(argmax, shape=(B, BLOCK)), _ptr(accept, shape=(B,)),
                                   _ptr(emitted, shape=(B,)), _ptr(out_tok, shape=(B, BLOCK)), _stream(stream)))


# ---------------------------------------------------------------------------
# The target's paged K/V cache
# ---------------------------------------------------------------------------
_POOL_DTYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.float16: F16}


class Cache:
    """Page tables of up to `max_slots` requests over the pages of a pool.

    The pool is the caller's tensor [2 * layers, >= num_pages, kv_heads,
    page_tokens, dim] (any strides with the rows contiguous), or a ScaledPool
    of 8-bit values, handed to the calls that move rows or read them.  ``length`` [max_slots], ``table``
    [max_slots, max_pages] and ``refs`` [num_pages] are int32 views of the
    workspace, to be read in stream order."""

    def __init__(self, max_slots: int, max_pages: int, num_pages: int, page_tokens: int = 64, device="cuda",
                 stream=None):
        L = lib()
        n = ctypes.c_size_t()
        _check("clk_cache_workspace_bytes", L.clk_cache_workspace_bytes(max_slots, max_pages, num_pages, ctypes.byref(n)))
        self.workspace_bytes = n.value
        self.workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
        h = _P()
        base = self.workspace.data_ptr()
        _check("clk_cache_create", L.clk_cache_create(ctypes.byref(h), max_slots, max_pages, num_pages, page_tokens,
                                                      base, n.value))
        self.handle = h
        self.max_slots, self.max_pages, self.num_pages = max_slots, max_pages, num_pages
        self.page_tokens = page_tokens
        self._at = [_P(), _P(), _P()]
        _check("clk_cache_buffers", L.clk_cache_buffers(h, *(ctypes.byref(p) for p in self._at)))
        self._views = [None, None, None]
        self.reset(stream)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                lib().clk_cache_destroy(h)
            except Exception:
                pass
            self.handle = None

    def _view(self, i: int, *shape):
        if self._views[i] is None:
            size = 1
            for x in shape:
                size *= x
            first = self._at[i].value - self.workspace.data_ptr()
            self._views[i] = self.workspace[first:first + 4 * size].view(torch.int32).view(shape)
        return self._views[i]

    @property
    def length(self) -> torch.Tensor:
        return self._view(0, self.max_slots)

    @property
    def table(self) -> torch.Tensor:
        return self._view(1, self.max_slots, self.max_pages)

    @property
    def refs(self) -> torch.Tensor:
        return self._view(2, self.num_pages)

    def reset(self, stream=None):
        """Every slot empty, every page free."""
        _check("clk_cache_reset", lib().clk_cache_reset(self.handle, _stream(stream)))

    # -- inspection (status synchronises) ---------------------------------
    def status(self, stream=None):
        st, det = _I32(), _I32()
        _check("clk_cache_status", lib().clk_cache_status(self.handle, ctypes.byref(st), ctypes.byref(det),
                                                          _stream(stream)))
        return st.value, det.value

    def status_clear(self, stream=None):
        _check("clk_cache_status_clear", lib().clk_cache_status_clear(self.handle, _stream(stream)))


class ScaledPool:
    """A pool of 8-bit values and their scales (clk_scales).

    ``data``: torch.float8_e4m3fn [2 * layers, >= num_pages, kv_heads,
    page_tokens, dim] (any strides with the rows contiguous); ``scale``:
    float32 [2 * layers, >= num_pages, kv_heads, page_tokens / T] (any
    strides), one for each block of T = 16, 32, 64 or 128 tokens.  An element
    stands for its value times its block's scale."""

    def __init__(self, data: torch.Tensor, scale: torch.Tensor):
        if data.dtype != torch.float8_e4m3fn or data.dim() != 5 or scale.dtype != torch.float32 or scale.dim() != 4:
            raise ValueError("data must be float8_e4m3fn [planes, pages, heads, page_tokens, dim], "
                             "scale float32 [planes, pages, heads, blocks]")
        tokens, blocks = data.shape[3], scale.shape[3]
        if not (data.is_cuda and scale.is_cuda) or data.device != scale.device:
            raise ValueError("data and scale must be CUDA tensors of one device")
        if data.shape[0] != scale.shape[0] or data.shape[2] != scale.shape[2] or scale.shape[1] < data.shape[1] \
                or blocks < 1 or tokens % blocks != 0 or tokens // blocks not in (16, 32, 64, 128):
            raise ValueError(f"scale must hold the blocks of 16, 32, 64 or 128 tokens of data's planes, pages and heads, "
                             f"got {tuple(scale.shape)} for {tuple(data.shape)}")
        if data.shape[4] > 1 and data.stride(4) != 1:
            raise ValueError("rows of data must be contiguous")
        self._data, self._scale = data, scale
        p, g, hd, b = scale.stride()
        self._desc = ScalesDesc(scale.data_ptr(), tokens // blocks, p, g, hd, b)

    # (not to be replaced: the calls have their addresses)
    data = property(lambda self: self._data)
    scale = property(lambda self: self._scale)

    @staticmethod
    def empty(layers: int, pages: int, kv_heads: int, page_tokens: int, dim: int, block: int = 16, device="cuda") -> "ScaledPool":
        """A pool of zeros with scales of 1."""
        shape = (2 * layers, pages, kv_heads)
        return ScaledPool(torch.zeros(shape + (page_tokens, dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                          torch.ones(shape + (page_tokens // block,), dtype=torch.float32, device=device))


def _pool8_desc(h: Cache, pool: ScaledPool) -> PoolDesc:
    data = pool._data
    planes, pages, heads, tokens, dim = data.shape
    if pages < h.num_pages or tokens != h.page_tokens:
        raise ValueError(f"pool must have >= {h.num_pages} pages and {h.page_tokens} tokens a page, got {tuple(data.shape)}")
    plane_st, page_st, head_st, tok_st, _ = data.stride()
    return PoolDesc(data.data_ptr(), E4M3, planes, heads, dim, plane_st, page_st, head_st, tok_st)


def _pool_desc(h: Cache, pool: torch.Tensor) -> PoolDesc:
    if not isinstance(pool, torch.Tensor):
        raise ValueError("pool must be a tensor here")
    if not pool.is_cuda or pool.dim() != 5:
        raise ValueError("pool must be a CUDA tensor [planes, pages, heads, page_tokens, dim]")
    planes, pages, heads, tokens, dim = pool.shape
    plane_st, page_st, head_st, tok_st, one = pool.stride()
    code = _POOL_DTYPES.get(pool.dtype)
    if code is None or (one != 1 and dim > 1) or pages < h.num_pages or tokens != h.page_tokens:
        raise ValueError(f"pool must be bfloat16, float16 or float32 with contiguous rows, >= {h.num_pages} pages and "
                         f"{h.page_tokens} tokens a page, got {pool.dtype} {tuple(pool.shape)}")
    return PoolDesc(pool.data_ptr(), code, planes, heads, dim, plane_st, page_st, head_st, tok_st)


def cache_grow(h: Cache, slots, count, stream=None):
    """Room for count[b] more tokens in each slot (clk_cache_grow)."""
    B = slots.numel()
    _check("clk_cache_grow", lib().clk_cache_grow(h.handle, _ptr(slots, name="slots"), B,
                                                  _ptr(count, shape=(B,), name="count"), _stream(stream)))


def _append_rows(B: int, d: PoolDesc, k, v, offsets):
    """Checks the rows of an append; their layers, N and strides (layer, row, head)."""
    if k.dim() != (4 if offsets is not None else 5) or k.shape != v.shape or not (k.is_cuda and v.is_cuda) \
            or (k.stride() != v.stride() and any(n > 1 and a != b for n, a, b in zip(k.shape, k.stride(), v.stride()))):
        raise ValueError("k and v must be CUDA tensors of one shape and layout, "
                         "[layers, B, N, heads, dim] or, with offsets, [layers, T, heads, dim]")
    if offsets is None:
        layers, Bk, N, heads, dim = k.shape
        layer_st, req, row, head, one = k.stride()
        if N == 1:  # the stride from request to request is that from row to row
            row = req if B > 1 else 0
        if Bk != B or (B > 1 and req != N * row):
            raise ValueError("k and v must hold B requests of N rows, one request's rows after another's")
    else:
        layers, N, heads, dim = k.shape
        layer_st, row, head, one = k.stride()
    if k.dtype != v.dtype or _POOL_DTYPES.get(k.dtype) is None or (d.dtype != E4M3 and _POOL_DTYPES[k.dtype] != d.dtype) \
            or heads != d.heads or dim != d.dim:
        raise ValueError("k and v must have the pool's type, heads and dim")
    if dim > 1 and one != 1:
        raise ValueError("rows of k and v must be contiguous")
    return layers, N, layer_st if layers > 1 else 0, row, head if heads > 1 else 0


def cache_append(h: Cache, slots, pool, k, v, count, layer: int = 0, path=None, offsets=None, stream=None):
    """K and V rows into the slots' last count[b] positions (clk_cache_append).

    k, v: [layers, B, N, kv_heads, dim], row ``path[b, i]`` (or i) of request
    b; or, with ``offsets`` (int64 [B+1]), [layers, T, kv_heads, dim].  Into a
    ScaledPool: cache_append_rotary without a rotation."""
    if isinstance(pool, ScaledPool):
        return cache_append_rotary(h, slots, pool, k, v, count, layer=layer, path=path, offsets=offsets, stream=stream)
    B = slots.numel()
    d = _pool_desc(h, pool)
    layers, N, layer_st, row, head = _append_rows(B, d, k, v, offsets)
    _check("clk_cache_append",
           lib().clk_cache_append(h.handle, _ptr(slots, name="slots"), B, ctypes.byref(d), layer, layers,
                                  k.data_ptr(), v.data_ptr(), layer_st, row, head, N,
                                  _ptr(offsets, torch.int64, (B + 1,), "offsets"),
                                  _ptr(path, shape=(B, N), name="path"), _ptr(count, shape=(B,), name="count"),
                                  _stream(stream)))


def cache_fork(h: Cache, src, dst, pool, stream=None):
    """Slots dst[b] (empty) become copies of src[b] (clk_cache_fork)."""
    B = src.numel()
    if isinstance(pool, ScaledPool):
        d = _pool8_desc(h, pool)
        _check("clk_cache_fork_scaled",
               lib().clk_cache_fork_scaled(h.handle, _ptr(src, name="src"), _ptr(dst, shape=(B,), name="dst"), B, ctypes.byref(d),
                                           ctypes.byref(pool._desc), _stream(stream)))
        return
    d = _pool_desc(h, pool)
    _check("clk_cache_fork", lib().clk_cache_fork(h.handle, _ptr(src, name="src"), _ptr(dst, shape=(B,), name="dst"), B,
                                                  ctypes.byref(d), _stream(stream)))


def cache_free(h: Cache, slots, stream=None):
    """Empties the slots (clk_cache_free)."""
    _check("clk_cache_free", lib().clk_cache_free(h.handle, _ptr(slots, name="slots"), slots.numel(), _stream(stream)))


def cache_compact(h: Cache, pool, moved=None, stream=None):
    """Moves the pages in use to the lowest numbers (clk_cache_compact);
    ``moved`` (int32 [1] or None) receives how many moved."""
    if isinstance(pool, ScaledPool):
        d = _pool8_desc(h, pool)
        _check("clk_cache_compact_scaled",
               lib().clk_cache_compact_scaled(h.handle, ctypes.byref(d), ctypes.byref(pool._desc),
                                              _ptr(moved, shape=(1,), name="moved"), _stream(stream)))
        return
    d = _pool_desc(h, pool)
    _check("clk_cache_compact", lib().clk_cache_compact(h.handle, ctypes.byref(d), _ptr(moved, shape=(1,), name="moved"),
                                                        _stream(stream)))


# ---------------------------------------------------------------------------
# Position rotation
# ---------------------------------------------------------------------------
class Rotary:
    """The angles of a position rotation (clk_rotary).

    ``table``: float32 [positions, 2, pairs] on the GPU, the cosines and sines
    of every position's pairs (``Rotary.of`` makes one); ``neighbours``: pairs
    are elements (2i, 2i + 1) instead of (i, i + pairs)."""

    def __init__(self, table: torch.Tensor, neighbours: bool = False):
        if not table.is_cuda or table.dtype != torch.float32 or table.dim() != 3 or table.shape[1] != 2 or not table.is_contiguous() \
                or table.numel() == 0:
            raise ValueError("table must be a contiguous float32 CUDA tensor [positions, 2, pairs]")
        self._table, self._neighbours = table, bool(neighbours)
        self._desc = RotaryDesc(table.data_ptr(), table.shape[0], table.shape[2], int(self.neighbours))

    # (not to be replaced: the calls have the address)
    table = property(lambda self: self._table)
    neighbours = property(lambda self: self._neighbours)

    @staticmethod
    def of(freq, positions: int, factor: float = 1.0, neighbours: bool = False, device="cuda") -> "Rotary":
        """For angles position * freq[i] (radians; computed in 64 bits), cosines and sines times ``factor``."""
        f = torch.as_tensor(freq, dtype=torch.float64, device=device)
        a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
        return Rotary((torch.stack([a.cos(), a.sin()], 1) * factor).float().contiguous(), neighbours)


def _heads(t: torch.Tensor, lead, dtype, dim: int, name: str):
    """Strides (request, row, head) of rows [lead.., heads, dim]."""
    if not t.is_cuda or t.dtype != dtype or t.shape[:-2] != lead or t.shape[-1] != dim or (dim > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor {tuple(lead)} + (heads, {dim}) with contiguous rows")
    st = t.stride()
    return (st[0] if len(lead) == 2 else 0), st[-3], st[-2]


def tree_rotate(h: Cache, slots, q, k, nodes, mask, rotary: Rotary, q_out, k_out, ctx=None, stream=None):
    """Rotates q and k of drafted trees by their nodes' positions (clk_tree_rotate).

    q [B, N, q_heads, dim], k [B, N, kv_heads, dim] (strided) into q_out and
    k_out (their own tensors too); mask int64 [B, N] of tree_masks; ctx (int32
    [B] or None: the slots' lengths)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, N, heads, dim]")
    shape, k_shape, dtype = q.shape, k.shape, q.dtype
    B, N, q_heads, D = shape
    code = _POOL_DTYPES.get(dtype)
    if code is None:
        raise ValueError("q and k must have one type of bfloat16, float16 or float32")
    if q_out.shape != shape or k_out.shape != k_shape:
        raise ValueError("q_out and k_out must have q's and k's shapes")
    lead = shape[:2]
    qs, ks = _heads(q, lead, dtype, D, "q"), _heads(k, lead, dtype, D, "k")
    qo = qs if q_out is q else _heads(q_out, lead, dtype, D, "q_out")
    ko = ks if k_out is k else _heads(k_out, lead, dtype, D, "k_out")
    t = TurnDesc(code, q_heads, k_shape[2], D, q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), *qs, *ks, *qo, *ko)
    _check("clk_tree_rotate",
           lib().clk_tree_rotate(h.handle, _ptr(slots, shape=(B,), name="slots"), B, ctypes.byref(t), N,
                                 _ptr(nodes, shape=(B,), name="nodes"), _ptr(mask, torch.int64, (B, N), "mask"),
                                 _ptr(ctx, shape=(B,), name="ctx"), ctypes.byref(rotary._desc), _stream(stream)))


def _flat_rows(t: torch.Tensor, lead, dtype, dim: int, name: str):
    """Strides (row, head) of rows [.., lead.., heads, dim] whose requests follow one another; one of what comes before."""
    st, shape = t.stride(), t.shape
    if not t.is_cuda or t.dtype != dtype or shape[-2 - len(lead):-2] != lead or shape[-1] != dim or (dim > 1 and st[-1] != 1):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor {tuple(lead)} + (heads, {dim}) with contiguous rows")
    row = st[-3]
    if len(lead) == 2:
        if lead[1] == 1:
            row = st[-4] if lead[0] > 1 else 0
        elif lead[0] > 1 and st[-4] != lead[1] * row:
            raise ValueError(f"{name} must hold one request's rows after another's")
    return row, st[-2]


def cache_append_rotary(h: Cache, slots, pool, k, v, count, rotary: Optional[Rotary] = None, layer: int = 0, path=None, offsets=None,
                        q=None, q_out=None, k_out=None, stream=None):
    """cache_append with the keys rotated by their positions on the way (rotary
    None: as they are), into a pool of their type or a ScaledPool
    (clk_cache_append_rotary).

    With one layer and without path, q [B, N, q_heads, dim] (or [T, q_heads,
    dim]) of the same tokens is rotated into q_out and the rotated keys are
    also written to k_out (k's shape); either may be the source itself."""
    B = slots.numel()
    eight = isinstance(pool, ScaledPool)
    d = _pool8_desc(h, pool) if eight else _pool_desc(h, pool)
    layers, N, layer_st, row, head = _append_rows(B, d, k, v, offsets)
    shape, dtype = k.shape, k.dtype
    code, t = _POOL_DTYPES[dtype], None
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if q is not None or k_out is not None:
        if rotary is None or layers != 1 or path is not None:
            raise ValueError("q and k_out need a rotation, one layer and no path")
        lead, dim = shape[1:-2], shape[-1]
        q_heads = q_at = q_row = q_head = qo_at = qo_row = qo_head = ko_at = ko_row = ko_head = 0
        if q is not None:
            if q_out.shape != q.shape or q.dim() != len(lead) + 2:
                raise ValueError("q must be one layer's rows, and q_out must have q's shape")
            q_heads, q_at, qo_at = q.shape[-2], q.data_ptr(), q_out.data_ptr()
            q_row, q_head = _flat_rows(q, lead, dtype, dim, "q")
            qo_row, qo_head = (q_row, q_head) if q_out is q else _flat_rows(q_out, lead, dtype, dim, "q_out")
        if k_out is not None:
            if k_out.shape != shape:
                raise ValueError("k_out must have k's shape")
            ko_at = k_out.data_ptr()
            ko_row, ko_head = _flat_rows(k_out, lead, dtype, dim, "k_out")
        t = TurnDesc(code, q_heads, shape[-2], dim, q_at, 0, qo_at, ko_at, 0, q_row, q_head, 0, 0, 0, 0, qo_row, qo_head,
                     0, ko_row, ko_head)
    _check("clk_cache_append_rotary",
           lib().clk_cache_append_rotary(h.handle, _ptr(slots, name="slots"), B, ctypes.byref(d),
                                         ctypes.byref(pool._desc) if eight else None, layer, layers, code, k.data_ptr(), v.data_ptr(),
                                         layer_st, row, head, N, _ptr(offsets, torch.int64, (B + 1,), "offsets"),
                                         _ptr(path, shape=(B, N), name="path"), _ptr(count, shape=(B,), name="count"),
                                         ctypes.byref(rotary._desc) if rotary is not None else None,
                                         ctypes.byref(t) if t is not None else None, _stream(stream)))


# ---------------------------------------------------------------------------
# Trees of drafted tokens, and attention
# ---------------------------------------------------------------------------
def tree_masks(parent, nodes, mask, stream=None):
    """Ancestor masks (int64 [B, N]) of trees given by their nodes' parents."""
    B, N = parent.shape
    _check("clk_tree_masks", lib().clk_tree_masks(B, N, _ptr(parent, name="parent"), _ptr(nodes, shape=(B,), name="nodes"),
                                                  _ptr(mask, torch.int64, (B, N), "mask"), _stream(stream)))


def tree_accept(tok, parent, nodes, argmax, accept, path, emitted, out_tok, stream=None):
    """Greedy verification of trees (clk_tree_accept); argmax: the target's
    answers at the nodes, verify_greedy's where N is 16 (or, a tree as N / 16
    of its blocks, a multiple of it)."""
    B, N = tok.shape
    _check("clk_tree_accept",
           lib().clk_tree_accept(B, N, _ptr(tok, name="tok"), _ptr(parent, shape=(B, N), name="parent"),
                                 _ptr(nodes, shape=(B,), name="nodes"), _ptr(argmax, shape=(B, N), name="argmax"),
                                 _ptr(accept, shape=(B,), name="accept"), _ptr(path, shape=(B, N), name="path"),
                                 _ptr(emitted, shape=(B,), name="emitted"), _ptr(out_tok, shape=(B, N), name="out_tok"),
                                 _stream(stream)))


def attend_scratch(q_heads: int, kv_heads: int, dim: int, device="cuda") -> torch.Tensor:
    """A zeroed scratch buffer for tree_attend / prompt_attend with these heads."""
    n = ctypes.c_size_t()
    _check("clk_attend_scratch_bytes", lib().clk_attend_scratch_bytes(q_heads, kv_heads, dim, ctypes.byref(n)))
    return torch.zeros(n.value, dtype=torch.uint8, device=device)


def attend_status(scratch: torch.Tensor, stream=None) -> int:
    """ECUDA where a wait inside an attention on this scratch has run out since it was zeroed, else OK
    (clk_attend_status; synchronises)."""
    st = _I32()
    _check("clk_attend_status", lib().clk_attend_status(_ptr(scratch, torch.uint8, name="scratch"), ctypes.byref(st),
                                                        _stream(stream)))
    return st.value


def _attn_desc(q, k, v, out, scale: float) -> AttnDesc:
    """q [.., q_heads, dim], k and v [.., kv_heads, dim], with 1 or 2 leading axes (prompt, tree)."""
    if q.dim() == 4:
        B, N, Hq, D = q.shape
        lead = (B, N)
        (q0, q1, q2, qd), (k0, k1, k2, kd), (v0, v1, v2, vd) = q.stride(), k.stride(), v.stride()
    else:
        N, Hq, D = q.shape
        lead = (N,)
        q0 = k0 = v0 = 0
        (q1, q2, qd), (k1, k2, kd), (v1, v2, vd) = q.stride(), k.stride(), v.stride()
    Hkv = k.shape[-2]
    if k.shape != lead + (Hkv, D) or v.shape != k.shape or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("q and out (contiguous) must have one shape, k and v another that differs in the heads only")
    if not (q.is_cuda and k.is_cuda and v.is_cuda and out.is_cuda):
        raise ValueError("q, k, v and out must be CUDA tensors")
    dt = q.dtype
    code = _POOL_DTYPES.get(dt)
    if code is None or k.dtype != dt or v.dtype != dt or out.dtype != dt:
        raise ValueError("q, k, v and out must have one type of bfloat16, float16 or float32")
    if D > 1 and not qd == kd == vd == 1:
        raise ValueError("rows of q, k and v must be contiguous")
    return AttnDesc(code, Hq, Hkv, D, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                    q0, q1, q2, k0, k1, k2, v0, v1, v2)


def tree_attend(h: Cache, slots, pool, layer: int, q, k, v, nodes, mask, scale: float, out, scratch, ctx=None,
                stream=None):
    """Attention of drafted trees over the cache (clk_tree_attend).

    q [B, N, q_heads, dim], k and v [B, N, kv_heads, dim] of the new tokens
    (strided), mask int64 [B, N], out [B, N, q_heads, dim]; ctx (int32 [B] or
    None: the slots' lengths) cached rows that are seen.  The pool is of q's
    type or a ScaledPool (clk_tree_attend_scaled)."""
    if not q.dim() == k.dim() == v.dim() == 4:
        raise ValueError("q, k and v must be [B, N, heads, dim]")
    B, N = q.shape[:2]
    a = _attn_desc(q, k, v, out, scale)
    if isinstance(pool, ScaledPool):
        d = _pool8_desc(h, pool)
        _check("clk_tree_attend_scaled",
               lib().clk_tree_attend_scaled(h.handle, _ptr(slots, shape=(B,), name="slots"), B, ctypes.byref(d),
                                            ctypes.byref(pool._desc), layer, ctypes.byref(a), N,
                                            _ptr(nodes, shape=(B,), name="nodes"), _ptr(mask, torch.int64, (B, N), "mask"),
                                            _ptr(ctx, shape=(B,), name="ctx"), _ptr(scratch, torch.uint8, name="scratch"),
                                            scratch.numel(), _stream(stream)))
        return
    d = _pool_desc(h, pool)
    _check("clk_tree_attend",
           lib().clk_tree_attend(h.handle, _ptr(slots, shape=(B,), name="slots"), B, ctypes.byref(d), layer,
                                 ctypes.byref(a), N, _ptr(nodes, shape=(B,), name="nodes"),
                                 _ptr(mask, torch.int64, (B, N), "mask"), _ptr(ctx, shape=(B,), name="ctx"),
                                 _ptr(scratch, torch.uint8, name="scratch"), scratch.numel(), _stream(stream)))


def prompt_attend(q, k, v, offsets, scale: float, out, scratch, cache: Optional[Cache] = None, slots=None, pool=None,
                  layer: int = 0, ctx=None, stream=None):
    """Causal attention of packed prompts (clk_prompt_attend).

    q [T, q_heads, dim], k and v [T, kv_heads, dim] (strided), request b's
    rows offsets[b] .. offsets[b+1] (int64 [B+1]), out [T, q_heads, dim].
    With cache, slots, pool (of q's type, or a ScaledPool) and ctx (int32 [B])
    the rows also see the slots' first ctx cached rows."""
    if not q.dim() == k.dim() == v.dim() == 3:
        raise ValueError("q, k and v must be [T, heads, dim]")
    B = offsets.numel() - 1
    if cache is None and (slots is not None or pool is not None or ctx is not None):
        raise ValueError("slots, pool and ctx need a cache")
    if cache is not None and (slots is None or pool is None):
        raise ValueError("a cache needs slots and a pool")
    a = _attn_desc(q, k, v, out, scale)
    if isinstance(pool, ScaledPool):
        d = _pool8_desc(cache, pool)
        _check("clk_prompt_attend_scaled",
               lib().clk_prompt_attend_scaled(ctypes.byref(a), _ptr(offsets, torch.int64, (B + 1,), "offsets"), B, q.shape[0],
                                              cache.handle, _ptr(slots, shape=(B,), name="slots"), ctypes.byref(d),
                                              ctypes.byref(pool._desc), layer, _ptr(ctx, shape=(B,), name="ctx"),
                                              _ptr(scratch, torch.uint8, name="scratch"), scratch.numel(), _stream(stream)))
        return
    d = _pool_desc(cache, pool) if cache is not None else None
    _check("clk_prompt_attend",
           lib().clk_prompt_attend(ctypes.byref(a), _ptr(offsets, torch.int64, (B + 1,), "offsets"), B, q.shape[0],
                                   cache.handle if cache is not None else None, _ptr(slots, shape=(B,), name="slots"),
                                   ctypes.byref(d) if d is not None else None, layer,
                                   _ptr(ctx, shape=(B,), name="ctx"), _ptr(scratch, torch.uint8, name="scratch"),
                                   scratch.numel(), _stream(stream)))


# ---------------------------------------------------------------------------
# Step driver: two launches per decode step
# ---------------------------------------------------------------------------
class Step:
    """Per-step buffers of one batch and the two launches of a step.

    ``pre(head)``    -> propose + scheduler + fusion: draft, k, j, length, block
    ``post(logits)`` -> verify + commit: argmax, accept, emitted, out_tok
    ``post_sample(logits, inv_temp, uniform)`` -> the same step verified by
    sampling (point-mass drafts): accept, emitted, out_tok; ``exact=True``
    samples on the fixed-point weights (clk_verify_sample_exact_append)
    The previous step's accept/length feed the scheduler.  The block lengths
    alternate between two buffers, so that ``post`` can pass the previous
    step's lengths as the verify launch's prediction while ``pre`` writes the
    new ones; ``length`` is the buffer of the latest ``pre``.  The buffers are
    owned here, so their pointers are resolved once; a call only checks the
    tensor it is given.  The logits must hold all 1 + head + tail rows of
    every request."""

    def __init__(self, lookup: Lookup, slots: torch.Tensor):
        self.h = lookup
        self.slots = slots
        B = slots.numel()
        dev = slots.device
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
        self.B = B
        self.draft, self.k, self.j = z(B, BLOCK), z(B), z(B)
        self._len = [z(B), z(B)]
        self._cur = 0
        self.block = z(B, BLOCK)
        self.argmax, self.accept, self.emitted, self.out_tok = z(B, BLOCK), z(B), z(B), z(B, BLOCK)
        _ptr(slots, shape=(B,), name="slots")
        self._p = {n: getattr(self, n).data_ptr() for n in
                   ("slots", "draft", "k", "j", "block", "argmax", "accept", "emitted", "out_tok")}
        self._lp = [t.data_ptr() for t in self._len]
        self._head_shape = (B, lookup.params.head)
        self._rows = lookup.params.long_len
        self._lib = lib()
        self._sscratch = None

    @property
    def length(self) -> torch.Tensor:
        return self._len[self._cur]

    def reset(self):
        """Forget the previous step (after the slots are set up again)."""
        for t in self._len:
            t.zero_()
        self.accept.zero_()

    def resume(self, accept, length):
        """Continue from a checkpoint: the previous step's accepted counts and
        block lengths (int32 [B], as ``accept`` and ``length`` held them when
        the lookup was snapshotted), the inputs of the next scheduler step."""
        for t, name in ((accept, "accept"), (length, "length")):
            if tuple(t.shape) != (self.B,):
                raise ValueError(f"{name} must have shape ({self.B},)")
        for t in self._len:
            t.copy_(length)
        self.accept.copy_(accept)

    def pre(self, head, stream=None):
        if tuple(head.shape) != self._head_shape or head.dtype != torch.int32 or not head.is_cuda \
                or not head.is_contiguous():
            raise ValueError(f"head must be contiguous int32 {self._head_shape} on the GPU")
        p, prev, new = self._p, self._cur, self._cur ^ 1
        _check("clk_propose_fuse_sched",
               self._lib.clk_propose_fuse_sched(self.h.handle, p["slots"], self.B, head.data_ptr(), p["accept"],
                                                self._lp[prev], p["draft"], p["k"], p["j"], self._lp[new],
                                                p["block"], _stream(stream)))
        self._cur = new

    def post(self, logits, stream=None):
        dt, rs, qs, V = _logits_args(logits)
        if logits.shape[0] != self.B or logits.shape[1] < self._rows:
            raise ValueError(f"logits must be [{self.B}, >= {self._rows}, V]")
        p = self._p
        _check("clk_verify_append",
               self._lib.clk_verify_append(self.h.handle, p["slots"], logits.data_ptr(), dt, rs, qs, V, self.B,
                                           p["block"], self._lp[self._cur], self._lp[self._cur ^ 1], p["argmax"],
                                           p["accept"], p["emitted"], p["out_tok"], _stream(stream)))

    def post_sample(self, logits, inv_temp, uniform, stream=None, exact: bool = False):
        """Verify the block by sampling at inverse temperatures inv_temp
        (float32 [B]) with the uniforms uniform (float32 [B, 16, 2]), and
        commit the emitted tokens.  Like ``post`` it passes the previous
        step's lengths as the prediction of the new ones.  exact=True: on the
        fixed-point weights (clk_verify_sample_exact_append)."""
        dt, rs, qs, V = _logits_args(logits)
        if logits.shape[0] != self.B or logits.shape[1] < self._rows:
            raise ValueError(f"logits must be [{self.B}, >= {self._rows}, V]")
        key = (logits.dtype, V, bool(exact))
        if self._sscratch is None or self._sscratch[0] != key:
            make = verify_sample_exact_scratch if exact else verify_sample_scratch
            self._sscratch = (key, make(logits.dtype, V, self.B, device=self.slots.device, stream=stream, halves=2))
        p = self._p
        sc = self._sscratch[1]
        name = "clk_verify_sample_exact_append" if exact else "clk_verify_sample_append"
        _check(name,
               getattr(self._lib, name)(self.h.handle, p["slots"], logits.data_ptr(), dt, rs, qs, V,
                                                  self.B, p["block"], self._lp[self._cur], self._lp[self._cur ^ 1],
                                                  _ptr(inv_temp, torch.float32, (self.B,), "inv_temp"),
                                                  _ptr(uniform, torch.float32, (self.B, BLOCK, 2), "uniform"),
                                                  p["accept"], p["emitted"], p["out_tok"], sc.data_ptr(), sc.numel(),
                                                  _stream(stream)))
