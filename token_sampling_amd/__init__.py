"""token_sampling_amd -- Python binding of libspecverify, the MI355X (gfx950)
verifier acceptance step for speculative decoding.

This module only marshals arguments: it checks tensor shapes, dtypes and
devices, allocates outputs and the workspace with torch, and calls the C ABI
declared in ``include/specverify.h`` on the current torch stream.  Every step
of the computation runs in the HIP kernels of ``libspecverify.so``; there is
no CPU or PyTorch fallback, and the calls raise if the library is missing.

The operation is the acceptance step of the SDCP Internet-Draft ("Speculative
Decoding Coordination Protocol (SDCP) for Distributed Inference with
Multi-Level Caches"), Sec. 4.1 (sampling profile) and Sec. 6.4 (Rule 1 greedy,
Rule 2 speculative sampling).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

BF16 = 0
FP32 = 1
FP16 = 2  # caches only
RULE_GREEDY = 1
RULE_SPECULATIVE = 2
RULE_RELAXED = 192  # private use: accept while p_i(x_i) > 0
OK = 0
ERR_ARG = -1
ERR_DEVICE = -2
ERR_WORKSPACE = -3
S_BAD_PROPOSAL = -1
S_LIMIT = -2
S_Q_UNAVAILABLE = -3
S_BAD_PROFILE = -4
S_BAD_LOGITS = -5
S_BAD_CONTROL = -6  # adjust_logits: penalties, slot, bias offsets or mask row out of range
S_NO_PAGES = -7  # cache_reserve: not enough free pages
S_BAD_CACHE = -8  # cache_*: slot out of range, listed twice, or pages missing

SAMPLING_DTYPE = np.dtype(
    [("temperature_milli", "<u4"), ("top_k", "<u4"), ("top_p_milli", "<u4"),
     ("reserved", "<u4"), ("session_key", "<u8")],
    align=True,
)
# SDCP Sec. 6.4 inputs of the verifier values: 16-octet session id, the
# profile's seed, the round (32 bytes, 8-aligned; sv_sdcp_session).
SDCP_SESSION_DTYPE = np.dtype(
    [("session_id", np.uint8, (16,)), ("seed", "<u8"), ("round", "<u4"), ("reserved", "<u4")],
    align=True,
)
# SDCP Sec. 6.5.2 actions and the commit step's records (sv_contract,
# sv_session_state, 64 bytes each).
ACT_CONTINUE, ACT_REDUCE, ACT_SWITCH, ACT_SELF_DECODE, ACT_FINISH, ACT_FAIL = range(6)
CONTRACT_DTYPE = np.dtype(
    [("m_max", "<u4"), ("max_new", "<u4"), ("low_rounds", "<u4"), ("low_ratio", "<u4"),
     ("n_stop", "<u4"), ("stop", "<i4", (8,)), ("n_fallback", "<u4"), ("fallback", "u1", (8,))],
    align=True,
)
STATE_DTYPE = np.dtype(
    [("digest", "u1", (32,)), ("n", "<u4"), ("m_cap", "<u4"), ("c", "<u4"), ("g", "<u4"),
     ("j", "<u4"), ("reserved", "<u4", (3,))],
    align=True,
)
EXPORTED = ("sv_workspace_bytes", "sv_verify", "sv_verify_sdcp", "sv_verify_qrows",
            "sv_verify_early", "sv_commit",
            "sv_prefix_digest", "sv_contract_digest", "sv_strerror", "sv_status_str",
            "sv_version", "sv_bench_row_events", "sv_verify_noalloc", "sv_verify_commit",
            "sv_adjust_logits", "sv_count_tokens", "sv_grammar_masks", "sv_grammar_advance",
            "sv_cache_workspace_bytes", "sv_cache_reserve", "sv_cache_keep", "sv_cache_fork",
            "sv_cache_compact", "sv_cache_write", "sv_cache_plan_bytes", "sv_cache_plan",
            "sv_cache_attention_bytes", "sv_cache_attention")
# Per-session penalties for repeated tokens (sv_penalties, 16 bytes).
PENALTIES_DTYPE = np.dtype([("repetition", "<f4"), ("frequency", "<f4"), ("presence", "<f4"),
                            ("reserved", "<u4")], align=True)


class SvError(RuntimeError):
    pass


class _Probe(ctypes.Structure):
    _fields_ = [("p_tok", ctypes.c_void_p), ("q_tok", ctypes.c_void_p)]


class _CommitIO(ctypes.Structure):
    _fields_ = [("contracts", ctypes.c_void_p), ("states", ctypes.c_void_p),
                ("self_decode_ok", ctypes.c_void_p), ("emitted_len", ctypes.c_void_p),
                ("action", ctypes.c_void_p)]


class _History(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("seen", ctypes.c_void_p), ("n_slots", ctypes.c_int32)]


class _Bias(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("values", ctypes.c_void_p),
                ("n", ctypes.c_int32)]


class _Masks(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("n_masks", ctypes.c_int32)]


class _Grammar(ctypes.Structure):
    _fields_ = [("next", ctypes.c_void_p), ("classes", ctypes.c_void_p),
                ("accept", ctypes.c_void_p), ("n_states", ctypes.c_int32),
                ("n_classes", ctypes.c_int32)]


class _Vocab(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("end", ctypes.c_void_p),
                ("n_bytes", ctypes.c_int32), ("n_end", ctypes.c_int32), ("V", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("k", "v", "table", "lens", "held", "refs")] + [
        (f, ctypes.c_int32) for f in ("dtype", "n_layers", "n_pages", "n_kv", "page", "head_dim",
                                      "n_slots", "max_pages")]


class _Rows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (f, ctypes.c_int64) for f in ("k_session", "k_row", "k_head", "v_session", "v_row", "v_head")]


class History(NamedTuple):
    """Which tokens each slot has had (sv_history): counts [n_slots, V] int32 of
    the output tokens, seen [n_slots, 2, W] int32 bit rows over the vocabulary, W
    = (V + 31) // 32 (plane 0: prompt, plane 1: output).  See make_history."""
    counts: "torch.Tensor"  # noqa: F821
    seen: "torch.Tensor"  # noqa: F821


class Bias(NamedTuple):
    """Sparse biases (sv_bias): session b's entries are offsets[b]..offsets[b+1]-1
    of ids (int32, strictly ascending within a session) and values (float32).
    See make_bias."""
    offsets: "torch.Tensor"  # noqa: F821
    ids: "torch.Tensor"  # noqa: F821
    values: "torch.Tensor"  # noqa: F821


class Grammar(NamedTuple):
    """A byte automaton (sv_grammar): next [n_states, n_classes] int32 (-1:
    refused), classes [256] uint8, accept [n_states] uint8.  See make_grammar."""
    next: "torch.Tensor"  # noqa: F821
    classes: "torch.Tensor"  # noqa: F821
    accept: "torch.Tensor"  # noqa: F821


class Vocab(NamedTuple):
    """The tokens' bytes (sv_vocab): bytes uint8, offsets [V + 1] int32, end: up to
    8 int32 ids of the tokens that end a text.  See make_vocab."""
    bytes: "torch.Tensor"  # noqa: F821
    offsets: "torch.Tensor"  # noqa: F821
    end: "torch.Tensor"  # noqa: F821


class Cache(NamedTuple):
    """A paged cache of keys and values (sv_cache): k, v [n_layers, n_pages, n_kv,
    page, head_dim] bf16/fp16, whose page * head_dim elements of a head stand in the
    matrix instructions' order (cache_order); table [n_slots, max_pages] the slots'
    pages (-1: none), lens and held [n_slots] their tokens and pages, refs [n_pages]
    how many lists hold each page, all int32.  See make_cache."""
    k: "torch.Tensor"  # noqa: F821
    v: "torch.Tensor"  # noqa: F821
    table: "torch.Tensor"  # noqa: F821
    lens: "torch.Tensor"  # noqa: F821
    held: "torch.Tensor"  # noqa: F821
    refs: "torch.Tensor"  # noqa: F821


class CachePlan(NamedTuple):
    """How a round's attention is split (cache_plan), for B sessions of up to R rows
    and n_heads query heads over a cache of n_kv heads of head_dim; status [B] int32;
    workspace_bytes: what cache_attention needs; lists: the cache's page, n_slots and
    max_pages, which say where its lists of pages end."""
    buffer: "torch.Tensor"  # noqa: F821
    status: "torch.Tensor"  # noqa: F821
    n_heads: int
    B: int
    R: int
    n_kv: int
    head_dim: int
    workspace_bytes: int
    lists: tuple = None


class HipEvent:
    """A raw hipEvent_t (for the benchmark hook's row-kernel timing slots)."""

    _hip = None

    def __init__(self):
        if HipEvent._hip is None:
            h = ctypes.CDLL("libamdhip64.so")
            h.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
            h.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                              ctypes.c_void_p]
            h.hipEventSynchronize.argtypes = [ctypes.c_void_p]
            h.hipEventDestroy.argtypes = [ctypes.c_void_p]
            HipEvent._hip = h
        self._destroy = HipEvent._hip.hipEventDestroy  # kept for interpreter shutdown
        self.handle = ctypes.c_void_p()
        rc = HipEvent._hip.hipEventCreate(ctypes.byref(self.handle))
        if rc != 0:
            raise SvError(f"hipEventCreate failed ({rc})")

    def elapsed_ms(self, end: "HipEvent") -> float:
        HipEvent._hip.hipEventSynchronize(end.handle)
        ms = ctypes.c_float()
        rc = HipEvent._hip.hipEventElapsedTime(ctypes.byref(ms), self.handle, end.handle)
        if rc != 0:
            raise SvError(f"hipEventElapsedTime failed ({rc})")
        return float(ms.value)

    def __del__(self):
        if self.handle:
            self._destroy(self.handle)


_lib = None


def lib():
    """Load libspecverify.so (raises SvError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise SvError(f"{LIB_PATH} is missing: run token_sampling_amd.build.build() first")
        L = ctypes.CDLL(LIB_PATH)
        L.sv_workspace_bytes.argtypes = [ctypes.c_int32] * 3
        L.sv_workspace_bytes.restype = ctypes.c_size_t
        L.sv_verify.argtypes = [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
            ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify.restype = ctypes.c_int
        L.sv_verify_sdcp.argtypes = [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
            ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify_sdcp.restype = ctypes.c_int
        L.sv_verify_qrows.argtypes = [
            ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
            ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify_qrows.restype = ctypes.c_int
        L.sv_verify_early.argtypes = [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32,
            ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
            ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify_early.restype = ctypes.c_int
        L.sv_commit.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int32, ctypes.c_int32,
                                                         ctypes.c_void_p, ctypes.c_void_p,
                                                         ctypes.c_void_p]
        L.sv_commit.restype = ctypes.c_int
        L.sv_prefix_digest.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_uint32,
                                       ctypes.c_char_p]
        L.sv_prefix_digest.restype = ctypes.c_int
        L.sv_contract_digest.argtypes = [ctypes.c_char_p, ctypes.c_size_t, ctypes.c_char_p]
        L.sv_contract_digest.restype = ctypes.c_int
        L.sv_strerror.argtypes = [ctypes.c_int]
        L.sv_strerror.restype = ctypes.c_char_p
        L.sv_status_str.argtypes = [ctypes.c_int]
        L.sv_status_str.restype = ctypes.c_char_p
        L.sv_version.argtypes = []
        L.sv_version.restype = ctypes.c_int
        L.sv_bench_row_events.argtypes = [ctypes.c_void_p] * 3
        L.sv_bench_row_events.restype = ctypes.c_int
        L.sv_verify_noalloc.argtypes = [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify_noalloc.restype = ctypes.c_int
        L.sv_verify_commit.argtypes = [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
            ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32,
            ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(_CommitIO),
            ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(_Probe), ctypes.c_void_p,
        ]
        L.sv_verify_commit.restype = ctypes.c_int
        p, i = ctypes.c_void_p, ctypes.c_int32
        L.sv_adjust_logits.argtypes = [
            p, ctypes.c_int64, ctypes.c_int64, i, p, p, p, ctypes.POINTER(_History), p,
            ctypes.POINTER(_Bias), ctypes.POINTER(_Masks), i, i, i, i, p, p, p]
        L.sv_count_tokens.argtypes = [ctypes.POINTER(_History), p, p, p, p, i, i, i, i, i, p]
        L.sv_grammar_masks.argtypes = [ctypes.POINTER(_Grammar), ctypes.POINTER(_Vocab), p, i, p, p]
        L.sv_grammar_advance.argtypes = [ctypes.POINTER(_Grammar), ctypes.POINTER(_Vocab), p, p, p,
                                         i, i, p, p, p]
        n, c = ctypes.c_size_t, ctypes.POINTER(_Cache)
        L.sv_cache_reserve.argtypes = [c, p, p, i, p, p, n, p]
        L.sv_cache_keep.argtypes = [c, p, p, i, i, p, p]
        L.sv_cache_fork.argtypes = [c, p, p, i, p, p]
        L.sv_cache_compact.argtypes = [c, p, p, p, n, p]
        L.sv_cache_write.argtypes = [c, i, ctypes.POINTER(_Rows), p, p, p, i, i, p]
        L.sv_cache_plan.argtypes = [c, p, p, i, i, i, p, p, n, p]
        L.sv_cache_attention.argtypes = [c, i, p] + [ctypes.c_int64] * 3 + [
            ctypes.c_float, p, i, i, i, p, p, n, p]
        for f in (L.sv_adjust_logits, L.sv_count_tokens, L.sv_grammar_masks, L.sv_grammar_advance,
                  L.sv_cache_reserve, L.sv_cache_keep, L.sv_cache_fork, L.sv_cache_compact,
                  L.sv_cache_write, L.sv_cache_plan, L.sv_cache_attention):
            f.restype = ctypes.c_int
        L.sv_cache_workspace_bytes.argtypes = [c, i]
        L.sv_cache_plan_bytes.argtypes = L.sv_cache_attention_bytes.argtypes = [c, i, i, i]
        for f in (L.sv_cache_workspace_bytes, L.sv_cache_plan_bytes, L.sv_cache_attention_bytes):
            f.restype = n
        _lib = L
    return _lib


def workspace_bytes(B: int, M: int, V: int) -> int:
    return int(lib().sv_workspace_bytes(B, M, V))


def strerror(code: int) -> str:
    return lib().sv_strerror(code).decode()


def status_str(status: int) -> str:
    return lib().sv_status_str(status).decode()


def make_sampling(B, temperature_milli=1000, top_k=0, top_p_milli=1000, session_key=None,
                  device="cuda"):
    """Pack per-session profiles into the [B] x 24-byte device array."""
    import torch

    s = np.zeros(B, dtype=SAMPLING_DTYPE)
    s["temperature_milli"] = temperature_milli
    s["top_k"] = top_k
    s["top_p_milli"] = top_p_milli
    s["session_key"] = np.arange(B, dtype=np.uint64) if session_key is None else session_key
    raw = np.ascontiguousarray(s).view(np.uint8).reshape(B, 24)
    return torch.from_numpy(raw.copy()).to(device)


def make_sdcp_sessions(B, seed, round_, session_ids=None, device="cuda"):
    """Pack per-session SDCP value inputs into the [B] x 32-byte device array.

    seed and round_ are scalars or length-B sequences; session_ids is a
    [B, 16] array of octets (default: b as the last eight octets, big-endian).
    """
    import torch

    s = np.zeros(B, dtype=SDCP_SESSION_DTYPE)
    if session_ids is None:
        ids = np.zeros((B, 16), dtype=np.uint8)
        ids[:, 8:] = np.arange(B, dtype=">u8").view(np.uint8).reshape(B, 8)
    else:
        ids = np.asarray(session_ids, dtype=np.uint8).reshape(B, 16)
    s["session_id"] = ids
    s["seed"] = seed
    s["round"] = round_
    raw = np.ascontiguousarray(s).view(np.uint8).reshape(B, 32)
    return torch.from_numpy(raw.copy()).to(device)


def make_contracts(B, m_max=8, max_new=256, low_rounds=3, low_ratio=0, stop=(),
                   fallback=(ACT_REDUCE, ACT_SWITCH, ACT_SELF_DECODE, ACT_FAIL), device="cuda"):
    """Pack per-session contract members (SDCP Sec. 4.1) into [B, 64] device bytes.
    Every argument is a scalar (or a sequence, for stop and fallback) shared by
    all sessions, or a list of B of them."""
    import torch

    c = np.zeros(B, dtype=CONTRACT_DTYPE)
    c["m_max"], c["max_new"], c["low_rounds"], c["low_ratio"] = m_max, max_new, low_rounds, low_ratio
    per = [stop] * B if len(stop) == 0 or np.isscalar(stop[0]) else stop
    for b, st in enumerate(per):
        c["n_stop"][b] = len(st)
        c["stop"][b, :min(len(st), 8)] = list(st)[:8]
    per = [fallback] * B if len(fallback) == 0 or np.isscalar(fallback[0]) else fallback
    for b, fb in enumerate(per):
        c["n_fallback"][b] = len(fb)
        c["fallback"][b, :min(len(fb), 8)] = list(fb)[:8]
    raw = np.ascontiguousarray(c).view(np.uint8).reshape(B, 64)
    return torch.from_numpy(raw.copy()).to(device)


def make_states(B, digest=b"\0" * 32, n=0, m_cap=8, device="cuda"):
    """Initial per-session states ([B, 64] device bytes): digest d[n] (32 bytes,
    or a [B, 32] array), n committed tokens, m_cap, counters zero."""
    import torch

    s = np.zeros(B, dtype=STATE_DTYPE)
    s["digest"] = np.asarray(np.frombuffer(digest, np.uint8) if isinstance(digest, bytes)
                             else digest, dtype=np.uint8)
    s["n"], s["m_cap"] = n, m_cap
    raw = np.ascontiguousarray(s).view(np.uint8).reshape(B, 64)
    return torch.from_numpy(raw.copy()).to(device)


def states_numpy(states):
    """Host copy of device state records as a STATE_DTYPE array."""
    raw = states.cpu().numpy().astype(np.uint8, copy=False)
    return raw.reshape(-1, 64).copy().view(STATE_DTYPE).reshape(-1)


def prefix_digest(contract_digest: bytes, prompt) -> bytes:
    """d[0] of SDCP Sec. 4.2 (host)."""
    p = np.ascontiguousarray(prompt, dtype=np.int32)
    out = ctypes.create_string_buffer(32)
    rc = lib().sv_prefix_digest(bytes(contract_digest), p.ctypes.data, p.shape[0], out)
    if rc != OK:
        raise SvError(f"sv_prefix_digest failed ({rc})")
    return out.raw


def contract_digest(cbor: bytes) -> bytes:
    """contract_digest of SDCP Sec. 4.1 over a deterministic CBOR encoding (host)."""
    out = ctypes.create_string_buffer(32)
    rc = lib().sv_contract_digest(bytes(cbor), len(cbor), out)
    if rc != OK:
        raise SvError(f"sv_contract_digest failed ({rc})")
    return out.raw


def commit(contracts, states, m, accepted_len, out_tokens, self_decode_ok=None, stream=None,
           out=None):
    """sv_commit on device tensors: contracts [B, 64] and states [B, 64] uint8
    (see make_contracts / make_states), m and accepted_len [B] int32, out_tokens
    [B, M+1] int32 (truncated in place), self_decode_ok [B] uint8 or None.
    Returns dict(emitted_len, action), both [B] int32."""
    import torch

    dev = out_tokens.device
    B, M1 = out_tokens.shape
    for t, name, dt in ((contracts, "contracts", torch.uint8), (states, "states", torch.uint8)):
        _check(t, name, dt, (B, 64), dev)
    _check(m, "m", torch.int32, (B,), dev)
    _check(accepted_len, "accepted_len", torch.int32, (B,), dev)
    _check(out_tokens, "out_tokens", torch.int32, (B, M1), dev)
    if self_decode_ok is not None:
        _check(self_decode_ok, "self_decode_ok", torch.uint8, (B,), dev)
    if out is None:
        out = {"emitted_len": torch.empty(B, dtype=torch.int32, device=dev),
               "action": torch.empty(B, dtype=torch.int32, device=dev)}
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    rc = lib().sv_commit(contracts.data_ptr(), states.data_ptr(), m.data_ptr(),
                         accepted_len.data_ptr(), out_tokens.data_ptr(),
                         None if self_decode_ok is None else self_decode_ok.data_ptr(), B, M1 - 1,
                         out["emitted_len"].data_ptr(), out["action"].data_ptr(),
                         stream.cuda_stream)
    if rc != OK:
        raise SvError(f"sv_commit failed: {strerror(rc)} ({rc})")
    return out


def _check(t, name, dtype, shape, device):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def verify(target, draft, tokens, m, rule, sampling, seed: int, round_: int, probe: bool = False,
           workspace=None, out=None, stream=None, row_events=None, sdcp_sessions=None,
           q_rows=None, early=None, commit=None):
    """sv_verify, sv_verify_sdcp, sv_verify_qrows or sv_verify_early on torch
    tensors (all on one GPU device).

    target [B, M+1, V] bf16/fp32, draft [B, M, V] same dtype or None, tokens
    [B, M] int32, m [B] int32, rule [B] int32, sampling [B, 24] uint8 (see
    make_sampling).  Returns a dict with accepted_len [B] and out_tokens
    [B, M+1] (int32), plus p_tok and q_tok [B, M] float64 if probe.  The call
    is asynchronous on ``stream`` (default: torch's current stream).
    row_events: optional (start, stop) or (start, mid, stop) HipEvents recorded
        around the row kernels, mid between the single-pass kernel and the other
        (the library's benchmark hook, sv_bench_row_events, set for this call).
    sdcp_sessions: optional [B, 32] uint8 device array (see make_sdcp_sessions);
        then the SDCP Sec. 6.4 values are used and seed, round_ are ignored.
    q_rows: optional [B, M, V] float32 draft distributions (SDCP q_rows) in place
        of draft logits (draft must then be None): sv_verify_qrows.
    early: the first window (1..65 positions) of the in-order reading,
        sv_verify_early (with either draft source and either value source); None:
        every row is read.
    commit: optional (contracts, states, self_decode_ok or None), device arrays
        as for commit(): the acceptance step and the commit step in one call,
        sv_verify_commit (draft logits, either value source, every row read);
        the result then also holds emitted_len and action [B] int32, and out_tokens
        is truncated as sv_commit truncates it.
    """
    import torch

    if not (isinstance(target, torch.Tensor) and target.dim() == 3):
        raise ValueError("target must be a [B, M+1, V] tensor")
    dev = target.device
    if dev.type != "cuda":
        raise ValueError("target must be a GPU tensor")
    B, M1, V = target.shape
    M = M1 - 1
    if target.dtype == torch.bfloat16:
        dt = BF16
    elif target.dtype == torch.float32:
        dt = FP32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    _check(target, "target", None, None, dev)
    if draft is not None:
        _check(draft, "draft", target.dtype, (B, M, V), dev)
    _check(tokens, "tokens", torch.int32, (B, M), dev)
    _check(m, "m", torch.int32, (B,), dev)
    _check(rule, "rule", torch.int32, (B,), dev)
    _check(sampling, "sampling", None, None, dev)
    if sampling.numel() * sampling.element_size() != 24 * B:
        raise ValueError("sampling must hold B 24-byte records")
    if q_rows is not None:
        if draft is not None:
            raise ValueError("give draft logits or q_rows, not both")
        _check(q_rows, "q_rows", torch.float32, (B, M, V), dev)
    if sdcp_sessions is not None:
        _check(sdcp_sessions, "sdcp_sessions", None, None, dev)
        if sdcp_sessions.numel() * sdcp_sessions.element_size() != 32 * B:
            raise ValueError("sdcp_sessions must hold B 32-byte records")

    cio = None
    if commit is not None:
        if q_rows is not None or early is not None:
            raise ValueError("commit= takes draft logits and reads every row")
        contracts, states, self_ok = commit
        for t, name in ((contracts, "contracts"), (states, "states")):
            _check(t, name, torch.uint8, (B, 64), dev)
        if self_ok is not None:
            _check(self_ok, "self_decode_ok", torch.uint8, (B,), dev)
    need = workspace_bytes(B, M, V)
    if need == 0:
        raise SvError("sizes out of range")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.numel() * workspace.element_size() < need:
        raise SvError("workspace too small")
    if out is None:
        out = {
            "accepted_len": torch.empty(B, dtype=torch.int32, device=dev),
            "out_tokens": torch.empty((B, M + 1), dtype=torch.int32, device=dev),
        }
        if probe:
            out["p_tok"] = torch.empty((B, M), dtype=torch.float64, device=dev)
            out["q_tok"] = torch.empty((B, M), dtype=torch.float64, device=dev)
    if commit is not None:
        for k in ("emitted_len", "action"):
            if k not in out:
                out[k] = torch.empty(B, dtype=torch.int32, device=dev)
        cio = ctypes.byref(_CommitIO(contracts.data_ptr(), states.data_ptr(),
                                     None if self_ok is None else self_ok.data_ptr(),
                                     out["emitted_len"].data_ptr(), out["action"].data_ptr()))
    pr = None
    if "p_tok" in out:
        pr = ctypes.byref(_Probe(out["p_tok"].data_ptr(), out["q_tok"].data_ptr()))
    evs = None
    if row_events is not None:
        evs = ([row_events[0].handle, None, row_events[1].handle] if len(row_events) == 2
               else [e.handle for e in row_events])
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    common = (target.data_ptr(), None if draft is None else draft.data_ptr(), dt,
              tokens.data_ptr(), m.data_ptr(), rule.data_ptr(), sampling.data_ptr())
    tail = (out["accepted_len"].data_ptr(), out["out_tokens"].data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), pr,
            stream.cuda_stream)
    sess = None if sdcp_sessions is None else sdcp_sessions.data_ptr()
    if evs is not None:
        lib().sv_bench_row_events(*evs)
    try:
        if cio is not None:
            name = "sv_verify_commit"
            rc = lib().sv_verify_commit(*common, sess, B, M, V, seed, round_, tail[0], tail[1],
                                        cio, *tail[2:])
        else:
            rc, name = _call(common, tail, target, q_rows, dt, sess, B, M, V, seed, round_,
                             early)
    finally:
        if evs is not None:
            lib().sv_bench_row_events(None, None, None)
    if rc != OK:
        raise SvError(f"{name} failed: {strerror(rc)} ({rc})")
    return out


def _call(common, tail, target, q_rows, dt, sess, B, M, V, seed, round_, early):
    if early is not None:
        name = "sv_verify_early"
        rc = lib().sv_verify_early(target.data_ptr(), common[1],
                                   None if q_rows is None else q_rows.data_ptr(), dt,
                                   *common[3:], sess, B, M, V, seed, round_, int(early), *tail)
    elif q_rows is not None:
        name = "sv_verify_qrows"
        rc = lib().sv_verify_qrows(target.data_ptr(), dt, q_rows.data_ptr(), *common[3:], sess,
                                   B, M, V, seed, round_, *tail)
    elif sess is None:
        name = "sv_verify"
        rc = lib().sv_verify(*common, B, M, V, seed, round_, *tail)
    else:
        name = "sv_verify_sdcp"
        rc = lib().sv_verify_sdcp(*common, sess, B, M, V, *tail)
    return rc, name


# ---------------------------------------------------------------------------
# Per-session rules on logits and the state they keep (sv_adjust_logits,
# sv_count_tokens, sv_grammar_masks, sv_grammar_advance).

def make_penalties(B, repetition=1.0, frequency=0.0, presence=0.0, device="cuda"):
    """Pack per-session penalties (scalars or length-B sequences) into the
    [B] x 16-byte device array."""
    import torch

    s = np.zeros(B, dtype=PENALTIES_DTYPE)
    s["repetition"], s["frequency"], s["presence"] = repetition, frequency, presence
    for f in ("repetition", "frequency", "presence"):
        if not np.isfinite(s[f]).all():
            raise ValueError(f"{f} must be finite")
    if not ((s["repetition"] >= 2.0**-64) & (s["repetition"] <= 2.0**64)).all():
        raise ValueError("repetition must be within 2^-64 .. 2^64")
    return torch.from_numpy(s.view(np.uint8).reshape(B, 16).copy()).to(device)


def make_history(n_slots, V, device="cuda"):
    """An empty History of n_slots slots for a vocabulary of V tokens (V * 4 + V / 4
    bytes a slot)."""
    import torch

    return History(torch.zeros((n_slots, V), dtype=torch.int32, device=device),
                   torch.zeros((n_slots, 2, (V + 31) // 32), dtype=torch.int32, device=device))


def make_bias(biases, V, device="cuda"):
    """Bias from one {token: bias} mapping per session (empty or None: none)."""
    import torch

    offsets, ids, values = [0], [], []
    for d in biases:
        for t in sorted(d or ()):
            if not 0 <= t < V:
                raise ValueError(f"bias for token {t}, outside the vocabulary of {V}")
            ids.append(t)
            values.append(d[t])
        offsets.append(len(ids))
    with np.errstate(over="ignore"):
        packed = np.asarray(values, dtype=np.float64).astype(np.float32)
    for t, x in zip(ids, packed):  # as they will be added: a large double is an infinity here
        if not x < np.inf:
            raise ValueError(f"bias of token {t} must be -inf or finite in binary32")
    return Bias(torch.tensor(offsets, dtype=torch.int32).to(device),
                torch.tensor(ids, dtype=torch.int32).to(device),
                torch.from_numpy(packed).to(device))


def make_masks(allowed, device="cuda"):
    """[n, V] truth values (allowed tokens) as [n, W] int32 bit rows."""
    import torch

    a = np.asarray(allowed, dtype=bool)
    if a.ndim != 2:
        raise ValueError("allowed must be [n, V]")
    full = np.zeros((a.shape[0], (a.shape[1] + 31) // 32 * 32), bool)
    full[:, :a.shape[1]] = a
    words = np.packbits(full, axis=1, bitorder="little").view("<i4")
    return torch.from_numpy(words.copy()).to(device)


def make_grammar(next_state, accept, device="cuda"):
    """Grammar from next_state [n_states, 256] (a byte's next state, -1: refused) and
    accept [n_states]: bytes that no state tells apart share a class."""
    import torch

    nxt = np.asarray(next_state)
    if nxt.ndim != 2 or nxt.shape[1] != 256 or nxt.shape[0] < 1:
        raise ValueError("next_state must be [n_states, 256]")
    acc = np.asarray(accept).astype(bool).astype(np.uint8)
    if acc.shape != (nxt.shape[0],):
        raise ValueError("accept must be [n_states]")
    if nxt.min() < -1 or nxt.max() >= nxt.shape[0]:
        raise ValueError("next_state holds a state outside [-1, n_states)")
    table, classes = np.unique(nxt, axis=1, return_inverse=True)
    return Grammar(torch.from_numpy(np.ascontiguousarray(table, dtype=np.int32)).to(device),
                   torch.from_numpy(classes.reshape(-1).astype(np.uint8)).to(device),
                   torch.from_numpy(acc).to(device))


def make_vocab(tokens, end=(), device="cuda"):
    """Vocab from the tokens' byte strings (b"" for control tokens) and the ids of
    the tokens that end a text (at most 8)."""
    import torch

    end = list(end)
    if len(end) > 8 or any(not 0 <= t < len(tokens) for t in end):
        raise ValueError("end must hold at most 8 ids of the vocabulary")
    offsets = np.zeros(len(tokens) + 1, np.int64)
    np.cumsum([len(t) for t in tokens], out=offsets[1:])
    if offsets[-1] > 1 << 30:
        raise ValueError("the tokens' bytes exceed 1 GiB")
    flat = np.frombuffer(b"".join(tokens), dtype=np.uint8)
    return Vocab(torch.from_numpy(flat.copy()).to(device),
                 torch.from_numpy(offsets.astype(np.int32)).to(device),
                 torch.tensor(end, dtype=torch.int32).to(device))


_HERE = contextlib.nullcontext()


def _launch(dev, stream):
    """(stream handle, context): the call's stream, and a context in which the
    tensors' device is current and new tensors belong to that stream."""
    import torch

    if dev.index == torch.cuda.current_device():
        here = torch._C._cuda_getCurrentRawStream(dev.index)
        if stream is None or stream.cuda_stream == here:
            return here, _HERE
        return stream.cuda_stream, torch.cuda.stream(stream)
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(dev))
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    else:
        both.enter_context(torch.cuda.stream(stream))
    return stream.cuda_stream, both


def _want(t, name, dtype, shape, device):
    """t's address, after _check's checks, quick where t is as it should be: these
    calls are short enough on the GPU for the host's checks to count."""
    try:
        if (t.dtype is dtype and t.get_device() == device.index and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, dtype, shape, device)
    return t.data_ptr()


def _device_of(t, name):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _int32(n, name):
    if n >= 1 << 31:
        raise ValueError(f"{name} holds 2^31 entries or more")
    return n


def _history_struct(history, V, dev):
    import torch

    n = history.counts.shape[0]
    return _History(_want(history.counts, "history.counts", torch.int32, (n, V), dev),
                    _want(history.seen, "history.seen", torch.int32, (n, 2, (V + 31) // 32), dev), n)


def adjust_logits(logits, tokens=None, m=None, penalties=None, history=None, slots=None, bias=None,
                  masks=None, mask_rows=None, out=None, status=None, stream=None):
    """sv_adjust_logits: penalties for repeated tokens, biases and masks on a round's
    logits, before verify().

    logits [B, R, V] bf16/fp32, the last axis contiguous (a slice of a padded
    vocabulary, or [R, B, V] transposed, will do); tokens [B, M] int32 the
    round's drafted tokens: R = M + 1 target rows or R = M draft rows (None: R =
    1, M = 0, a decoding step); m [B] int32 or None for M.  Each rule may be left
    out: penalties [B, 16] uint8 (make_penalties) with history (make_history,
    count_tokens) and slots [B] int32 (None: slot b); bias (make_bias); masks
    [n, W] int32 bit rows (make_masks, grammar_masks) with mask_rows [B, R] int32
    (-1: no mask).
    out: None for a new contiguous tensor; a contiguous one like it; or logits
    itself (in place, no two of its B * R rows may then overlap).  Rows that a session does
    not use are not written.  Returns dict(logits=out, status=[B] int32: 0, or
    why a session failed, whose rows are then NaN).
    """
    import torch

    dev = _device_of(logits, "logits")
    if logits.dim() != 3 or logits.numel() == 0:
        raise ValueError("logits must be a [B, R, V] tensor")
    B, R, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = BF16
    elif logits.dtype == torch.float32:
        dt = FP32
    else:
        raise TypeError("logits must be bfloat16 or float32")
    sb, sr, sv_ = logits.stride()
    if V > 1 and sv_ != 1:
        raise ValueError("the logits of a row must be contiguous")
    p_tokens = p_m = p_pen = p_slots = hist = bs = mk = None
    if tokens is None:
        if R != 1:
            raise ValueError("tokens may be left out only for one row a session")
        M = 0
        if m is not None:
            raise ValueError("m needs tokens")
    else:
        M = R - 1 if tokens.dim() == 2 and tokens.shape[1] == R - 1 else R
        p_tokens = _want(tokens, "tokens", torch.int32, (B, M), dev)
        if m is not None:
            p_m = _want(m, "m", torch.int32, (B,), dev)
    if penalties is not None:
        p_pen = _want(penalties, "penalties", torch.uint8, (B, 16), dev)
    if history is not None:
        hist = ctypes.byref(_history_struct(history, V, dev))
        if slots is None and history.counts.shape[0] < B:
            raise ValueError("history has fewer slots than sessions")
    if slots is not None:
        p_slots = _want(slots, "slots", torch.int32, (B,), dev)
    if bias is not None:
        n = _int32(bias.ids.numel(), "bias")
        bs = ctypes.byref(_Bias(_want(bias.offsets, "bias.offsets", torch.int32, (B + 1,), dev),
                                _want(bias.ids, "bias.ids", torch.int32, (n,), dev),
                                _want(bias.values, "bias.values", torch.float32, (n,), dev), n))
    if (masks is None) != (mask_rows is None):
        raise ValueError("masks and mask_rows go together")
    if masks is not None:
        n = masks.shape[0]
        if n < 1:
            raise ValueError("masks must hold a row")
        mk = ctypes.byref(_Masks(_want(masks, "masks", torch.int32, (n, (V + 31) // 32), dev),
                                 _want(mask_rows, "mask_rows", torch.int32, (B, R), dev), n))
    handle, on = _launch(dev, stream)
    with on:
        if out is None:
            out = torch.empty((B, R, V), dtype=logits.dtype, device=dev)
        elif out is not logits and out.data_ptr() == logits.data_ptr() and out.stride() == (sb, sr, sv_):
            _check_like(out, logits)
        elif out is not logits:
            _want(out, "out", logits.dtype, (B, R, V), dev)
            lo, hi = logits.data_ptr(), logits.data_ptr() + ((B - 1) * sb + (R - 1) * sr + V) * logits.element_size()
            if out.data_ptr() < hi and lo < out.data_ptr() + out.numel() * out.element_size():
                raise ValueError("out overlaps logits")
        if out.data_ptr() == logits.data_ptr() and not _rows_apart(sb, sr, B, R, V):
            raise ValueError("rows overlap: logits cannot be adjusted in place")
        if status is None:
            status = torch.empty(B, dtype=torch.int32, device=dev)
        else:
            _want(status, "status", torch.int32, (B,), dev)
        rc = lib().sv_adjust_logits(logits.data_ptr(), sb, sr, dt, p_tokens, p_m, p_pen, hist,
                                    p_slots, bs, mk, B, M, R, V, out.data_ptr(),
                                    status.data_ptr(), handle)
    if rc != OK:
        raise SvError(f"sv_adjust_logits failed: {strerror(rc)} ({rc})")
    return {"logits": out, "status": status}


def _rows_apart(sb, sr, B, R, V):
    """Whether no two of the B * R rows that start at b * sb + r * sr share one of
    their V logits."""
    near, far = sorted(((sb, B), (sr, R)))
    if near[1] == 1:  # all rows at one stride
        return far[1] == 1 or far[0] >= V
    if near[0] < V or (far[1] > 1 and far[0] < V):
        return False
    width = (near[1] - 1) * near[0] + V
    # the near stride's multiples on both sides of d far strides, as far as they reach
    for d in range(1, min(far[1], (width - 1) // far[0] + 1)):
        q = min(d * far[0] // near[0], near[1] - 1)
        if d * far[0] - q * near[0] < V or (q + 1 < near[1] and (q + 1) * near[0] - d * far[0] < V):
            return False
    return True


def _check_like(out, logits):
    if out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must have the logits' shape and dtype")


def count_tokens(history, tokens, slots=None, lens=None, offsets=None, prompt=False, clear=False,
                 stream=None):
    """sv_count_tokens: notes tokens in the history, in place.

    tokens [B, L] int32, the first lens[b] (None: L) of each row; or, with offsets
    [B + 1] int32, one line of tokens of which session b has offsets[b] ..
    offsets[b + 1] - 1.  Tokens outside the vocabulary (the -1 of out_tokens) are
    skipped.  slots [B] int32 (None: slot b; -1: skip).  prompt: prompt tokens
    rather than output tokens; clear: empty the listed slots first.  After
    commit(): count_tokens(history, out["out_tokens"], slots,
    lens=out["emitted_len"])."""
    import torch

    dev = _device_of(tokens, "tokens")
    V = history.counts.shape[-1]
    hist = _history_struct(history, V, dev)
    p_offsets = p_lens = p_slots = None
    if offsets is not None:
        if lens is not None:
            raise ValueError("give lens or offsets, not both")
        B, L = offsets.numel() - 1, _int32(tokens.numel(), "tokens")
        p_tokens = _want(tokens, "tokens", torch.int32, (L,), dev)
        p_offsets = _want(offsets, "offsets", torch.int32, (B + 1,), dev)
    else:
        if tokens.dim() != 2:
            raise ValueError("tokens must be [B, L] (or one line, with offsets)")
        B, L = tokens.shape
        p_tokens = _want(tokens, "tokens", torch.int32, tokens.shape, dev)
        if lens is not None:
            p_lens = _want(lens, "lens", torch.int32, (B,), dev)
    if slots is not None:
        p_slots = _want(slots, "slots", torch.int32, (B,), dev)
    elif history.counts.shape[0] < B:
        raise ValueError("history has fewer slots than sessions")
    handle, on = _launch(dev, stream)
    with on:
        rc = lib().sv_count_tokens(ctypes.byref(hist), p_slots, p_tokens, p_offsets, p_lens, B, L, V,
                                   0 if prompt else 1, int(clear), handle)
    if rc != OK:
        raise SvError(f"sv_count_tokens failed: {strerror(rc)} ({rc})")


def _grammar_structs(grammar, vocab, dev):
    import torch

    S, C = grammar.next.shape
    V = vocab.offsets.numel() - 1
    n, ends = _int32(vocab.bytes.numel(), "vocab.bytes"), vocab.end.numel()
    g = _Grammar(_want(grammar.next, "grammar.next", torch.int32, (S, C), dev),
                 _want(grammar.classes, "grammar.classes", torch.uint8, (256,), dev),
                 _want(grammar.accept, "grammar.accept", torch.uint8, (S,), dev), S, C)
    v = _Vocab(_want(vocab.bytes, "vocab.bytes", torch.uint8, (n,), dev),
               _want(vocab.offsets, "vocab.offsets", torch.int32, (V + 1,), dev),
               _want(vocab.end, "vocab.end", torch.int32, (ends,), dev), n, ends, V)
    return ctypes.byref(g), ctypes.byref(v), V


def grammar_masks(grammar, vocab, states, out=None, stream=None):
    """sv_grammar_masks: the masks of automaton states, [n, W] int32 bit rows for
    states [n] int32 (-1: every token allowed)."""
    import torch

    dev = _device_of(states, "states")
    g, v, V = _grammar_structs(grammar, vocab, dev)
    n = _int32(states.numel(), "states")
    p_states = _want(states, "states", torch.int32, (n,), dev)
    handle, on = _launch(dev, stream)
    with on:
        if out is None:
            out = torch.empty((n, (V + 31) // 32), dtype=torch.int32, device=dev)
        else:
            _want(out, "out", torch.int32, (n, (V + 31) // 32), dev)
        rc = lib().sv_grammar_masks(g, v, p_states, n, out.data_ptr(), handle)
    if rc != OK:
        raise SvError(f"sv_grammar_masks failed: {strerror(rc)} ({rc})")
    return out


def grammar_advance(grammar, vocab, states, tokens, lens=None, out=None, stream=None):
    """sv_grammar_advance: automaton states along tokens [B, L] int32 (the first
    lens[b], None: L) from states [B] int32 (-1: no grammar).  Returns
    dict(states=[B, L + 1] int32, the states after 0, 1, .. tokens; last=[B] int32,
    the state after all of them).  states, passed as mask_rows with the masks of
    all states, are the masks of a round's rows."""
    import torch

    dev = _device_of(tokens, "tokens")
    g, v, _ = _grammar_structs(grammar, vocab, dev)
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, L]")
    B, L = tokens.shape
    p_tokens = _want(tokens, "tokens", torch.int32, tokens.shape, dev)
    p_states = _want(states, "states", torch.int32, (B,), dev)
    p_lens = None if lens is None else _want(lens, "lens", torch.int32, (B,), dev)
    handle, on = _launch(dev, stream)
    with on:
        if out is None:
            out = {"states": torch.empty((B, L + 1), dtype=torch.int32, device=dev),
                   "last": torch.empty(B, dtype=torch.int32, device=dev)}
        else:
            _want(out["states"], "out['states']", torch.int32, (B, L + 1), dev)
            _want(out["last"], "out['last']", torch.int32, (B,), dev)
        rc = lib().sv_grammar_advance(g, v, p_states, p_tokens, p_lens, B, L,
                                      out["states"].data_ptr(), out["last"].data_ptr(), handle)
    if rc != OK:
        raise SvError(f"sv_grammar_advance failed: {strerror(rc)} ({rc})")
    return out


# ---------------------------------------------------------------------------
# The paged cache of keys and values and the attention that reads it (sv_cache_*).

def make_cache(n_slots, n_pages, max_pages, n_kv, head_dim, n_layers=1, page=64, dtype=None,
               device="cuda"):
    """An empty Cache: n_pages pages of `page` tokens (32, 64, 128 or 256) in each
    layer, n_slots sessions of at most max_pages pages.  head_dim 64, 96, 128 or 256;
    dtype torch.bfloat16 (None) or torch.float16."""
    import torch

    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("caches are bfloat16 or float16")
    if page not in (32, 64, 128, 256):
        raise ValueError("page must be 32, 64, 128 or 256")
    if head_dim not in (64, 96, 128, 256):
        raise ValueError("head_dim must be 64, 96, 128 or 256")
    shape = (n_layers, n_pages, n_kv, page, head_dim)

    def ints(value, *size):
        return torch.full(size, value, dtype=torch.int32, device=device)

    return Cache(torch.empty(shape, dtype=dtype, device=device),
                 torch.empty(shape, dtype=dtype, device=device), ints(-1, n_slots, max_pages),
                 ints(0, n_slots), ints(0, n_slots), ints(0, n_pages))


def cache_order(page, head_dim):
    """Where token t's dimension d of a head stands among the page * head_dim elements
    of a page: two [page, head_dim] int64 arrays, for keys and for values.  With
    them k[layer, p, head].flatten()[keys] are the page's keys by token."""
    place = np.arange(page * head_dim)
    keys = place.reshape(page // 32, 2, head_dim // 32, 4, 4, 4, 8).transpose(0, 4, 1, 5, 2, 3, 6)
    values = place.reshape(page // 32, head_dim // 16, 4, 16, 8).transpose(0, 2, 4, 1, 3)
    return keys.reshape(page, head_dim), values.reshape(page, head_dim)


def _cache_struct(cache, dev):
    """sv_cache of a Cache; its checks at once where all is as it should be (a round makes
    a call of this kind in every layer)."""
    import torch

    k, v, table, lens, held, refs = cache
    try:
        dtype, int32, i, shape = k.dtype, torch.int32, dev.index, k.shape
        n_layers, n_pages, n_kv, page, head_dim = shape
        n_slots, max_pages = table.shape
        slots = lens.shape
        good = (v.dtype is dtype and v.shape == shape and table.dtype is int32 and lens.dtype is int32
                and held.dtype is int32 and refs.dtype is int32 and slots == held.shape
                and slots[0] == n_slots and len(slots) == 1 and refs.shape == (n_pages,)
                and k.get_device() == i and v.get_device() == i and table.get_device() == i
                and lens.get_device() == i and held.get_device() == i and refs.get_device() == i
                and k.is_contiguous() and v.is_contiguous() and table.is_contiguous()
                and lens.is_contiguous() and held.is_contiguous() and refs.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        good = False
    if not good:
        for t, name in zip(cache, Cache._fields):
            _check(t, f"cache.{name}", torch.int32 if t is not k and t is not v else None, None, dev)
        if k.dim() != 5 or table.dim() != 2:
            raise ValueError("cache.k must be [n_layers, n_pages, n_kv, page, head_dim], cache.table "
                             "[n_slots, max_pages]")
        _check(v, "cache.v", k.dtype, k.shape, dev)
        for t, name, n in ((lens, "lens", table.shape[0]), (held, "held", table.shape[0]),
                           (refs, "refs", k.shape[1])):
            _check(t, f"cache.{name}", torch.int32, (n,), dev)
    if dtype is torch.bfloat16:
        code = BF16
    elif dtype is torch.float16:
        code = FP16
    else:
        raise TypeError("caches are bfloat16 or float16")
    return _Cache(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), held.data_ptr(),
                  refs.data_ptr(), code, n_layers, n_pages, n_kv, page, head_dim, n_slots, max_pages)


def _cache_slots(cache, slots, B, dev):
    import torch

    if slots is not None:
        return _want(slots, "slots", torch.int32, (B,), dev)
    if cache.table.shape[0] < B:
        raise ValueError("the cache has fewer slots than sessions")
    return None


def _status(status, B, dev):
    import torch

    if status is None:
        return torch.empty(B, dtype=torch.int32, device=dev)
    _want(status, "status", torch.int32, (B,), dev)
    return status


def _bytes(workspace, need, name, dev):
    """A workspace of at least need bytes (need 0: sizes that the library refuses)."""
    import torch

    if need == 0:
        raise SvError("sizes out of range")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _check(workspace, name, None, None, dev)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise SvError(f"{name} too small")
    return workspace, have


def _raise(rc, name):
    if rc != OK:
        raise SvError(f"{name} failed: {strerror(rc)} ({rc})")


def cache_reserve(cache, add, slots=None, status=None, workspace=None, stream=None):
    """sv_cache_reserve: pages for add [B] int32 more tokens of the sessions on slots
    [B] int32 (None: slot b; -1: none), and a copy of the page that the next token
    falls into where other lists hold it too.  Returns status [B] int32: 0,
    S_NO_PAGES, S_LIMIT or S_BAD_CACHE."""
    import torch

    dev = _device_of(add, "add")
    c = _cache_struct(cache, dev)
    B = add.numel()
    p_add = _want(add, "add", torch.int32, (B,), dev)
    p_slots = _cache_slots(cache, slots, B, dev)
    handle, on = _launch(dev, stream)
    with on:
        status = _status(status, B, dev)
        need = lib().sv_cache_workspace_bytes(ctypes.byref(c), B)
        workspace, size = _bytes(workspace, need, "workspace", dev)
        rc = lib().sv_cache_reserve(ctypes.byref(c), p_slots, p_add, B, status.data_ptr(),
                                    workspace.data_ptr(), size, handle)
    _raise(rc, "sv_cache_reserve")
    return status


def cache_keep(cache, count, slots=None, absolute=False, status=None, stream=None):
    """sv_cache_keep: the sessions' lengths become lens + count [B] int32 (the
    emitted_len of a commit), or count itself (absolute), and the pages behind are
    let go.  Returns status [B] int32: 0, S_LIMIT or S_BAD_CACHE."""
    import torch

    dev = _device_of(count, "count")
    c = _cache_struct(cache, dev)
    B = count.numel()
    p_count = _want(count, "count", torch.int32, (B,), dev)
    p_slots = _cache_slots(cache, slots, B, dev)
    handle, on = _launch(dev, stream)
    with on:
        status = _status(status, B, dev)
        rc = lib().sv_cache_keep(ctypes.byref(c), p_slots, p_count, int(absolute), B,
                                 status.data_ptr(), handle)
    _raise(rc, "sv_cache_keep")
    return status


def cache_fork(cache, src, dst, status=None, stream=None):
    """sv_cache_fork: slot dst[i] (empty, listed once) takes over the tokens of slot
    src[i] (no dst of this call), [n] int32 each (-1: none), sharing its pages.
    Returns status [n] int32: 0 or S_BAD_CACHE."""
    import torch

    dev = _device_of(src, "src")
    c = _cache_struct(cache, dev)
    n = src.numel()
    p_src = _want(src, "src", torch.int32, (n,), dev)
    p_dst = _want(dst, "dst", torch.int32, (n,), dev)
    handle, on = _launch(dev, stream)
    with on:
        status = _status(status, n, dev)
        rc = lib().sv_cache_fork(ctypes.byref(c), p_src, p_dst, n, status.data_ptr(), handle)
    _raise(rc, "sv_cache_fork")
    return status


def cache_compact(cache, used=None, moved=None, workspace=None, stream=None):
    """sv_cache_compact: moves the pages in use to the pool's front, the lists with
    them.  Returns used [1] int32, the pages in use.  moved: None, or [n_pages] int32
    for where each page went (-1: it was free)."""
    import torch

    dev = _device_of(cache.k, "cache.k")
    c = _cache_struct(cache, dev)
    p_moved = None if moved is None else _want(moved, "moved", torch.int32, (c.n_pages,), dev)
    handle, on = _launch(dev, stream)
    with on:
        if used is None:
            used = torch.empty(1, dtype=torch.int32, device=dev)
        else:
            _want(used, "used", torch.int32, (1,), dev)
        need = lib().sv_cache_workspace_bytes(ctypes.byref(c), 1)
        workspace, size = _bytes(workspace, need, "workspace", dev)
        rc = lib().sv_cache_compact(ctypes.byref(c), used.data_ptr(), p_moved,
                                    workspace.data_ptr(), size, handle)
    _raise(rc, "sv_cache_compact")
    return used


def _row_strides(t, name, shape, dtype, dev):
    """A tensor's address and strides, its last axis contiguous; strides of axes of one
    place do not count."""
    import torch

    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev.index
            and t.shape == shape):
        _check(t, name, dtype, shape, dev)
    if t.numel() == 0:
        return None, [0] * (len(shape) - 1)
    strides = [s if n > 1 else 0 for s, n in zip(t.stride(), shape)]
    if strides.pop() != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    address = t.data_ptr()
    for s in strides:
        address |= 2 * s
    if address % 16:
        raise ValueError(f"rows of {name} must begin at multiples of 16 bytes")
    return t.data_ptr(), strides


def cache_write(cache, layer, k, v, slots=None, rows=None, offsets=None, stream=None):
    """sv_cache_write: rows of keys and values into the pages of a layer, from position
    lens on (lengths stay, see cache_keep).  k, v [B, R, n_kv, head_dim] (slices of a
    wider projection will do), of which session b has rows[b] (None: R); or, with
    offsets [B + 1] int32, [N, n_kv, head_dim], session b's being offsets[b] ..
    offsets[b + 1] - 1.  Rows without pages that the session alone holds are
    skipped (cache_reserve's status tells)."""
    import torch

    dev = _device_of(k, "k")
    c = _cache_struct(cache, dev)
    p_rows = p_offsets = None
    if offsets is not None:
        if rows is not None:
            raise ValueError("give rows or offsets, not both")
        if k.dim() != 3:
            raise ValueError("k must be [N, n_kv, head_dim] with offsets")
        B, R = offsets.numel() - 1, _int32(k.shape[0], "k")
        p_offsets = _want(offsets, "offsets", torch.int32, (B + 1,), dev)
        shape = (R, c.n_kv, c.head_dim)
    else:
        if k.dim() != 4:
            raise ValueError("k must be [B, R, n_kv, head_dim] (or one line, with offsets)")
        B, R = k.shape[:2]
        shape = (B, R, c.n_kv, c.head_dim)
        if rows is not None:
            p_rows = _want(rows, "rows", torch.int32, (B,), dev)
    p_k, k_strides = _row_strides(k, "k", shape, cache.k.dtype, dev)
    p_v, v_strides = _row_strides(v, "v", shape, cache.k.dtype, dev)
    if offsets is not None:
        k_strides, v_strides = [0] + k_strides, [0] + v_strides
    p_slots = _cache_slots(cache, slots, B, dev)
    handle, on = _launch(dev, stream)
    with on:
        rc = lib().sv_cache_write(ctypes.byref(c), layer,
                                  ctypes.byref(_Rows(p_k, p_v, *k_strides, *v_strides)), p_slots,
                                  p_rows, p_offsets, B, R, handle)
    _raise(rc, "sv_cache_write")


def cache_plan(cache, n_heads, R, rows=None, slots=None, B=None, out=None, stream=None):
    """sv_cache_plan: how the attention of a round of up to R rows a session is split,
    for all layers, as long as the cache's lists and lengths, slots [B] int32 (None:
    slot b) and rows [B] int32 (None: R; B then tells how many) stay as they are.  Keys
    that neighbouring sessions share are read once for all of them.  out: a CachePlan
    of the same sizes to write again."""
    import torch

    dev = _device_of(cache.k, "cache.k")
    c = _cache_struct(cache, dev)
    given = rows if rows is not None else slots
    if given is not None:
        if B is not None and B != given.numel():
            raise ValueError("B does not go with rows or slots")
        B = given.numel()
    elif B is None:
        B = c.n_slots
    p_rows = None if rows is None else _want(rows, "rows", torch.int32, (B,), dev)
    p_slots = _cache_slots(cache, slots, B, dev)
    need = lib().sv_cache_plan_bytes(ctypes.byref(c), n_heads, B, R)
    handle, on = _launch(dev, stream)
    with on:
        if out is not None and (out.n_heads, out.B, out.R) != (n_heads, B, R):
            raise ValueError("out is a plan of other sizes")
        buffer, size = _bytes(None if out is None else out.buffer, need, "out.buffer", dev)
        status = _status(None if out is None else out.status, B, dev)
        rc = lib().sv_cache_plan(ctypes.byref(c), p_slots, p_rows, n_heads, B, R, status.data_ptr(),
                                 buffer.data_ptr(), size, handle)
    _raise(rc, "sv_cache_plan")
    return CachePlan(buffer, status, n_heads, B, R, c.n_kv, c.head_dim,
                     lib().sv_cache_attention_bytes(ctypes.byref(c), n_heads, B, R),
                     (c.page, c.n_slots, c.max_pages))


def cache_attention(cache, layer, q, plan, scale=None, out=None, workspace=None, stream=None):
    """sv_cache_attention: attention of a round's rows q [B, R, n_heads, head_dim] (a
    slice of a wider projection will do) over a layer of the cache, row r of a session
    over positions 0 .. lens + r; its own keys and values must be written.  scale:
    None for 1 / sqrt(head_dim).  out: None for a new tensor, or one like it.  Rows
    that a session does not use are not written, rows of a failed session become NaN."""
    import torch

    dev = _device_of(q, "q")
    c = _cache_struct(cache, dev)
    B, R, n_heads = plan.B, plan.R, plan.n_heads
    shape = (B, R, n_heads, c.head_dim)
    p_q, strides = _row_strides(q, "q", shape, cache.k.dtype, dev)
    scale = c.head_dim ** -0.5 if scale is None else float(scale)
    if (plan.n_kv, plan.head_dim) != (c.n_kv, c.head_dim):
        raise ValueError("plan is of a cache of other heads")
    if plan.lists is not None and plan.lists != (c.page, c.n_slots, c.max_pages):
        raise ValueError("plan is of a cache of other pages, slots or lists")
    p_plan = _want(plan.buffer, "plan.buffer", torch.uint8, plan.buffer.shape, dev)
    handle, on = _launch(dev, stream)
    with on:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
        else:
            _want(out, "out", q.dtype, shape, dev)
            lo = out.data_ptr()
            hi = lo + 2 * out.numel()
            if lo < p_q + 2 * (sum(s * (n - 1) for s, n in zip(strides, shape)) + c.head_dim) and p_q < hi:
                raise ValueError("out overlaps q")
            plane = 2 * cache.k.numel()
            if (lo < c.k + plane and c.k < hi) or (lo < c.v + plane and c.v < hi):
                raise ValueError("out overlaps the cache")
        workspace, size = _bytes(workspace, plan.workspace_bytes, "workspace", dev)
        rc = lib().sv_cache_attention(ctypes.byref(c), layer, p_q, *strides, scale, p_plan,
                                      n_heads, B, R, out.data_ptr(),
                                      workspace.data_ptr(), size, handle)
    _raise(rc, "sv_cache_attention")
    return out
