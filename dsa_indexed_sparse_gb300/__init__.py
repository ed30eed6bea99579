"""Python binding of libdsa (the GB300 DSA sparse-attention path).

Argument marshalling only: every step runs in the CUDA kernels behind the C ABI
declared in ``include/dsa.h``.  torch is used for device memory and streams.
There is no CPU fallback: importing this package raises if ``libdsa.so`` has
not been built (``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK = 0
STATUS_NAMES = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_WORKSPACE",
                4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT", 6: "DSA_ERR_DEVICE_CHECK"}
DSA_F32, DSA_BF16, DSA_E4M3, DSA_MXFP8_E4M3, DSA_E4M3_T128, DSA_E2M1, DSA_MXFP4_E2M1 = 0, 1, 2, 3, 4, 5, 6
E2M1_ROW_BYTES = 432                # a DSA_E2M1 latent row
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

EXPORTED = ("dsa_abi_version", "dsa_status_string", "dsa_last_error", "dsa_last_plan",
            "dsa_indexer_scores", "dsa_topk", "dsa_sparse_mla_attn_workspace_size",
            "dsa_sparse_mla_attn", "dsa_decode_workspace_size", "dsa_decode_step",
            "dsa_decode_step_static_ws", "dsa_index_cache_append", "dsa_index_cache_append_mx",
            "dsa_latent_cache_append", "dsa_debug_withhold_arrival",
            "dsa_indexer_prolog_workspace_size", "dsa_indexer_prolog",
            "dsa_rope_turns", "dsa_rope", "dsa_latent_cache_append_rope", "dsa_index_cache_append_rope",
            "dsa_latent_cache_read", "dsa_index_cache_append_mx4", "dsa_index_query_quantize", "dsa_index_cache_read",
            "dsa_block_topk", "dsa_block_mla_attn_workspace_size", "dsa_block_mla_attn",
            "dsa_block_decode_workspace_size", "dsa_block_decode_step", "dsa_check_status")
STATIC_WORKSPACE_BYTES = 32 << 20   # DSA_STATIC_WORKSPACE_BYTES


class SeqDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("max_ctx", ctypes.c_int32),
                ("q_per_seq", ctypes.c_int32), ("q_seq", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("cache_rows", ctypes.c_int64)]


class IndexerDesc(ctypes.Structure):
    _fields_ = [("H_I", ctypes.c_int32), ("D_I", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p)]


class MlaDesc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_latent", ctypes.c_int32), ("d_rope", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("q", ctypes.c_void_p), ("kv_cache", ctypes.c_void_p),
                ("row_bytes", ctypes.c_int64), ("softmax_scale", ctypes.c_float)]


class PrologDesc(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_q", ctypes.c_int32), ("H_I", ctypes.c_int32),
                ("D_I", ctypes.c_int32), ("x", ctypes.c_void_p), ("x_q", ctypes.c_void_p), ("w_q", ctypes.c_void_p),
                ("w_k", ctypes.c_void_p), ("w_w", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
                ("beta", ctypes.c_void_p)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("d_rot", ctypes.c_int32), ("layout", ctypes.c_int), ("turns", ctypes.c_void_p),
                ("magnitude", ctypes.c_float)]


class DSAError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first (__graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, C = ctypes.c_void_p, ctypes.c_int
    sig = {
        "dsa_abi_version": (C, []),
        "dsa_status_string": (ctypes.c_char_p, [C]),
        "dsa_last_error": (ctypes.c_char_p, []),
        "dsa_last_plan": (ctypes.c_char_p, []),
        "dsa_indexer_scores": (C, [P, P, P, ctypes.c_int64, P]),
        "dsa_topk": (C, [P, P, ctypes.c_int64, ctypes.c_int32, P, P]),
        "dsa_sparse_mla_attn_workspace_size": (ctypes.c_size_t, [P, P, ctypes.c_int32]),
        "dsa_sparse_mla_attn": (C, [P, P, P, ctypes.c_int32, P, P, P, ctypes.c_size_t, P]),
        "dsa_decode_workspace_size": (ctypes.c_size_t, [P, P, P, ctypes.c_int32]),
        "dsa_decode_step": (C, [P, P, P, ctypes.c_int32, P, P, P, P, ctypes.c_size_t, P]),
        "dsa_decode_step_static_ws": (C, [P, P, P, ctypes.c_int32, P, P, P, P]),
        "dsa_index_cache_append": (C, [P, ctypes.c_int32, C, P, P, P, P]),
        "dsa_index_cache_append_mx": (C, [P, ctypes.c_int32, C, P, P, P, P]),
        "dsa_latent_cache_append": (C, [P, P, P, P, P]),
        "dsa_debug_withhold_arrival": (C, [ctypes.c_int32, ctypes.c_uint64]),
        "dsa_indexer_prolog_workspace_size": (ctypes.c_size_t, [P, P]),
        "dsa_indexer_prolog": (C, [P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
        "dsa_rope_turns": (C, [ctypes.c_int32, ctypes.c_double, C, ctypes.c_double, ctypes.c_double,
                               ctypes.c_double, ctypes.c_double, P, P]),
        "dsa_rope": (C, [P, ctypes.c_int32, ctypes.c_int32, P, C, P, ctypes.c_int64, ctypes.c_int64, P,
                         ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, P]),
        "dsa_latent_cache_append_rope": (C, [P, P, P, P, ctypes.c_int64, P, ctypes.c_int64, P, P]),
        "dsa_index_cache_append_rope": (C, [P, P, ctypes.c_int32, ctypes.c_int32, C, C, P, ctypes.c_int64, P, P, P]),
        "dsa_latent_cache_read": (C, [P, P, P, C, P, ctypes.c_int64, P]),
        "dsa_index_cache_append_mx4": (C, [P, ctypes.c_int32, C, P, P, P, P]),
        "dsa_index_query_quantize": (C, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, C, C, P, ctypes.c_int64,
                                         ctypes.c_int64, P, P, P]),
        "dsa_index_cache_read": (C, [P, ctypes.c_int32, C, P, P, C, P, ctypes.c_int64, P]),
        "dsa_block_topk": (C, [P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P]),
        "dsa_block_mla_attn_workspace_size": (ctypes.c_size_t, [P, P, ctypes.c_int32]),
        "dsa_block_mla_attn": (C, [P, P, P, ctypes.c_int32, P, P, P, ctypes.c_size_t, P]),
        "dsa_block_decode_workspace_size": (ctypes.c_size_t, [P, P, ctypes.c_int32]),
        "dsa_block_decode_step": (C, [P, P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P, P,
                                      ctypes.c_size_t, P]),
        "dsa_check_status": (C, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load()


def abi_version() -> int:
    return _lib.dsa_abi_version()


def last_plan() -> str:
    return _lib.dsa_last_plan().decode()


def last_error() -> str:
    return _lib.dsa_last_error().decode()


def _check(status: int):
    if status != DSA_OK:
        raise DSAError(status, last_error())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdsa must be contiguous")
    return t.data_ptr()


# The current stream's handle without a Stream object around it: 0.1 us against 2.9, of
# the 3.4 that a small step's C call takes.
# Both are there in a torch with CUDA; one without still imports this module.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device   # once a CUDA tensor was seen
_FLOAT_CODES = {torch.float32: DSA_F32, torch.bfloat16: DSA_BF16}


def _stream(stream, dev: Optional[int] = None) -> int:
    if stream is None:
        return _raw_stream(torch.cuda.current_device() if dev is None else dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows(t: torch.Tensor, name: str, dev: int) -> int:
    """Data pointer of a tensor whose values are contiguous along its last dim, on GPU dev."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device, not on {t.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dim of {name} must be contiguous")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return DSA_E4M3
    if t.dtype == torch.float32:
        return DSA_F32
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _flat(dev: int, *tensors: torch.Tensor) -> None:
    """Refuses tensors that are not contiguous or not on GPU dev."""
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"the tensors of a call must be on the current CUDA device, not on {t.device}")
        if not t.is_contiguous():
            raise ValueError("tensors passed to libdsa must be contiguous")


def _cache_ptr(t: torch.Tensor, name: str, dev: int) -> int:
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdsa must be contiguous")
    return _rows(t, name, dev)


def _on_current(*records: "_CachedDesc") -> int:
    """The current GPU's index.  Refuses records with tensors off it (a descriptor holds their addresses)."""
    dev = records[0]._gpu
    if dev is None:
        dev = records[0].gpu()
    if dev >= 0 and dev == _current_device():
        for r in records:
            if r._gpu != dev and r.gpu() != dev:
                break
        else:
            return dev
    raise ValueError("the tensors of a call must be on the current CUDA device")


class _CachedDesc:
    """The C descriptor is built on first use and kept until a field is reassigned
    (a step call then costs no Python-side struct building).  Tensors are
    referenced by their data pointers, so resizing a tensor in place needs the
    field reassigned."""

    def __setattr__(self, name, value):
        if name != "_desc":
            object.__setattr__(self, "_desc", None)
            object.__setattr__(self, "_gpu", None)
        object.__setattr__(self, name, value)

    def gpu(self) -> int:
        """The index of the GPU that every tensor of the record is on, or -1."""
        g = self.__dict__.get("_gpu")
        if g is None:
            on = {v.get_device() for v in vars(self).values() if isinstance(v, torch.Tensor)}
            g = on.pop() if len(on) == 1 else -1
            object.__setattr__(self, "_gpu", g)
        return g

    def desc(self):
        d = self.__dict__.get("_desc")
        if d is None:
            d = self._build_desc()
            object.__setattr__(self, "_desc", d)
        return d


@dataclasses.dataclass
class Seq(_CachedDesc):
    """Queries and paging (device int32 tensors); see dsa_seq_desc_t."""
    q_seq: torch.Tensor
    q_pos: torch.Tensor
    block_table: torch.Tensor          # [B, bt_stride]
    max_ctx: int
    cache_rows: int
    page_size: int = 64
    q_per_seq: int = 0

    def _build_desc(self) -> SeqDesc:
        B, stride = self.block_table.shape
        return SeqDesc(B, self.q_seq.shape[0], self.max_ctx, self.q_per_seq, _ptr(self.q_seq),
                       _ptr(self.q_pos), _ptr(self.block_table), stride, self.page_size, self.cache_rows)


@dataclasses.dataclass
class Indexer(_CachedDesc):
    """Lightning-indexer inputs; see dsa_indexer_desc_t."""
    q: torch.Tensor                    # [T, H_I, D_I] e4m3 codes (uint8) or fp32; MXFP4: uint8 [T, H_I, D_I/2]
    w: torch.Tensor                    # [T, H_I] fp32
    k_cache: torch.Tensor              # [cache_rows, D_I]; MXFP4: uint8 [cache_rows, D_I/2]
    q_scale: Optional[torch.Tensor] = None   # fp32 [T, H_I], or uint8 E8M0 [T, H_I, D_I/32] (MXFP8, MXFP4)
    k_scale: Optional[torch.Tensor] = None   # fp32 [cache_rows], or uint8 E8M0 [cache_rows, D_I/32] (MXFP8, MXFP4)
    dtype: Optional[int] = None              # DSA_MXFP8_E4M3 or DSA_MXFP4_E2M1 for such codes; else from k_cache

    def _build_desc(self) -> IndexerDesc:
        _, H_I, D_I = self.q.shape
        dt = self.dtype if self.dtype is not None else _dtype_code(self.k_cache)
        if dt == DSA_MXFP4_E2M1:
            T, rows, D_I = self.q.shape[0], self.k_cache.shape[0], 2 * D_I
            want = ((self.q, (T, H_I, D_I // 2)), (self.q_scale, (T, H_I, D_I // 32)),
                    (self.k_cache, (rows, D_I // 2)), (self.k_scale, (rows, D_I // 32)))
            if any(t is None or t.dtype != torch.uint8 or t.shape != n for t, n in want):
                raise ValueError("MXFP4: q and k_cache must be uint8 [T, H_I, D_I/2] and [cache_rows, D_I/2], their "
                                 "scales uint8 [T, H_I, D_I/32] and [cache_rows, D_I/32]")
        return IndexerDesc(H_I, D_I, dt, _ptr(self.q), _ptr(self.q_scale),
                           _ptr(self.w), _ptr(self.k_cache), _ptr(self.k_scale))


@dataclasses.dataclass
class Mla(_CachedDesc):
    """Latent attention inputs; see dsa_mla_desc_t.  kv_cache is [cache_rows, row] of
    bf16/fp32 values, or uint8 656-byte FP8 or 432-byte 4-bit rows (dtype given explicitly
    then)."""
    q: torch.Tensor                    # [T, H, d_latent + d_rope]
    kv_cache: torch.Tensor
    d_latent: int
    d_rope: int
    softmax_scale: float
    dtype: Optional[int] = None

    def _build_desc(self) -> MlaDesc:
        dt = self.dtype if self.dtype is not None else _dtype_code(self.kv_cache)
        row_bytes = self.kv_cache.stride(0) * self.kv_cache.element_size()
        return MlaDesc(self.q.shape[1], self.d_latent, self.d_rope, dt, _ptr(self.q), _ptr(self.kv_cache),
                       row_bytes, self.softmax_scale)


@dataclasses.dataclass
class Prolog(_CachedDesc):
    """Indexer prolog inputs; see dsa_prolog_desc_t (bf16 tensors, weights as
    [output, input])."""
    x: torch.Tensor                    # [T, d_model] bf16
    x_q: torch.Tensor                  # [T, d_q] bf16
    w_q: torch.Tensor                  # [H_I * D_I, d_q] bf16
    w_k: torch.Tensor                  # [D_I, d_model] bf16
    w_w: torch.Tensor                  # [H_I, d_model] bf16
    gamma: torch.Tensor                # [D_I] fp32
    beta: torch.Tensor                 # [D_I] fp32

    def _build_desc(self) -> PrologDesc:
        return PrologDesc(self.x.shape[1], self.x_q.shape[1], self.w_w.shape[0], self.w_k.shape[0], _ptr(self.x),
                          _ptr(self.x_q), _ptr(self.w_q), _ptr(self.w_k), _ptr(self.w_w), _ptr(self.gamma),
                          _ptr(self.beta))


@dataclasses.dataclass
class Rope(_CachedDesc):
    """A rotation's frequencies, kept on the device; see dsa_rope_desc_t.  `make`
    computes them."""
    d_rot: int
    turns: torch.Tensor                # int64 [d_rot / 2]: turns per position in units of 2**-64 (unsigned)
    magnitude: float = 1.0
    layout: str = "interleaved"

    @classmethod
    def make(cls, d_rot: int, theta: float = 10000.0, layout: str = "interleaved", scaling: str = "none",
             factor: float = 1.0, original_ctx: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
             magnitude: Optional[float] = None, device="cuda") -> "Rope":
        """scaling: "none", "linear", "ntk" or "yarn" (with factor; "yarn" also
        original_ctx and the betas).  magnitude overrides the factor on cosine and
        sine (1, or YaRN's 0.1 ln(factor) + 1)."""
        if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
            raise ValueError(f"layout must be one of {list(ROPE_LAYOUTS)}, scaling one of {list(ROPE_SCALINGS)}")
        host = (ctypes.c_uint64 * (max(int(d_rot), 0) // 2))()
        mag = ctypes.c_float()
        _check(_lib.dsa_rope_turns(d_rot, theta, ROPE_SCALINGS[scaling], factor, original_ctx, beta_fast, beta_slow,
                                   host, ctypes.byref(mag)))
        turns = torch.frombuffer(host, dtype=torch.int64).to(device, copy=True)
        return cls(d_rot, turns, mag.value if magnitude is None else float(magnitude), layout)

    def _build_desc(self) -> RopeDesc:
        if self.turns.dtype != torch.int64 or self.turns.numel() != self.d_rot // 2:
            raise ValueError("turns must be int64 [d_rot / 2]")
        if not self.turns.is_contiguous():
            raise ValueError("turns must be contiguous")
        return RopeDesc(self.d_rot, ROPE_LAYOUTS[self.layout], self.turns.data_ptr(), self.magnitude)


def rope(plan: Rope, pos: torch.Tensor, x: torch.Tensor, out: torch.Tensor, inverse: bool = False,
         stream=None) -> torch.Tensor:
    """Rotates x [T, H, d_rot] (or [T, d_rot]; bf16 or fp32) by the positions pos
    (int32 [T]) into out, of the same shape and type.  Both may be strided views
    whose last dim is contiguous: q[..., 512:] rotates that part of a head.  out is
    x (in place) or shares no value with it.  inverse: the transposed matrix -- the
    gradient of the rotation."""
    d = plan.desc()
    shape, xs, os_ = x.shape, x.stride(), out.stride()
    n = len(shape)
    if n not in (2, 3) or shape[-1] != d.d_rot or out.shape != shape:
        raise ValueError("x and out must be [T, H, d_rot] or [T, d_rot]")
    if xs[-1] != 1 or os_[-1] != 1:
        raise ValueError("the last dim of x and out must be contiguous")
    dtype = _FLOAT_CODES.get(x.dtype)
    if dtype is None or out.dtype != x.dtype:
        raise ValueError("x and out must both be bfloat16 or float32")
    T = shape[0]
    if pos.dtype != torch.int32 or pos.dim() != 1 or pos.numel() != T or not pos.is_contiguous():
        raise ValueError("pos must be contiguous int32 [T]")
    dev = _on_current(plan)
    if pos.get_device() != dev or x.get_device() != dev or out.get_device() != dev:
        raise ValueError("pos, x and out must be on the current CUDA device")
    H, xh, oh = (shape[1], xs[1], os_[1]) if n == 3 else (1, 0, 0)
    _check(_lib.dsa_rope(ctypes.byref(d), T, H, pos.data_ptr(), dtype, x.data_ptr(), xs[0], xh, out.data_ptr(),
                         os_[0], oh, 1 if inverse else 0, _stream(stream, dev)))
    return out


def indexer_prolog_workspace_size(seq: Seq, pro: Prolog) -> int:
    s, d = seq.desc(), pro.desc()
    return _lib.dsa_indexer_prolog_workspace_size(ctypes.byref(s), ctypes.byref(d))


def indexer_prolog(seq: Seq, pro: Prolog, q_codes: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor,
                   k_cache: torch.Tensor, k_scale: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """The indexer's query (E4M3 codes + per-head scales), head weights and the new
    tokens' normalised keys (quantised into k_cache / k_scale at their positions)."""
    s, d = seq.desc(), pro.desc()
    _check(_lib.dsa_indexer_prolog(ctypes.byref(s), ctypes.byref(d), _ptr(q_codes), _ptr(q_scale), _ptr(w),
                                   _ptr(k_cache), _ptr(k_scale), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)))


def indexer_scores(seq: Seq, idx: Indexer, scores: torch.Tensor, stream=None) -> torch.Tensor:
    s, x = seq.desc(), idx.desc()
    _check(_lib.dsa_indexer_scores(ctypes.byref(s), ctypes.byref(x), _ptr(scores), scores.stride(0),
                                   _stream(stream)))
    return scores


def topk(seq: Seq, scores: torch.Tensor, K: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    s = seq.desc()
    _check(_lib.dsa_topk(ctypes.byref(s), _ptr(scores), scores.stride(0), K, _ptr(out), _stream(stream)))
    return out


def sparse_mla_attn_workspace_size(seq: Seq, mla: Mla, K: int) -> int:
    s, m = seq.desc(), mla.desc()
    return _lib.dsa_sparse_mla_attn_workspace_size(ctypes.byref(s), ctypes.byref(m), K)


def sparse_mla_attn(seq: Seq, mla: Mla, idx: torch.Tensor, K: int, out: torch.Tensor,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    s, m = seq.desc(), mla.desc()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.dsa_sparse_mla_attn(ctypes.byref(s), ctypes.byref(m), _ptr(idx), K, _ptr(out), _ptr(lse),
                                    _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def decode_workspace_size(seq: Seq, idx: Indexer, mla: Mla, K: int) -> int:
    s, x, m = seq.desc(), idx.desc(), mla.desc()
    return _lib.dsa_decode_workspace_size(ctypes.byref(s), ctypes.byref(x), ctypes.byref(m), K)


def decode_step(seq: Seq, idx: Indexer, mla: Mla, K: int, out: torch.Tensor, workspace: torch.Tensor,
                lse: Optional[torch.Tensor] = None, idx_out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    s, x, m = seq.desc(), idx.desc(), mla.desc()
    _check(_lib.dsa_decode_step(ctypes.byref(s), ctypes.byref(x), ctypes.byref(m), K, _ptr(out), _ptr(lse),
                                _ptr(idx_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)))
    return out


def decode_step_static_ws(seq: Seq, idx: Indexer, mla: Mla, K: int, out: torch.Tensor,
                          lse: Optional[torch.Tensor] = None, idx_out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """decode_step with the scratch in the library's own device array (no workspace
    argument, nothing allocated) -- for callers that cannot allocate device memory.
    Calls overlapping on the GPU race on that shared array."""
    s, x, m = seq.desc(), idx.desc(), mla.desc()
    _check(_lib.dsa_decode_step_static_ws(ctypes.byref(s), ctypes.byref(x), ctypes.byref(m), K, _ptr(out),
                                          _ptr(lse), _ptr(idx_out), _stream(stream)))
    return out


def _codes_check(dtype: int, D: int, rows: int, codes: torch.Tensor, scale: Optional[torch.Tensor], names: str) -> None:
    """Codes and scales of at least `rows` index vectors of D values in the format dtype."""
    if dtype == DSA_MXFP4_E2M1:
        per, size, scales = D // 2, 1, rows * (D // 32)
    elif dtype == DSA_MXFP8_E4M3:
        per, size, scales = D, 1, rows * (D // 32)
    elif dtype == DSA_E4M3:
        per, size, scales = D, 4, rows
    else:
        raise ValueError("dtype must be DSA_E4M3, DSA_MXFP8_E4M3 or DSA_MXFP4_E2M1")
    if codes.element_size() != 1 or codes.numel() < rows * per:
        raise ValueError(f"{names}: codes must be one-byte [{rows}, {per}]")
    if scale is None:
        if size == 1:
            raise ValueError(f"{names}: scales are required")
    elif scale.element_size() != size or scale.numel() < scales:
        raise ValueError(f"{names}: scales must be fp32 [{rows}] (DSA_E4M3) or uint8 [{rows}, D_I / 32]")


def _dense(t: torch.Tensor, name: str, dev: int, dtype: torch.dtype, shape) -> int:
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}")
    _flat(dev, t)
    return t.data_ptr()


def _outputs(s: SeqDesc, m: MlaDesc, out: torch.Tensor, lse: Optional[torch.Tensor], dev: int):
    """Pointers of an attention's out [T, H, d_latent] and lse [T, H] (or None)."""
    T, H = s.T, m.H
    o = _dense(out, "out", dev, torch.float32 if m.dtype == DSA_F32 else torch.bfloat16, (T, H, m.d_latent))
    return o, None if lse is None else _dense(lse, "lse", dev, torch.float32, (T, H))


def _scratch(workspace: Optional[torch.Tensor], dev: int):
    if workspace is None:
        return None, 0
    _flat(dev, workspace)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def block_topk(seq: Seq, scores: torch.Tensor, n_blocks: int, out: torch.Tensor, first: int = 1, last: int = 1,
               stream=None) -> torch.Tensor:
    """The n_blocks blocks (pages) of each query with the best score in each (scores:
    fp32 [T, ld], of indexer_scores), the `first` first and `last` last ones always
    among them: out int32 [T, n_blocks], ascending, -1 behind them."""
    s = seq.desc()
    T, shape = s.T, scores.shape
    if len(shape) != 2 or scores.dtype != torch.float32 or shape[0] != T:
        raise ValueError("scores must be float32 [T, ld]")
    dev = _on_current(seq)
    if out.dtype != torch.int32 or out.shape != (T, n_blocks):
        raise ValueError("out must be int32 [T, n_blocks]")
    _flat(dev, scores, out)
    _check(_lib.dsa_block_topk(ctypes.byref(s), scores.data_ptr(), shape[1], n_blocks, first, last, out.data_ptr(),
                               _stream(stream, dev)))
    return out


def block_mla_attn_workspace_size(seq: Seq, mla: Mla, n_blocks: int) -> int:
    s, m = seq.desc(), mla.desc()
    return _lib.dsa_block_mla_attn_workspace_size(ctypes.byref(s), ctypes.byref(m), n_blocks)


def block_mla_attn(seq: Seq, mla: Mla, block_idx: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sparse_mla_attn over whole blocks: block_idx int32 [T, n_blocks] names pages of
    each query's sequence (-1: none), of which the positions up to the query's own count."""
    s, m = seq.desc(), mla.desc()
    if block_idx.dim() != 2:
        raise ValueError("block_idx must be int32 [T, n_blocks]")
    dev = _on_current(seq, mla)
    o, l = _outputs(s, m, out, lse, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    n = block_idx.shape[1]
    _check(_lib.dsa_block_mla_attn(ctypes.byref(s), ctypes.byref(m), _dense(block_idx, "block_idx", dev, torch.int32, (s.T, n)),
                                   n, o, l, ws, ws_bytes, _stream(stream, dev)))
    return out


def block_decode_workspace_size(seq: Seq, mla: Mla, n_blocks: int) -> int:
    s, m = seq.desc(), mla.desc()
    return _lib.dsa_block_decode_workspace_size(ctypes.byref(s), ctypes.byref(m), n_blocks)


def block_decode_step(seq: Seq, idx: Indexer, mla: Mla, n_blocks: int, out: torch.Tensor, workspace: torch.Tensor,
                      first: int = 1, last: int = 1, lse: Optional[torch.Tensor] = None,
                      block_idx_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """indexer_scores, block_topk and block_mla_attn in one call (scratch:
    block_decode_workspace_size bytes)."""
    s, x, m = seq.desc(), idx.desc(), mla.desc()
    dev = _on_current(seq, idx, mla)
    o, l = _outputs(s, m, out, lse, dev)
    sel = None if block_idx_out is None else _dense(block_idx_out, "block_idx_out", dev, torch.int32, (s.T, n_blocks))
    ws, ws_bytes = _scratch(workspace, dev)
    _check(_lib.dsa_block_decode_step(ctypes.byref(s), ctypes.byref(x), ctypes.byref(m), n_blocks, first, last, o, l, sel, ws,
                                      ws_bytes, _stream(stream, dev)))
    return out


def index_cache_append(seq: Seq, k_new: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
                       stream=None, mx: bool = False, dtype: Optional[int] = None) -> None:
    """Quantises the new tokens' index keys k_new [T, D_I] (fp32 or bf16) to e4m3
    + per-token fp32 scale (k_scale [cache_rows]), or with mx to MXFP8 (k_scale
    uint8 [cache_rows, D_I / 32] E8M0 bytes), and writes them at their
    positions' cache rows.  dtype (DSA_E4M3, DSA_MXFP8_E4M3 or DSA_MXFP4_E2M1:
    k_cache uint8 [cache_rows, D_I / 2]) names the format instead of mx."""
    s = seq.desc()
    if dtype == DSA_MXFP4_E2M1:
        shape, src = k_new.shape, _FLOAT_CODES.get(k_new.dtype)
        if len(shape) != 2 or shape[0] != s.T or src is None:
            raise ValueError("k_new must be float32 or bfloat16 [T, D_I]")
        D = shape[1]
        _codes_check(dtype, D, s.cache_rows, k_cache, k_scale, "k_cache, k_scale")
        dev = _on_current(seq)
        _flat(dev, k_new, k_cache, k_scale)
        _check(_lib.dsa_index_cache_append_mx4(ctypes.byref(s), D, src, k_new.data_ptr(), k_cache.data_ptr(),
                                               k_scale.data_ptr(), _stream(stream, dev)))
        return
    if dtype not in (None, DSA_E4M3, DSA_MXFP8_E4M3):
        raise ValueError("dtype must be DSA_E4M3, DSA_MXFP8_E4M3 or DSA_MXFP4_E2M1")
    fn = _lib.dsa_index_cache_append_mx if (mx if dtype is None else dtype == DSA_MXFP8_E4M3) else _lib.dsa_index_cache_append
    _check(fn(ctypes.byref(s), k_new.shape[1], _dtype_code(k_new), _ptr(k_new), _ptr(k_cache), _ptr(k_scale),
              _stream(stream)))


def index_query_quantize(q: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor, dtype: int = DSA_E4M3,
                         stream=None) -> None:
    """Query heads q [T, H_I, D_I] (fp32 or bf16; a strided view whose last dim is
    contiguous is fine) to the codes and scales that Indexer takes as q and q_scale:
    codes uint8 [T, H_I, D_I] ([T, H_I, D_I / 2] for DSA_MXFP4_E2M1), scale fp32
    [T, H_I] (DSA_E4M3) or uint8 [T, H_I, D_I / 32]."""
    shape, src = q.shape, _FLOAT_CODES.get(q.dtype)
    if len(shape) != 3 or src is None:
        raise ValueError("q must be float32 or bfloat16 [T, H_I, D_I]")
    if scale is None:
        raise ValueError("scale is required")
    T, H, D = shape
    _codes_check(dtype, D, T * H, codes, scale, "codes, scale")
    st, sh, last = q.stride()
    if last != 1 and D > 1:
        raise ValueError("the last dim of q must be contiguous")
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError("q must be on the current CUDA device")
    _flat(dev, codes, scale)
    _check(_lib.dsa_index_query_quantize(T, H, D, src, dtype, q.data_ptr(), st, sh, codes.data_ptr(), scale.data_ptr(),
                                         _stream(stream, dev)))


def index_cache_read(seq: Seq, k_cache: torch.Tensor, k_scale: Optional[torch.Tensor], out: torch.Tensor,
                     dtype: int = DSA_E4M3, stream=None) -> torch.Tensor:
    """The cached index keys of the positions of seq (q_seq, q_pos) as the values they
    stand for: out [T, D_I], bf16 or fp32 (a row-strided view is fine)."""
    s = seq.desc()
    shape, kind = out.shape, _FLOAT_CODES.get(out.dtype)
    if len(shape) != 2 or shape[0] != s.T or kind is None:
        raise ValueError("out must be float32 or bfloat16 [T, D_I]")
    D = shape[1]
    _codes_check(dtype, D, s.cache_rows, k_cache, k_scale, "k_cache, k_scale")
    stride, last = out.stride()
    if last != 1 and D > 1:
        raise ValueError("the last dim of out must be contiguous")
    dev = _on_current(seq)
    if out.get_device() != dev:
        raise ValueError("out must be on the current CUDA device")
    _flat(dev, k_cache)
    scale = None
    if k_scale is not None:
        _flat(dev, k_scale)
        scale = k_scale.data_ptr()
    _check(_lib.dsa_index_cache_read(ctypes.byref(s), D, dtype, k_cache.data_ptr(), scale, kind, out.data_ptr(), stride,
                                     _stream(stream, dev)))
    return out


def latent_cache_append(seq: Seq, mla: Mla, kv_new: torch.Tensor, stream=None) -> None:
    """Writes the new tokens' latent rows kv_new [T, d_latent + d_rope] into
    mla.kv_cache (copied, or quantised into 656-byte FP8 or 432-byte 4-bit rows)."""
    s, m = seq.desc(), mla.desc()
    _check(_lib.dsa_latent_cache_append(ctypes.byref(s), ctypes.byref(m), _ptr(kv_new), _ptr(mla.kv_cache),
                                        _stream(stream)))


def latent_cache_append_rope(seq: Seq, mla: Mla, plan: Rope, latent: torch.Tensor, k_rope: torch.Tensor,
                             stream=None) -> None:
    """Writes the new tokens' latent rows latent [T, d_latent] and k_rope
    [T, d_rope] (bf16, or fp32 for an fp32 cache; row-strided views are fine) into
    mla.kv_cache, with k_rope rotated by the tokens' positions on the way."""
    s, m, r = seq.desc(), mla.desc(), plan.desc()
    want = torch.float32 if m.dtype == DSA_F32 else torch.bfloat16
    if latent.dtype != want or k_rope.dtype != want:
        raise ValueError(f"latent and k_rope must be {want} for this cache")
    T = s.T
    if latent.shape != (T, m.d_latent) or k_rope.shape != (T, m.d_rope):
        raise ValueError("latent must be [T, d_latent] and k_rope [T, d_rope]")
    (lt, l1), (kt, k1) = latent.stride(), k_rope.stride()
    if l1 != 1 or k1 != 1:
        raise ValueError("the last dim of latent and k_rope must be contiguous")
    dev = _on_current(seq, mla, plan)
    if latent.get_device() != dev or k_rope.get_device() != dev:
        raise ValueError("latent and k_rope must be on the current CUDA device")
    _check(_lib.dsa_latent_cache_append_rope(ctypes.byref(s), ctypes.byref(m), ctypes.byref(r), latent.data_ptr(), lt,
                                             k_rope.data_ptr(), kt, m.kv_cache, _stream(stream, dev)))


def index_cache_append_rope(seq: Seq, plan: Rope, k_new: torch.Tensor, k_cache: torch.Tensor, k_scale: torch.Tensor,
                            offset: int = 0, stream=None, mx: bool = False, dtype: Optional[int] = None) -> None:
    """index_cache_append with dims [offset, offset + d_rot) of every new key
    rotated by the token's position before it is quantised (k_new may be a
    row-strided view)."""
    s, r = seq.desc(), plan.desc()
    if k_new.dim() != 2 or k_new.shape[0] != s.T:
        raise ValueError("k_new must be [T, D_I]")
    D = k_new.shape[1]
    fmt = (DSA_MXFP8_E4M3 if mx else DSA_E4M3) if dtype is None else dtype
    per = D // 2 if fmt == DSA_MXFP4_E2M1 else D
    if k_cache.element_size() != 1 or k_cache.numel() < s.cache_rows * per:
        raise ValueError("k_cache must be one-byte codes [cache_rows, D_I] (MXFP4: [cache_rows, D_I / 2])")
    blocks = fmt != DSA_E4M3
    if k_scale.element_size() != (1 if blocks else 4) or k_scale.numel() < s.cache_rows * (D // 32 if blocks else 1):
        raise ValueError("k_scale must be fp32 [cache_rows], or with mx uint8 [cache_rows, D_I / 32]")
    dev = _on_current(seq, plan)
    _check(_lib.dsa_index_cache_append_rope(ctypes.byref(s), ctypes.byref(r), D, offset,
                                            _dtype_code(k_new), fmt,
                                            _rows(k_new, "k_new", dev), k_new.stride(0),
                                            _cache_ptr(k_cache, "k_cache", dev), _cache_ptr(k_scale, "k_scale", dev),
                                            _stream(stream, dev)))


def latent_cache_read(seq: Seq, mla: Mla, out: torch.Tensor, stream=None) -> torch.Tensor:
    """The latent rows of the positions of seq (q_seq, q_pos) in mla.kv_cache as the
    values they stand for: out [T, d_latent + d_rope], bf16 or fp32 (a row-strided
    view is fine)."""
    s, m = seq.desc(), mla.desc()
    if out.shape != (s.T, m.d_latent + m.d_rope):
        raise ValueError("out must be [T, d_latent + d_rope]")
    dtype = _FLOAT_CODES.get(out.dtype)
    if dtype is None:
        raise ValueError("out must be bfloat16 or float32")
    stride, last = out.stride()
    if last != 1:
        raise ValueError("the last dim of out must be contiguous")
    dev = _on_current(seq, mla)
    if out.get_device() != dev:
        raise ValueError("out must be on the current CUDA device")
    _check(_lib.dsa_latent_cache_read(ctypes.byref(s), ctypes.byref(m), m.kv_cache, dtype, out.data_ptr(), stride,
                                      _stream(stream, dev)))
    return out


def debug_withhold_arrival(enable: bool, wait_limit_ns: int = 2_000_000) -> None:
    """Testing aid of the failure-detection path: while enabled, tensor-core
    attention launches have one producer warp withhold an arrival so a bounded
    wait runs out (after wait_limit_ns) and check_status() raises DSA_ERR_TIMEOUT."""
    _check(_lib.dsa_debug_withhold_arrival(1 if enable else 0, int(wait_limit_ns)))


def check_status(stream=None) -> None:
    """Synchronises the stream and raises DSAError if a device-side check fired."""
    _check(_lib.dsa_check_status(_stream(stream)))
