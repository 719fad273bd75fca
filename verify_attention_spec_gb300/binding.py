"""Thin ctypes binding over libvas.so (declared in include/vas.h).

Argument marshalling only: torch tensors become device pointers and sizes, the current
torch stream becomes the cudaStream_t, and a non-zero status becomes a ``VasError``.
Every step of the computation runs in the library's CUDA kernels.  Importing this
module raises ``ImportError`` when the library has not been built; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvas.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m verify_attention_spec_gb300._build` "
        "(or __graft_entry__.build()); this package has no CPU fallback")

_lib = ctypes.CDLL(LIB_PATH)

# status codes and device error bits (include/vas.h)
VAS_OK = 0
VAS_E_INVALID_ARG = -1
VAS_E_UNSUPPORTED = -2
VAS_E_WORKSPACE = -3
VAS_E_CUDA = -4
VAS_E_NOMEM = -5
VAS_E_NOT_FOUND = -6
VAS_E_EXISTS = -7
VAS_DEV_BAD_PAGE = 0x1
VAS_DEV_BAD_LENGTHS = 0x2
VAS_DEV_BAD_TOKEN = 0x4
VAS_DEV_EMPTY_ROW = 0x8
VAS_DEV_TIMEOUT = 0x10
VAS_DEV_BAD_TREE = 0x20
VAS_DEV_BAD_POSITION = 0x40
VAS_DEV_RESIDUAL_FALLBACK = 0x100
VAS_F32 = 0
VAS_BF16 = 1
VAS_FP8_E4M3 = 2
VAS_INT8 = 3
VAS_SHARE_AUTO = 0
VAS_SHARE_ALWAYS = 1

_c_void_p, _i32, _i64, _u32, _u64, _f32, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                  ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float,
                                                  ctypes.c_size_t)


class vas_attn_dims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("total_q_tokens", _i32), ("num_q_heads", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("max_pages_per_seq", _i32), ("kv_dtype", _i32),
                ("scale", _f32)]


class vas_append_dims(ctypes.Structure):
    _fields_ = [("num_seqs", _i32), ("total_tokens", _i32), ("num_q_heads", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("max_pages_per_seq", _i32), ("kv_dtype", _i32),
                ("rotary_dim", _i32), ("interleaved", _i32), ("max_position", _i32),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("eps", _f32)]


class vas_pool_dims(ctypes.Structure):
    _fields_ = [("num_layers", _i32), ("num_pages", _i32), ("page_size", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("kv_dtype", _i32)]


_P_dims = ctypes.POINTER(vas_attn_dims)
_P_append = ctypes.POINTER(vas_append_dims)
_P_pool = ctypes.POINTER(vas_pool_dims)
_sig = {
    "paged_attn_workspace_size": ([_P_dims], _sz),
    "paged_attn_workspace_min": ([_P_dims], _sz),
    "paged_attn_fwd": ([_c_void_p] * 8 + [_P_dims, _c_void_p, _sz, _c_void_p], ctypes.c_int),
    "paged_attn_fwd_tree": ([_c_void_p] * 9 + [_P_dims, _c_void_p, _sz, _c_void_p], ctypes.c_int),
    "paged_attn_fwd_quant": ([_c_void_p] * 11 + [_P_dims, _c_void_p, _sz, _c_void_p], ctypes.c_int),
    "paged_attn_fwd_prefix": ([_c_void_p] * 13 + [_P_dims, _i32, _i32, _c_void_p, _sz, _c_void_p],
                              ctypes.c_int),
    "paged_attn_prefix_workspace_size": ([_P_dims, _i32], _sz),
    "paged_attn_prefix_workspace_min": ([_P_dims, _i32], _sz),
    "paged_kv_append": ([_c_void_p] * 15 + [_P_append, _c_void_p], ctypes.c_int),
    "paged_kv_copy": ([_c_void_p] * 7 + [_i32, _P_pool, _c_void_p], ctypes.c_int),
    "paged_kv_keep_path": ([_c_void_p] * 7 + [_i32, _i32] + [_c_void_p] * 3 +
                           [_i32, _i32, _P_pool, _c_void_p], ctypes.c_int),
    "spec_verify": ([_c_void_p, _c_void_p, _c_void_p, _u64, _c_void_p, _c_void_p, _i32, _i32, _i32,
                     _c_void_p], ctypes.c_int),
    "spec_verify_tree": ([_c_void_p] * 4 + [_u64] + [_c_void_p] * 3 + [_i32, _i32, _i32, _c_void_p],
                         ctypes.c_int),
    "vas_last_device_error": ([ctypes.POINTER(_i32), _c_void_p], ctypes.c_int),
    "vas_philox4x32_10": ([_c_void_p, _u32, _u32, _c_void_p, _i64, _c_void_p], ctypes.c_int),
    "vas_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "vas_pool_create": ([_i32, _i32, _u64], _c_void_p),
    "vas_pool_destroy": ([_c_void_p], None),
    "vas_pool_free_pages": ([_c_void_p], _i32),
    "vas_pool_num_seqs": ([_c_void_p], _i32),
    "vas_pool_can_allocate": ([_c_void_p, _i32], ctypes.c_int),
    "vas_seq_pages_needed": ([_c_void_p, _i64, _i32], _i32),
    "vas_seq_len": ([_c_void_p, _i64], _i32),
    "vas_seq_admit": ([_c_void_p, _i64, _i32], ctypes.c_int),
    "vas_seq_grow": ([_c_void_p, _i64, _i32], ctypes.c_int),
    "vas_seq_rollback": ([_c_void_p, _i64, _i32], ctypes.c_int),
    "vas_seq_free": ([_c_void_p, _i64], ctypes.c_int),
    "vas_pool_preempt_newest": ([_c_void_p, ctypes.POINTER(_i64)], ctypes.c_int),
    "vas_seq_fork": ([_c_void_p, _i64, _i64, _i32], ctypes.c_int),
    "vas_seq_fork_tail": ([_c_void_p, _i64, _i64, _i32, ctypes.POINTER(_i32),
                           ctypes.POINTER(_i32)], _i32),
    "vas_pool_compact": ([_c_void_p, _c_void_p, _c_void_p, _i32], _i32),
    "vas_build_prefix_groups": ([_c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p], _i32),
    "vas_page_refcount": ([_c_void_p, _i32], _i32),
    "vas_build_block_table": ([_c_void_p, _c_void_p, _i32, _c_void_p, _i32, _c_void_p], ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class VasError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_lib.vas_status_string(status).decode()} ({status})")


def _check(fn: str, status: int) -> None:
    if status != VAS_OK:
        raise VasError(fn, status)


def _stream_ptr(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> ctypes.c_void_p:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


_KV_CODES = {torch.bfloat16: VAS_BF16, torch.float32: VAS_F32}


_QUANT_CODES = {"fp8": VAS_FP8_E4M3, "int8": VAS_INT8}
_SHARE_CODES = {"auto": VAS_SHARE_AUTO, "always": VAS_SHARE_ALWAYS}


def attn_dims(q: torch.Tensor, k_pages: torch.Tensor, block_table: torch.Tensor,
              seq_lens: torch.Tensor, scale: float = 0.0, quant: Optional[str] = None) -> vas_attn_dims:
    """vas_attn_dims from tensor shapes: q [T, Hq, D], k_pages [num_pages, P, Hkv, D],
    block_table [B, max_pages], seq_lens [B].  quant: None (k_pages share q's dtype), or
    "fp8" / "int8" for a pool of 8-bit codes (uint8 tensors) with a bf16 q."""
    T, Hq, D = q.shape
    num_pages, P, Hkv, D2 = k_pages.shape
    if D2 != D:
        raise ValueError("head_dim of q and k_pages differ")
    if quant is not None:
        if quant not in _QUANT_CODES or q.dtype != torch.bfloat16 or k_pages.dtype != torch.uint8:
            raise ValueError("a quantised pool is uint8 codes with a bf16 q")
        code = _QUANT_CODES[quant]
    else:
        if q.dtype not in _KV_CODES or k_pages.dtype != q.dtype:
            raise ValueError("q and k_pages must share a dtype in {bf16, fp32}")
        code = _KV_CODES[q.dtype]
    return vas_attn_dims(num_seqs=int(seq_lens.shape[0]), total_q_tokens=int(T), num_q_heads=int(Hq),
                         num_kv_heads=int(Hkv), head_dim=int(D), page_size=int(P),
                         num_pages=int(num_pages), max_pages_per_seq=int(block_table.shape[1]),
                         kv_dtype=code, scale=float(scale))


def paged_attn_workspace_size(dims: vas_attn_dims) -> int:
    return int(_lib.paged_attn_workspace_size(ctypes.byref(dims)))


def paged_attn_workspace_min(dims: vas_attn_dims) -> int:
    return int(_lib.paged_attn_workspace_min(ctypes.byref(dims)))


def alloc_workspace(dims: vas_attn_dims, device=None, nbytes: Optional[int] = None) -> torch.Tensor:
    n = paged_attn_workspace_size(dims) if nbytes is None else int(nbytes)
    if n <= 0:
        raise ValueError("invalid attention dims")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def paged_attn_fwd(q, k_pages, v_pages, block_table, seq_lens, query_lens, out, lse, workspace,
                   *, scale: float = 0.0, dims: Optional[vas_attn_dims] = None, stream=None) -> None:
    """Paged decode/verify attention (include/vas.h: paged_attn_fwd).  All tensors on the
    same CUDA device; out [T, Hq, D] (dtype of q) and lse fp32 [T, Hq] are written."""
    if dims is None:
        dims = attn_dims(q, k_pages, block_table, seq_lens, scale)
    st = _lib.paged_attn_fwd(
        _dev(q, "q"), _dev(k_pages, "k_pages", q.dtype), _dev(v_pages, "v_pages", q.dtype),
        _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        _dev(query_lens, "query_lens", torch.int32), _dev(out, "out", q.dtype),
        _dev(lse, "lse", torch.float32), ctypes.byref(dims), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check("paged_attn_fwd", st)


def paged_attn_fwd_tree(q, k_pages, v_pages, block_table, seq_lens, query_lens, tree_mask, out,
                        lse, workspace, *, scale: float = 0.0, dims: Optional[vas_attn_dims] = None,
                        stream=None) -> None:
    """Draft-tree attention (include/vas.h: paged_attn_fwd_tree).  tree_mask [T] int64 (the
    bits of a uint64 per query token: its ancestors among its sequence's draft tokens)."""
    if dims is None:
        dims = attn_dims(q, k_pages, block_table, seq_lens, scale)
    if tree_mask.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise ValueError("tree_mask must be a 64-bit integer tensor")
    if tree_mask.numel() != q.shape[0]:
        raise ValueError("tree_mask needs one word per query token")
    st = _lib.paged_attn_fwd_tree(
        _dev(q, "q"), _dev(k_pages, "k_pages", q.dtype), _dev(v_pages, "v_pages", q.dtype),
        _dev(block_table, "block_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        _dev(query_lens, "query_lens", torch.int32), _dev(tree_mask, "tree_mask"),
        _dev(out, "out", q.dtype), _dev(lse, "lse", torch.float32), ctypes.byref(dims),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check("paged_attn_fwd_tree", st)


def paged_attn_fwd_quant(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, query_lens,
                         out, lse, workspace, *, quant: str, tree_mask=None, scale: float = 0.0,
                         dims: Optional[vas_attn_dims] = None, stream=None) -> None:
    """Attention over a quantised pool (include/vas.h: paged_attn_fwd_quant).  k_pages /
    v_pages uint8 codes [num_pages, P, Hkv, D] ("fp8" E4M3 or "int8"); k_scale / v_scale
    fp32 [num_pages, Hkv, P]; q and out bf16; tree_mask as for paged_attn_fwd_tree or None."""
    if dims is None:
        dims = attn_dims(q, k_pages, block_table, seq_lens, scale, quant=quant)
    tm = ctypes.c_void_p(0)
    if tree_mask is not None:
        if tree_mask.numel() != q.shape[0]:
            raise ValueError("tree_mask needs one word per query token")
        tm = _dev(tree_mask, "tree_mask")
    st = _lib.paged_attn_fwd_quant(
        _dev(q, "q", torch.bfloat16), _dev(k_pages, "k_pages", torch.uint8),
        _dev(v_pages, "v_pages", torch.uint8), _dev(k_scale, "k_scale", torch.float32),
        _dev(v_scale, "v_scale", torch.float32), _dev(block_table, "block_table", torch.int32),
        _dev(seq_lens, "seq_lens", torch.int32), _dev(query_lens, "query_lens", torch.int32), tm,
        _dev(out, "out", torch.bfloat16), _dev(lse, "lse", torch.float32), ctypes.byref(dims),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check("paged_attn_fwd_quant", st)


def _here(dev: int, t: Optional[torch.Tensor], name: str, shape=None, dtype=None):
    """The address of a contiguous tensor on device `dev` (None: a null pointer)."""
    if t is None:
        return None
    if (t.get_device() == dev and (shape is None or t.shape == shape) and
            (dtype is None or t.dtype is dtype) and t.is_contiguous()):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


# The current stream as an address, without the Stream object around it (1 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_address(dev: int, stream: Optional[torch.cuda.Stream]) -> int:
    """The cudaStream_t of `stream`, or of the current stream of device `dev`."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def paged_attn_prefix_workspace_size(dims: vas_attn_dims, num_groups: int) -> int:
    return int(_lib.paged_attn_prefix_workspace_size(ctypes.byref(dims), num_groups))


def paged_attn_prefix_workspace_min(dims: vas_attn_dims, num_groups: int) -> int:
    return int(_lib.paged_attn_prefix_workspace_min(ctypes.byref(dims), num_groups))


def alloc_prefix_workspace(dims: vas_attn_dims, num_groups: int, device=None,
                           nbytes: Optional[int] = None) -> torch.Tensor:
    n = paged_attn_prefix_workspace_size(dims, num_groups) if nbytes is None else int(nbytes)
    if n <= 0:
        raise ValueError("invalid attention dims")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _dims_fit(d: vas_attn_dims, q, k_pages, block_table, seq_lens, quant: Optional[str]) -> bool:
    """Whether every extent the kernels take from d is that of the tensors."""
    T, Hq, D = q.shape
    n, P, Hkv, Dk = k_pages.shape
    code = _KV_CODES.get(q.dtype) if quant is None else _QUANT_CODES.get(quant)
    return Dk == D and (
        (d.num_seqs, d.total_q_tokens, d.num_q_heads, d.num_kv_heads, d.head_dim, d.page_size, d.num_pages,
         d.max_pages_per_seq, d.kv_dtype) ==
        (seq_lens.shape[0], T, Hq, Hkv, D, P, n, block_table.shape[-1], code))


def paged_attn_fwd_prefix(q, k_pages, v_pages, block_table, seq_lens, query_lens, group_start,
                          prefix_lens, out, lse, workspace, *, k_scale=None, v_scale=None,
                          quant: Optional[str] = None, tree_mask=None, share: str = "auto",
                          scale: float = 0.0, dims: Optional[vas_attn_dims] = None,
                          stream=None) -> None:
    """Attention of groups of sequences that share a prefix (include/vas.h:
    paged_attn_fwd_prefix).  group_start [G + 1] and prefix_lens [G] int32; share "auto"
    (where it pays) or "always"; the other arguments are those of paged_attn_fwd, or with
    quant those of paged_attn_fwd_quant.  dims, when given, are those of these tensors
    (attn_dims)."""
    if share not in _SHARE_CODES:
        raise ValueError('share is "auto" or "always"')
    if dims is None:
        dims = attn_dims(q, k_pages, block_table, seq_lens, scale, quant=quant)
    elif not _dims_fit(dims, q, k_pages, block_table, seq_lens, quant):
        raise ValueError("dims are those of another batch, pool or table")
    dev = torch.cuda.current_device()
    i32, f32 = torch.int32, torch.float32
    G = prefix_lens.shape[0]
    n, P, Hkv, _ = pool = k_pages.shape
    if tree_mask is not None and (tree_mask.numel() != q.shape[0] or tree_mask.element_size() != 8):
        raise ValueError("tree_mask needs one 64-bit word per query token")
    kv = torch.uint8 if quant is not None else q.dtype
    B = seq_lens.shape
    st = _lib.paged_attn_fwd_prefix(
        _here(dev, q, "q"), _here(dev, k_pages, "k_pages", None, kv),
        _here(dev, v_pages, "v_pages", pool, kv), _here(dev, k_scale, "k_scale", (n, Hkv, P), f32),
        _here(dev, v_scale, "v_scale", (n, Hkv, P), f32),
        _here(dev, block_table, "block_table", (*B, block_table.shape[-1]), i32),
        _here(dev, seq_lens, "seq_lens", None, i32), _here(dev, query_lens, "query_lens", B, i32),
        _here(dev, group_start, "group_start", (G + 1,), i32),
        _here(dev, prefix_lens, "prefix_lens", (G,), i32), _here(dev, tree_mask, "tree_mask"),
        _here(dev, out, "out", q.shape, q.dtype), _here(dev, lse, "lse", q.shape[:2], f32),
        ctypes.byref(dims), G, _SHARE_CODES[share], _here(dev, workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream_address(dev, stream))
    _check("paged_attn_fwd_prefix", st)


def _heads(dev: int, t: torch.Tensor, name: str, shape, dtype):
    """Address and token stride of a [T, H, D] tensor whose heads are contiguous."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the current device, cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    T, H, D = shape
    s = t.stride()
    if T * H > 0 and (s[2] != 1 or (H > 1 and s[1] != D)):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return t.data_ptr(), (s[0] if T > 1 else H * D)


def paged_kv_append(q, k, v, block_table, seq_lens, query_lens, q_out, k_pages, v_pages, *,
                    cos_sin=None, positions=None, q_weight=None, k_weight=None,
                    interleaved: bool = False, eps: float = 1e-6, k_scale=None, v_scale=None,
                    quant: Optional[str] = None, stream=None) -> None:
    """Norms, rotation and store of this step's tokens (include/vas.h: paged_kv_append).
    q [T, Hq, D], k and v [T, Hkv, D] (rows any 16-byte multiple apart, heads contiguous),
    cos_sin [max_position, rotary_dim] fp32 or None, positions [T] int32 or None; q and
    q_out may both be None.  k_pages / v_pages [num_pages, P, Hkv, D], with quant uint8
    codes and k_scale / v_scale [num_pages, Hkv, P]."""
    num_pages, P, Hkv, D = pool = k_pages.shape
    T, B, act = k.shape[0], seq_lens.shape[0], k.dtype
    if B == 0 and T > 0:  # the call would do nothing, and leave q_out as it was
        raise ValueError(f"{T} tokens of no sequence")
    dev = torch.cuda.current_device()
    i32, f32 = torch.int32, torch.float32
    if quant is not None:
        if quant not in _QUANT_CODES or act != torch.bfloat16 or k_pages.dtype != torch.uint8:
            raise ValueError("a quantised pool is uint8 codes with bf16 q, k and v")
        code = _QUANT_CODES[quant]
    else:
        if act not in _KV_CODES or k_pages.dtype != act:
            raise ValueError("k and k_pages must share a dtype in {bf16, fp32}")
        code = _KV_CODES[act]
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    Hq = 0 if q is None else q.shape[1]
    kp, ks = _heads(dev, k, "k", (T, Hkv, D), act)
    vp, vs = _heads(dev, v, "v", (T, Hkv, D), act)
    qp, qs = _heads(dev, q, "q", (T, Hq, D), act) if Hq else (None, 0)
    if cos_sin is not None and cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rotary_dim]")
    table = (0, 0) if cos_sin is None else cos_sin.shape
    maxp = block_table.shape[-1]
    dims = vas_append_dims(B, T, Hq, Hkv, D, P, num_pages, maxp, code, table[1], int(interleaved),
                           table[0], qs, ks, vs, eps)
    st = _lib.paged_kv_append(
        qp, kp, vp, _here(dev, q_weight, "q_weight", (D,), act),
        _here(dev, k_weight, "k_weight", (D,), act), _here(dev, cos_sin, "cos_sin", None, f32),
        _here(dev, positions, "positions", (T,), i32),
        _here(dev, block_table, "block_table", (B, maxp), i32),
        _here(dev, seq_lens, "seq_lens", None, i32), _here(dev, query_lens, "query_lens", (B,), i32),
        _here(dev, q_out, "q_out", (T, Hq, D), act), _here(dev, k_pages, "k_pages"),
        _here(dev, v_pages, "v_pages", pool, k_pages.dtype),
        _here(dev, k_scale, "k_scale", (num_pages, Hkv, P), f32),
        _here(dev, v_scale, "v_scale", (num_pages, Hkv, P), f32), ctypes.byref(dims),
        _stream_address(dev, stream))
    _check("paged_kv_append", st)


def _pool(dev: int, k_pages, v_pages, k_scale, v_scale):
    """Addresses and vas_pool_dims of [num_pages, P, Hkv, D] pools, or [layers, num_pages, P,
    Hkv, D]."""
    shape = k_pages.shape
    if len(shape) not in (4, 5):
        raise ValueError("a pool is [num_pages, P, Hkv, D], or that for each layer")
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale come together")
    *lead, n, P, Hkv, D = shape
    if k_pages.dtype == torch.uint8:
        code = VAS_FP8_E4M3  # either kind of code: they are moved as bytes
    elif k_pages.dtype in _KV_CODES:
        code = _KV_CODES[k_pages.dtype]
    else:
        raise ValueError("k_pages must be bf16, fp32 or uint8 codes")
    scales = (*lead, n, Hkv, P)
    return (_here(dev, k_pages, "k_pages"), _here(dev, v_pages, "v_pages", shape, k_pages.dtype),
            _here(dev, k_scale, "k_scale", scales, torch.float32),
            _here(dev, v_scale, "v_scale", scales, torch.float32),
            vas_pool_dims(lead[0] if lead else 1, n, P, Hkv, D, code))


def _host_list(x, name: str):
    """A host list of page numbers or token counts as int32 (kept alive by the caller)."""
    import numpy as np
    a = np.asarray(x)
    if a.ndim != 1 or (a.size and a.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of integers")
    if a.dtype != np.int32:
        if a.size and (a.min() < 0 or a.max() > 2**31 - 1):
            raise ValueError(f"{name} is outside the range of page numbers")
        a = a.astype(np.int32)
    return a if a.flags.c_contiguous else np.ascontiguousarray(a)


def _address(a) -> int:
    return a.__array_interface__["data"][0]


def paged_kv_copy(k_pages, v_pages, src, dst, *, tokens=None, k_scale=None, v_scale=None,
                  stream=None) -> None:
    """Copy pages src[i] -> dst[i] of K and V (include/vas.h: paged_kv_copy).  src, dst and
    tokens are host sequences of integers; pools as in paged_kv_append, or with a leading
    layer dimension."""
    dev = torch.cuda.current_device()
    kp, vp, ks, vs, dims = _pool(dev, k_pages, v_pages, k_scale, v_scale)
    s, d = _host_list(src, "src"), _host_list(dst, "dst")
    t = None if tokens is None else _host_list(tokens, "tokens")
    if len(s) != len(d) or (t is not None and len(t) != len(s)):
        raise ValueError("src, dst and tokens differ in length")
    st = _lib.paged_kv_copy(kp, vp, ks, vs, _address(s), _address(d),
                            None if t is None else _address(t), len(s), ctypes.byref(dims),
                            _stream_address(dev, stream))
    _check("paged_kv_copy", st)


def paged_kv_keep_path(k_pages, v_pages, block_table, seq_lens, query_lens, path, accepted_len, *,
                       seq_index=None, k_scale=None, v_scale=None, stream=None) -> None:
    """Move the accepted nodes of draft trees behind their roots (include/vas.h:
    paged_kv_keep_path).  path [B, n] and accepted_len [B] int32 as spec_verify_tree writes
    them; seq_index [B] int32 gives the batch row of each (default: row b); pools as in
    paged_kv_copy."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    kp, vp, ks, vs, dims = _pool(dev, k_pages, v_pages, k_scale, v_scale)
    B, n = path.shape
    N, maxp = seq_lens.shape[0], block_table.shape[-1]
    st = _lib.paged_kv_keep_path(
        kp, vp, ks, vs, _here(dev, block_table, "block_table", (N, maxp), i32),
        _here(dev, seq_lens, "seq_lens", None, i32), _here(dev, query_lens, "query_lens", (N,), i32),
        N, maxp, _here(dev, seq_index, "seq_index", (B,), i32), _here(dev, path, "path", None, i32),
        _here(dev, accepted_len, "accepted_len", (B,), i32), B, n, ctypes.byref(dims),
        _stream_address(dev, stream))
    _check("paged_kv_keep_path", st)


def spec_verify_tree(p, q, draft_tokens, parents, seed: int, accepted_len, out_tokens, path, *,
                     stream=None) -> None:
    """Verification of a draft tree (include/vas.h: spec_verify_tree).  p [B, n+1, V] fp32,
    q [B, n, V] fp32, draft_tokens and parents [B, n] int32 -> accepted_len [B],
    out_tokens [B, n+1], path [B, n]."""
    B, n1, V = p.shape
    st = _lib.spec_verify_tree(_dev(p, "p", torch.float32), _dev(q, "q", torch.float32),
                               _dev(draft_tokens, "draft_tokens", torch.int32),
                               _dev(parents, "parents", torch.int32),
                               ctypes.c_uint64(seed & (2**64 - 1)),
                               _dev(accepted_len, "accepted_len", torch.int32),
                               _dev(out_tokens, "out_tokens", torch.int32),
                               _dev(path, "path", torch.int32), B, n1 - 1, V, _stream_ptr(stream))
    _check("spec_verify_tree", st)


def spec_verify(p, q, draft_tokens, seed: int, accepted_len, out_tokens, *, stream=None) -> None:
    """Modified rejection sampling (include/vas.h: spec_verify).  p [B, k+1, V] fp32,
    q [B, k, V] fp32, draft_tokens [B, k] int32 -> accepted_len [B], out_tokens [B, k+1]."""
    B, k1, V = p.shape
    k = k1 - 1
    qp = _dev(q, "q", torch.float32) if k > 0 else ctypes.c_void_p(0)
    xp = _dev(draft_tokens, "draft_tokens", torch.int32) if k > 0 else ctypes.c_void_p(0)
    st = _lib.spec_verify(_dev(p, "p", torch.float32), qp, xp, ctypes.c_uint64(seed & (2**64 - 1)),
                          _dev(accepted_len, "accepted_len", torch.int32),
                          _dev(out_tokens, "out_tokens", torch.int32), B, k, V, _stream_ptr(stream))
    _check("spec_verify", st)


def vas_last_device_error(stream=None) -> int:
    bits = _i32(0)
    _check("vas_last_device_error", _lib.vas_last_device_error(ctypes.byref(bits), _stream_ptr(stream)))
    return int(bits.value)


def vas_philox4x32_10(counters: torch.Tensor, key0: int, key1: int, out: torch.Tensor, stream=None) -> None:
    n = counters.shape[0]
    _check("vas_philox4x32_10",
           _lib.vas_philox4x32_10(_dev(counters, "counters", torch.int32), key0 & 0xFFFFFFFF,
                                  key1 & 0xFFFFFFFF, _dev(out, "out", torch.int32), n,
                                  _stream_ptr(stream)))


def vas_status_string(status: int) -> str:
    return _lib.vas_status_string(status).decode()


class PagePool:
    """Host page allocator and block-table builder (include/vas.h: vas_pool_*)."""

    def __init__(self, num_pages: int, page_size: int, seed: int = 0):
        self._h = _lib.vas_pool_create(num_pages, page_size, ctypes.c_uint64(seed))
        if not self._h:
            raise ValueError("invalid pool arguments")
        self.num_pages, self.page_size = num_pages, page_size

    def close(self):
        if self._h:
            _lib.vas_pool_destroy(self._h)
            self._h = None

    __del__ = close

    @property
    def free_pages(self) -> int:
        return int(_lib.vas_pool_free_pages(self._h))

    @property
    def num_seqs(self) -> int:
        return int(_lib.vas_pool_num_seqs(self._h))

    def can_allocate(self, n_tokens: int) -> bool:
        return bool(_lib.vas_pool_can_allocate(self._h, n_tokens))

    def pages_needed(self, seq_id: int, n_tokens: int) -> int:
        r = int(_lib.vas_seq_pages_needed(self._h, seq_id, n_tokens))
        if r < 0:
            raise VasError("vas_seq_pages_needed", r)
        return r

    def seq_len(self, seq_id: int) -> int:
        r = int(_lib.vas_seq_len(self._h, seq_id))
        if r < 0:
            raise VasError("vas_seq_len", r)
        return r

    def admit(self, seq_id: int, n_tokens: int) -> int:
        return int(_lib.vas_seq_admit(self._h, seq_id, n_tokens))

    def grow(self, seq_id: int, n_tokens: int) -> int:
        return int(_lib.vas_seq_grow(self._h, seq_id, n_tokens))

    def rollback(self, seq_id: int, n_tokens: int) -> int:
        return int(_lib.vas_seq_rollback(self._h, seq_id, n_tokens))

    def free(self, seq_id: int) -> int:
        return int(_lib.vas_seq_free(self._h, seq_id))

    def fork(self, parent: int, child: int, n_tokens: int) -> int:
        return int(_lib.vas_seq_fork(self._h, parent, child, n_tokens))

    def fork_tail(self, parent: int, child: int, n_tokens: int):
        """(source page, target page, tokens) of the copy a fork leaves, or None."""
        a, b = _i32(-1), _i32(-1)
        r = int(_lib.vas_seq_fork_tail(self._h, parent, child, n_tokens, ctypes.byref(a),
                                       ctypes.byref(b)))
        if r < 0:
            raise VasError("vas_seq_fork_tail", r)
        return (int(a.value), int(b.value), r) if r else None

    def compact(self):
        """Pages in use move to the lowest ids: (src, dst) of the copies to make."""
        import numpy as np
        n = int(_lib.vas_pool_compact(self._h, None, None, 0))
        if n < 0:
            raise VasError("vas_pool_compact", n)
        src, dst = np.empty(n, dtype=np.int32), np.empty(n, dtype=np.int32)
        r = int(_lib.vas_pool_compact(self._h, src.ctypes.data_as(_c_void_p),
                                      dst.ctypes.data_as(_c_void_p), n))
        if r < 0:
            raise VasError("vas_pool_compact", r)
        return src, dst

    def prefix_groups(self, seq_ids, query_lens=None):
        """(group_start, prefix_lens) of consecutive sequences with common first pages."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        ql = None if query_lens is None else np.ascontiguousarray(query_lens, dtype=np.int32)
        if ql is not None and ql.shape != ids.shape:
            raise ValueError("query_lens needs one entry per sequence")
        start, lens = np.zeros(len(ids) + 1, np.int32), np.zeros(max(len(ids), 1), np.int32)
        g = int(_lib.vas_build_prefix_groups(
            self._h, ids.ctypes.data_as(_c_void_p), len(ids),
            ctypes.c_void_p(0) if ql is None else ql.ctypes.data_as(_c_void_p),
            start.ctypes.data_as(_c_void_p), lens.ctypes.data_as(_c_void_p)))
        if g < 0:
            raise VasError("vas_build_prefix_groups", g)
        return start[:g + 1], lens[:g]

    def refcount(self, page: int) -> int:
        return int(_lib.vas_page_refcount(self._h, page))

    def preempt_newest(self):
        v = _i64(0)
        st = int(_lib.vas_pool_preempt_newest(self._h, ctypes.byref(v)))
        return (st, int(v.value))

    def block_table(self, seq_ids, max_pages: int):
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        bt = np.empty((len(ids), max_pages), dtype=np.int32)
        lens = np.empty(len(ids), dtype=np.int32)
        st = _lib.vas_build_block_table(self._h, ids.ctypes.data_as(_c_void_p), len(ids),
                                        bt.ctypes.data_as(_c_void_p), max_pages,
                                        lens.ctypes.data_as(_c_void_p))
        _check("vas_build_block_table", st)
        return bt, lens
