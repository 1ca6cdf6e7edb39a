"""GB300-native DeepSeek-style Sparse Attention decode path: thin Python binding.

Every call here only marshals arguments (device pointers, sizes, the current CUDA
stream) into the C ABI of ``libdsa.so`` (declared in ``include/dsa.h``); every step of
the path runs in the library's CUDA kernels.  If the library is missing or a call fails,
an exception is raised -- there is no other implementation to fall back to.

Where a call takes ``stream``, its inputs must be ready on that stream; a result or workspace that
the caller does not pass is allocated on it, and the caller waits for it before reading a result.

Functions (same names as the C entry points, without the ``dsa_`` prefix):

* ``quant_kv_mxfp8(k, slot_mapping, k_cache)``  -- cache writer, MXFP8 indexer keys
* ``quant_kv_fp8(kv, slot_mapping, kv_cache)``   -- cache writer, FP8 MLA latent rows
* ``quant_kv(k, kv, slot_mapping, k_cache, kv_cache)`` -- both writers in one launch
* ``rope(x, pos, turns, ...)``  -- rotary positions: turn part of every head
* ``rope_quant_kv(k, kv, pos, slot_mapping, k_cache, kv_cache, turns, ...)`` -- the cache
  writers with the rotation on the way
* ``decode_step(...)``  -- writers, indexer + Top-K and SFA of one decode step in one call
* ``indexer_topk(...)``                          -- fused Lightning Indexer + Top-K
* ``indexer_scores(...)``                        -- the same scores written in full
* ``sparse_attn(...)``                           -- Sparse Flash Attention
* ``prefix_attn(...)``                           -- dense attention of a batch that shares a prefix
* ``rope_turns(rot, ...)``                       -- the frequency table the two rotary calls
  take, plain or scaled for long contexts (host arithmetic)
* ``device_status()``                            -- read and clear the device status word
"""

import ctypes
import math
import os

import torch
import torch.autograd.forward_ad as forward_ad

from . import workloads  # noqa: F401  (seeded inputs; no computation of the method)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

PAGE_SIZE = 64
INDEX_DIM = 128
LATENT_DIM = 576
V_DIM = 512
KCACHE_PAGE_BYTES = 8448
KVCACHE_TOKEN_BYTES = 608

STATUS_BITS = {1: "BAD_PAGE", 2: "BAD_SEQ", 4: "BAD_LEN", 8: "BAD_INDEX", 16: "TIMEOUT", 32: "NAN_SCORE", 64: "INTERNAL"}

_lib = None


class DsaError(RuntimeError):
    """A non-zero return of the C ABI."""

    def __init__(self, code, msg):
        super().__init__(f"dsa error {code}: {msg}")
        self.code = code


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGS = {
    "dsa_quant_kv_mxfp8": (ctypes.c_int, [_P, _P, _I32, _P, _I64, _P]),
    "dsa_quant_kv_fp8": (ctypes.c_int, [_P, _P, _I32, _P, _I64, _P]),
    "dsa_quant_kv": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I64, _P]),
    "dsa_indexer_topk": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _P, _I32, _P, _P, _P,
                                        _I32, _I32, _I32, _P, _P, _P]),
    "dsa_indexer_scores": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _I64, _P, _I32, _P, _P, _P,
                                          _I32, _I32, _P, _P]),
    "dsa_sparse_attn_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "dsa_sparse_attn": (ctypes.c_int, [_P, _I32, _I32, _P, _I64, _P, _I32, _P, _P, _I32, _P, _I32,
                                       _F32, _P, _P, _P, _SZ, _P]),
    "dsa_sparse_attn_noalloc": (ctypes.c_int, [_P, _I32, _I32, _P, _I64, _P, _I32, _P, _P, _I32, _P, _I32,
                                               _F32, _P, _P, _P]),
    "dsa_decode_step": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _I64, _P, _I32, _P, _I32, _I32, _I32,
                                       _P, _P, _I32, _P, _P, _I32, _I32, _P, _P, _I32, _F32, _P, _P, _P, _SZ,
                                       _P]),
    "dsa_rope": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _I32, _I64, _I64, _I64, _I64, _P, _P, _I32, _I32, _I32,
                                _F32, _I32, _P]),
    "dsa_rope_quant_kv": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _I32, _P, _P, _I64, _P, _F32, _I32, _I32, _I32,
                                         _P]),
    "dsa_prefix_attn_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "dsa_prefix_attn": (ctypes.c_int, [_P, _I32, _I32, _P, _I64, _P, _I32, _P, _I32, _P, _I32, _P, _P, _I32, _F32, _P,
                                       _P, _P, _SZ, _P]),
    "dsa_device_status": (ctypes.c_int, [_P]),
    "dsa_test_stall_indexer": (ctypes.c_int, [_I32]),
    "dsa_test_prefix_plan": (ctypes.c_int, [_I32, _I32, _I32, _I32, _I32, _P]),
    "dsa_topk_merge": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "dsa_lse_combine": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "dsa_last_error": (ctypes.c_char_p, []),
    "dsa_version": (ctypes.c_int, []),
}

SYMBOLS = tuple(_SIGS)


def lib():
    """Load libdsa.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m dsa_sparse_attention_topk_gb300.build")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def _check(rc):
    if rc != 0:
        raise DsaError(rc, lib().dsa_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _same_device(what, *tensors):
    """The index of the CUDA device that every tensor (None: absent) lies on."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()  # (-1: not a CUDA tensor)
        if dev is None:
            dev = d
        if d != dev or d < 0:
            raise ValueError(f"{what}: tensors must be CUDA tensors on one device (got one on {t.device})")
    return dev


def _tangents():
    """Whether a level of forward-mode differentiation is open."""
    return getattr(forward_ad, "_current_level", -1) >= 0


def _need_no_grad(what, hint, *tensors):
    """Refuse a tensor whose gradient (or tangent) is asked for: the result would come back without.
    (Called where one may be: a small call is bound by this host code.)"""
    grad, tangents = torch.is_grad_enabled(), _tangents()
    for t in tensors:
        if t is not None and ((grad and t.requires_grad) or (tangents and forward_ad.unpack_dual(t).tangent is not None)):
            raise ValueError(f"{what}: a tensor needs a gradient, which this call does not record ({hint})")


def _need_shaped(t, dtype, shape, name):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")


def _scratch(stream, size, device):
    """`size` bytes for a call on `stream` (None: the device's current one), which may be dropped once the call
    is issued: the block belongs to that stream, so the allocator hands it to no other one meanwhile."""
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _result(stream, shape, dtype, device):
    """A result that a call on `stream` writes and its caller reads.  As `_scratch`; and since the caller's
    current stream is another one, the block also waits for that one when it is dropped."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _call_on(device, stream, fn, *args):
    """Call a C entry point with device number `device` current, on `stream` (that device's current one).
    Pointers come as plain integers: a step of small launches is bound by this host code."""
    s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    if rc:
        _check(rc)


# ---- cache allocation (plain torch allocations of the documented layouts) ----------

def alloc_k_cache(num_pages, device="cuda"):
    return torch.zeros(num_pages * KCACHE_PAGE_BYTES, dtype=torch.uint8, device=device)


def alloc_kv_cache(num_pages, device="cuda"):
    return torch.zeros(num_pages * PAGE_SIZE * KVCACHE_TOKEN_BYTES, dtype=torch.uint8, device=device)


# ---- entry points --------------------------------------------------------------------

def quant_kv_mxfp8(k, slot_mapping, k_cache, stream=None):
    """k: bf16 [n, 128]; slot_mapping: int64 [n]; k_cache: uint8 buffer of whole pages."""
    _need(k, torch.bfloat16, "k")
    _need(slot_mapping, torch.int64, "slot_mapping")
    num_slots = k_cache.numel() // KCACHE_PAGE_BYTES * PAGE_SIZE
    _check(lib().dsa_quant_kv_mxfp8(_ptr(k), _ptr(slot_mapping), k.shape[0], _ptr(k_cache),
                                    num_slots, _stream(stream)))


def quant_kv_fp8(kv, slot_mapping, kv_cache, stream=None):
    """kv: bf16 [n, 576]; slot_mapping: int64 [n]; kv_cache: uint8 buffer of whole pages."""
    _need(kv, torch.bfloat16, "kv")
    _need(slot_mapping, torch.int64, "slot_mapping")
    num_slots = kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES) * PAGE_SIZE
    _check(lib().dsa_quant_kv_fp8(_ptr(kv), _ptr(slot_mapping), kv.shape[0], _ptr(kv_cache),
                                  num_slots, _stream(stream)))


def quant_kv(k, kv, slot_mapping, k_cache, kv_cache, stream=None):
    """Both cache writers in one launch: k bf16 [n, 128] -> k_cache, kv bf16 [n, 576] ->
    kv_cache, at the same int64 slots [n]."""
    _need(k, torch.bfloat16, "k")
    _need(kv, torch.bfloat16, "kv")
    _need(slot_mapping, torch.int64, "slot_mapping")
    if k.shape[0] != kv.shape[0] or k.shape[0] != slot_mapping.shape[0]:
        raise ValueError("quant_kv: k, kv and slot_mapping must have the same number of tokens")
    num_slots = min(k_cache.numel() // KCACHE_PAGE_BYTES,
                    kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES)) * PAGE_SIZE
    _check(lib().dsa_quant_kv(_ptr(k), _ptr(kv), _ptr(slot_mapping), k.shape[0], _ptr(k_cache), _ptr(kv_cache),
                              num_slots, _stream(stream)))


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def rope_turns(rot, base=10000.0, scaling=None, factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0,
               device="cuda"):
    """Frequency table of a rotary part of ``rot`` dims: (turns int64 [rot / 2] on `device`,
    amplitude).  Frequency i is base^(-2 i / rot) radians a position; ``turns`` holds it as
    2^-64 turns.  ``scaling`` stretches it to `factor` times the original context length:

    * None      as it is;
    * "linear"  every frequency / factor;
    * "ntk"     base * factor^(rot / (rot - 2)): the lowest frequency is divided by factor;
    * "yarn"    by parts: a frequency that makes beta_fast turns or more in original_len
                positions stays, one that makes beta_slow or fewer is divided by factor, a
                linear ramp over the index in between; amplitude 0.1 ln(factor) + 1.  A model that
                has this factor in its softmax scale already takes 1.0 in the amplitude's place.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rope_turns: rot must be even and at least 2 (got {rot})")
    if not (base > 1.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("rope_turns: base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rope_turns: unknown scaling {scaling!r}")
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("rope_turns: ntk scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    amplitude = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if original_len < 1 or not 0.0 < beta_slow < beta_fast:
            raise ValueError("rope_turns: yarn needs original_len >= 1 and 0 < beta_slow < beta_fast")

        def index_of(n_turns):  # the (fractional) index whose frequency makes n_turns in original_len
            return rot * math.log(original_len / (2.0 * math.pi * n_turns)) / (2.0 * math.log(base))

        low = max(math.floor(index_of(beta_fast)), 0)
        high = min(math.ceil(index_of(beta_slow)), rot - 1)
        width = max(high - low, 1e-3)
        ramp = [min(max((i - low) / width, 0.0), 1.0) for i in range(rot // 2)]
        freq = [f * (1.0 - r) + f / factor * r for f, r in zip(freq, ramp)]
        amplitude = 0.1 * math.log(factor) + 1.0
    turns = [round(f / (2.0 * math.pi) * 2.0 ** 64) for f in freq]
    return torch.tensor(turns, dtype=torch.int64, device=device), amplitude


def _layout(name):
    if name not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)} (got {name!r})")
    return ROPE_LAYOUTS[name]


def rope(x, pos, turns, offset=0, layout="interleaved", amplitude=1.0, transpose=False, out=None, stream=None):
    """Rotary positions: dims [offset, offset + 2 len(turns)) of every head of x turned to
    pos.  x: bf16, fp16 or fp32 [n, d] or [n, h, d], last dim contiguous, any other strides;
    pos: int32 [n]; turns, amplitude: from rope_turns; layout: "interleaved" (pairs 2i, 2i+1)
    or "half" (pairs i, i + rot / 2).  transpose=True gives the gradient with respect to x,
    given that of the result.  out=x works in place (only the rotary part is touched);
    otherwise out must not overlap x.  Tensors that need a gradient are refused: call it under
    torch.no_grad(), or in the two halves of an autograd function.  Returns out."""
    if x.requires_grad or _tangents() or (out is not None and out.requires_grad):
        _need_no_grad("rope", "transpose=True gives it", x, out)
    shape, code = x.shape, _DTYPES.get(x.dtype)
    if len(shape) not in (2, 3) or code is None:
        raise ValueError("rope: x must be [n, d] or [n, h, d] of bf16, fp16 or fp32")
    if out is None:
        out = _result(stream, shape, x.dtype, x.device)
    elif out.shape != shape or out.dtype != x.dtype:
        raise ValueError("rope: out must have x's shape and dtype")
    dev = _same_device("rope", x, pos, turns, out)
    _need_shaped(pos, torch.int32, shape[:1], "rope: pos")
    _need_shaped(turns, torch.int64, turns.shape[:1], "rope: turns")
    xs, os_ = x.stride(), out.stride()
    if (xs[-1] != 1 or os_[-1] != 1) and shape[-1] > 1:
        raise ValueError("rope: the last dim of x and out must be contiguous")
    h, xh, oh = (shape[1], xs[1], os_[1]) if len(shape) == 3 else (1, 0, 0)
    _call_on(dev, stream, lib().dsa_rope, x.data_ptr(), out.data_ptr(), code, shape[0], h, shape[-1], xs[0], xh,
             os_[0], oh, pos.data_ptr(), turns.data_ptr(), 2 * turns.shape[0], offset, _layout(layout), amplitude,
             1 if transpose else 0)
    return out


def rope_quant_kv(k, kv, pos, slot_mapping, k_cache, kv_cache, turns, amplitude=1.0, k_offset=0, k_layout="half",
                  kv_layout="interleaved", stream=None):
    """quant_kv with the rotation on the way: k bf16 [n, 128] (rotary dims [k_offset,
    k_offset + 64), layout k_layout) -> k_cache, kv bf16 [n, 576] (rotary dims [512, 576),
    layout kv_layout) -> kv_cache, turned to the positions pos int32 [n] and quantised from
    fp32, at the int64 slots [n] (negative: skipped).  Rows may lie further apart than their
    width (a slice of a wider projection).  k and k_cache, or kv and kv_cache, may be None."""
    if k is None and kv is None:
        raise ValueError("rope_quant_kv: k or kv must be given")
    first = k if k is not None else kv
    rows = first.shape[:1]
    pages = 1 << 48
    for t, cache, width, page_bytes, name in ((k, k_cache, INDEX_DIM, KCACHE_PAGE_BYTES, "k"),
                                              (kv, kv_cache, LATENT_DIM, PAGE_SIZE * KVCACHE_TOKEN_BYTES, "kv")):
        if (t is None) != (cache is None):
            raise ValueError(f"rope_quant_kv: {name} and {name}_cache go together")
        if t is None:
            continue
        if t.dtype != torch.bfloat16 or t.shape != (*rows, width) or t.stride(1) != 1:
            raise ValueError(f"{name} must be bf16 [n, {width}] with contiguous rows")
        if cache.dtype != torch.uint8 or not cache.is_contiguous():
            raise ValueError(f"{name}_cache must be a contiguous uint8 tensor")
        pages = min(pages, cache.numel() // page_bytes)
    dev = _same_device("rope_quant_kv", first, k, kv, pos, slot_mapping, k_cache, kv_cache, turns)
    _need_shaped(pos, torch.int32, rows, "rope_quant_kv: pos")
    _need_shaped(slot_mapping, torch.int64, rows, "rope_quant_kv: slot_mapping")
    _need_shaped(turns, torch.int64, (32,), "rope_quant_kv: turns")
    _call_on(dev, stream, lib().dsa_rope_quant_kv,
             *((None, 0) if k is None else (k.data_ptr(), k.stride(0))),
             *((None, 0) if kv is None else (kv.data_ptr(), kv.stride(0))),
             pos.data_ptr(), slot_mapping.data_ptr(), rows[0], None if k is None else k_cache.data_ptr(),
             None if kv is None else kv_cache.data_ptr(), pages * PAGE_SIZE, turns.data_ptr(), amplitude, k_offset,
             _layout(k_layout), _layout(kv_layout))


def indexer_topk(q, w, k_cache, page_table, seq_lens, q_seq, q_pos, topk, max_ctx,
                 q_group=1, out_idx=None, out_scores=None, stream=None):
    """Fused indexer + Top-K.  q: bf16 [n_q, h_i, 128]; w: fp32 [n_q, h_i];
    page_table: int32 [n_seq, max_pages]; seq_lens: int32 [n_seq]; q_seq, q_pos: int32
    [n_q].  Returns (out_idx int32 [n_q, topk], out_scores fp32 or None)."""
    n_q, h_i, _ = q.shape
    if out_idx is None:
        out_idx = _result(stream, (n_q, topk), torch.int32, q.device)
    num_pages = k_cache.numel() // KCACHE_PAGE_BYTES
    _check(lib().dsa_indexer_topk(_ptr(q), _ptr(w), n_q, h_i, q_group, _ptr(k_cache), num_pages,
                                  _ptr(page_table), page_table.shape[1], _ptr(seq_lens), _ptr(q_seq),
                                  _ptr(q_pos), seq_lens.shape[0], max_ctx, topk, _ptr(out_idx),
                                  _ptr(out_scores), _stream(stream)))
    return out_idx, out_scores


def indexer_scores(q, w, k_cache, page_table, seq_lens, q_seq, q_pos, max_ctx, q_group=1,
                   out=None, stream=None):
    """All scores [n_q, max_ctx] fp32 (-inf where a row may not select)."""
    n_q, h_i, _ = q.shape
    if out is None:
        out = _result(stream, (n_q, max_ctx), torch.float32, q.device)
    num_pages = k_cache.numel() // KCACHE_PAGE_BYTES
    _check(lib().dsa_indexer_scores(_ptr(q), _ptr(w), n_q, h_i, q_group, _ptr(k_cache), num_pages,
                                    _ptr(page_table), page_table.shape[1], _ptr(seq_lens), _ptr(q_seq),
                                    _ptr(q_pos), seq_lens.shape[0], max_ctx, _ptr(out), _stream(stream)))
    return out


def sparse_attn_workspace_size(n_q, h_s, topk):
    return int(lib().dsa_sparse_attn_workspace_size(n_q, h_s, topk))


def sparse_attn(q, kv_cache, page_table, seq_lens, q_seq, topk_idx, sm_scale, out=None,
                out_lse=None, workspace=None, stream=None):
    """Sparse Flash Attention.  q: bf16 [n_q, h_s, 576]; topk_idx: int32 [n_q, K].
    Returns (out bf16 [n_q, h_s, 512], out_lse or None)."""
    n_q, h_s, _ = q.shape
    topk = topk_idx.shape[1]
    if out is None:
        out = _result(stream, (n_q, h_s, V_DIM), torch.bfloat16, q.device)
    ws_need = sparse_attn_workspace_size(n_q, h_s, topk)
    if workspace is None and ws_need:
        workspace = _scratch(stream, ws_need, q.device)
    num_pages = kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES)
    _check(lib().dsa_sparse_attn(_ptr(q), n_q, h_s, _ptr(kv_cache), num_pages, _ptr(page_table),
                                 page_table.shape[1], _ptr(seq_lens), _ptr(q_seq), seq_lens.shape[0],
                                 _ptr(topk_idx), topk, float(sm_scale), _ptr(out), _ptr(out_lse),
                                 _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                 _stream(stream)))
    return out, out_lse


def decode_step(k_new, kv_new, slot_mapping, k_cache, kv_cache, q_idx, w, q_sfa, page_table, seq_lens,
                q_seq, q_pos, topk, max_ctx, sm_scale, q_group=1, out_idx=None, out=None, out_lse=None,
                workspace=None, stream=None):
    """One decode step in one call: write k_new / kv_new (bf16 [n_new, 128] / [n_new, 576],
    int64 slots [n_new]) into the caches, then the fused indexer + Top-K, then Sparse Flash
    Attention over the selected entries.  Returns (out bf16 [n_q, h_s, 512], out_lse or
    None, out_idx int32 [n_q, topk])."""
    _need(k_new, torch.bfloat16, "k_new")
    _need(kv_new, torch.bfloat16, "kv_new")
    _need(slot_mapping, torch.int64, "slot_mapping")
    n_new = k_new.shape[0]
    if kv_new.shape[0] != n_new or slot_mapping.shape[0] != n_new:
        raise ValueError("decode_step: k_new, kv_new and slot_mapping must have the same number of tokens")
    n_q, h_i, _ = q_idx.shape
    h_s = q_sfa.shape[1]
    if out_idx is None:
        out_idx = _result(stream, (n_q, topk), torch.int32, q_idx.device)
    if out is None:
        out = _result(stream, (n_q, h_s, V_DIM), torch.bfloat16, q_idx.device)
    ws_need = sparse_attn_workspace_size(n_q, h_s, topk)
    if workspace is None and ws_need:
        workspace = _scratch(stream, ws_need, q_idx.device)
    num_pages = min(k_cache.numel() // KCACHE_PAGE_BYTES, kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES))
    _check(lib().dsa_decode_step(_ptr(k_new), _ptr(kv_new), _ptr(slot_mapping), n_new, _ptr(k_cache),
                                 _ptr(kv_cache), num_pages, _ptr(page_table), page_table.shape[1],
                                 _ptr(seq_lens), seq_lens.shape[0], max_ctx, n_q, _ptr(q_seq), _ptr(q_pos),
                                 q_group, _ptr(q_idx), _ptr(w), h_i, topk, _ptr(out_idx), _ptr(q_sfa), h_s,
                                 float(sm_scale), _ptr(out), _ptr(out_lse), _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), _stream(stream)))
    return out, out_lse, out_idx


def sparse_attn_noalloc(q, kv_cache, page_table, seq_lens, q_seq, topk_idx, sm_scale, out=None,
                        out_lse=None, stream=None):
    """Sparse Flash Attention with the split-merge scratch kept in the library's fixed
    array, for callers that cannot allocate device memory.  Same result as sparse_attn.
    Calls that overlap on the GPU share that array and must not run concurrently."""
    n_q, h_s, _ = q.shape
    topk = topk_idx.shape[1]
    if out is None:
        out = _result(stream, (n_q, h_s, V_DIM), torch.bfloat16, q.device)
    num_pages = kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES)
    _check(lib().dsa_sparse_attn_noalloc(_ptr(q), n_q, h_s, _ptr(kv_cache), num_pages, _ptr(page_table),
                                         page_table.shape[1], _ptr(seq_lens), _ptr(q_seq), seq_lens.shape[0],
                                         _ptr(topk_idx), topk, float(sm_scale), _ptr(out), _ptr(out_lse),
                                         _stream(stream)))
    return out, out_lse


def prefix_attn_workspace_size(n_q, h_s, n_seq, prefix_len, max_ctx):
    return int(lib().dsa_prefix_attn_workspace_size(n_q, h_s, n_seq, prefix_len, max_ctx))


def prefix_attn(q, kv_cache, prefix_pages, prefix_len, page_table, seq_lens, q_seq, q_pos, max_ctx, sm_scale,
                out=None, out_lse=None, workspace=None, stream=None):
    """Dense attention of query rows whose sequences share their first prefix_len positions,
    read once for all from prefix_pages (int32 [ceil(prefix_len / 64)]); each row then sees
    its own sequence's positions up to q_pos.  q: bf16 [n_q, h_s, 576]; page_table: int32
    [n_seq, max_pages] (entries before prefix_len / 64 are not read); seq_lens: int32 [n_seq],
    prefix included; q_seq, q_pos: int32 [n_q]; max_ctx: host-side bound of seq_lens.
    Tensors that need a gradient are refused (there is no backward pass).  Returns
    (out bf16 [n_q, h_s, 512], out_lse or None)."""
    if q.requires_grad or _tangents() or (out is not None and out.requires_grad) or (
            out_lse is not None and out_lse.requires_grad):
        _need_no_grad("prefix_attn", "there is no backward pass", q, out, out_lse)
    if q.dim() != 3 or q.shape[2] != LATENT_DIM:
        raise ValueError("prefix_attn: q must be [n_q, h_s, 576]")
    n_q, h_s, _ = q.shape
    n_seq = seq_lens.shape[0]
    dev = _same_device("prefix_attn", q, kv_cache, prefix_pages, page_table, seq_lens, q_seq, q_pos, out, out_lse,
                       workspace)
    _need_shaped(q, torch.bfloat16, q.shape, "prefix_attn: q")
    _need_shaped(kv_cache, torch.uint8, kv_cache.shape, "prefix_attn: kv_cache")
    _need_shaped(seq_lens, torch.int32, (n_seq,), "prefix_attn: seq_lens")
    _need_shaped(q_seq, torch.int32, (n_q,), "prefix_attn: q_seq")
    _need_shaped(q_pos, torch.int32, (n_q,), "prefix_attn: q_pos")
    if prefix_pages is not None:
        _need_shaped(prefix_pages, torch.int32, prefix_pages.shape, "prefix_attn: prefix_pages")
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() < (prefix_len + PAGE_SIZE - 1) // PAGE_SIZE):
        raise ValueError("prefix_attn: prefix_pages must name ceil(prefix_len / 64) pages")
    max_pages = 0
    if page_table is not None:
        max_pages = page_table.shape[-1]
        _need_shaped(page_table, torch.int32, (n_seq, max_pages), "prefix_attn: page_table")
    if out is None:
        out = _result(stream, (n_q, h_s, V_DIM), torch.bfloat16, q.device)
    else:
        _need_shaped(out, torch.bfloat16, (n_q, h_s, V_DIM), "prefix_attn: out")
    if out_lse is not None:
        _need_shaped(out_lse, torch.float32, (n_q, h_s), "prefix_attn: out_lse")
    if workspace is None:
        # (the plan goes by the device's multiprocessors: ask with that device current)
        size = lib().dsa_prefix_attn_workspace_size
        if dev == torch._C._cuda_getDevice():
            need = size(n_q, h_s, n_seq, prefix_len, max_ctx)
        else:
            with torch.cuda.device(dev):
                need = size(n_q, h_s, n_seq, prefix_len, max_ctx)
        workspace = _scratch(stream, need, q.device)
    elif not workspace.is_contiguous():  # (its elements might lie on one another)
        raise ValueError("prefix_attn: workspace must be contiguous")
    _call_on(dev, stream, lib().dsa_prefix_attn, q.data_ptr(), n_q, h_s, kv_cache.data_ptr(),
             kv_cache.numel() // (PAGE_SIZE * KVCACHE_TOKEN_BYTES),
             None if prefix_pages is None else prefix_pages.data_ptr(), prefix_len,
             None if page_table is None else page_table.data_ptr(), max_pages, seq_lens.data_ptr(), n_seq,
             q_seq.data_ptr(), q_pos.data_ptr(), max_ctx, sm_scale, out.data_ptr(),
             None if out_lse is None else out_lse.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    return out, out_lse


NOALLOC_SCRATCH_BYTES = 40 * 1024 * 1024


def topk_merge(cand_idx, cand_scores, topk, part_offsets=None, local_lo=None, local_hi=None, out_idx=None,
               out_scores=None, stream=None):
    """The K highest of several parts' candidates per row (context parallelism).
    cand_idx int32 / cand_scores fp32 [n_parts, n_q, k_in] (part-local positions, -1 empty);
    part_offsets int32 [n_parts, n_q] or None.  Returns (out_idx int32 [n_q, topk] global
    positions by score then position, out_scores fp32, out_local int32 [n_q, topk] or None:
    the positions inside [local_lo, local_hi) relative to local_lo, -1 elsewhere)."""
    _need(cand_idx, torch.int32, "cand_idx")
    _need(cand_scores, torch.float32, "cand_scores")
    n_parts, n_q, k_in = cand_idx.shape
    if out_idx is None:
        out_idx = _result(stream, (n_q, topk), torch.int32, cand_idx.device)
    if out_scores is None:
        out_scores = _result(stream, (n_q, topk), torch.float32, cand_idx.device)
    out_local = None
    if local_lo is not None:
        out_local = _result(stream, (n_q, topk), torch.int32, cand_idx.device)
    _check(lib().dsa_topk_merge(_ptr(cand_idx), _ptr(cand_scores), _ptr(part_offsets), n_parts, n_q, k_in, topk,
                                _ptr(out_idx), _ptr(out_scores), _ptr(local_lo), _ptr(local_hi), _ptr(out_local),
                                _stream(stream)))
    return out_idx, out_scores, out_local


def lse_combine(o_parts, lse_parts, out=None, out_lse=None, stream=None):
    """Combine attention outputs over disjoint entry sets: o_parts bf16 [n_parts, n_q, h, 512],
    lse_parts fp32 [n_parts, n_q, h].  Returns (out bf16 [n_q, h, 512], out_lse fp32)."""
    _need(o_parts, torch.bfloat16, "o_parts")
    _need(lse_parts, torch.float32, "lse_parts")
    n_parts, n_q, h, _ = o_parts.shape
    if out is None:
        out = _result(stream, (n_q, h, V_DIM), torch.bfloat16, o_parts.device)
    if out_lse is None:
        out_lse = _result(stream, (n_q, h), torch.float32, o_parts.device)
    _check(lib().dsa_lse_combine(_ptr(o_parts), _ptr(lse_parts), n_parts, n_q, h, _ptr(out), _ptr(out_lse),
                                 _stream(stream)))
    return out, out_lse


def device_status(stream=None):
    """Synchronise the stream and return (and clear) the device status bits."""
    rc = lib().dsa_device_status(_stream(stream))
    if rc < 0:
        _check(rc)
    return rc


def test_stall_indexer(wait_limit_us):
    """Testing aid for the bounded waits (dsa_test_stall_indexer): a positive limit makes
    every following indexer launch stall its copy producer and give up waiting after that
    many microseconds; 0 restores normal operation."""
    _check(lib().dsa_test_stall_indexer(int(wait_limit_us)))


def test_prefix_plan(n_q, h_s, n_seq, prefix_len, max_ctx):
    """Testing aid (dsa_test_prefix_plan): how prefix_attn would split a call of these sizes."""
    plan = (_I32 * 8)()
    _check(lib().dsa_test_prefix_plan(n_q, h_s, n_seq, prefix_len, max_ctx, plan))
    return dict(zip(("group", "tiles_prefix", "splits_prefix", "tail_first", "tiles_tail", "splits_tail", "few_parts",
                     "few_first"), plan))


def status_names(bits):
    return [n for b, n in STATUS_BITS.items() if bits & b]
