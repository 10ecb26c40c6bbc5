"""Binding of the verify round's operators beside its MoE feed-forward (verify_ops.h).

    round_slots     block table, slot map, positions and tree masks from the requests' lengths
    qk_norm_rope    norm and rotary position of query and key heads, keys and values into the paged cache
    tree_attention  each request's tree of drafted rows over its paged cache (decode: a tree of one)
    token_logprobs  log probabilities of given tokens, entropy and top alternatives of logits rows

As with the MoE round's binding this module checks tensors (types, shapes, devices), passes raw device
pointers and maps status codes to exceptions; what is computed is computed in the HIP library, and
include/verify_ops.h has each call's definition and limits.  All calls are asynchronous on the current
stream of the tensors' device and may be captured into a graph.  Outputs that are not given are
allocated, as is the scratch memory (from torch's allocator, on that stream).
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from . import binding
from .binding import OK, MoeRoundError

F32, BF16, F16 = 0, 1, 2
TYPE_CODES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
MAX_TREE_ROWS = 64
MAX_ALTERNATIVES = 16

# The argument structs of verify_ops.h, packed (native alignment; each starts with its own size).
_SLOTS = struct.Struct("@q3Pq8P6i")
_ROPE = struct.Struct("@q11P15q9if")
_ATTENTION = struct.Struct("@q8P12q9if")
_LOGPROBS = struct.Struct("@q6Pq6i")

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = binding.load()
        i32, i64, vp, args = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p
        for name, res, sig in (
                ("verify_round_slots", i32, [args, vp]),
                ("verify_qk_norm_rope", i32, [args, vp]),
                ("verify_tree_attention_workspace", i64, [args]),
                ("verify_tree_attention", i32, [args, vp, i64, vp]),
                ("verify_token_logprobs_workspace", i64, [args]),
                ("verify_token_logprobs", i32, [args, vp, i64, vp]),
                ("verify_last_hip_error", i32, [])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, sig
        _lib = lib
    return _lib


def _raise(status: int, what: str):
    raise MoeRoundError(status, what, _lib.verify_last_hip_error() if status == binding.ERR_HIP else 0)


# The checks below run on every call of a round's hot path, so each takes the few attribute reads that tell
# that all is well, and looks for what is wrong only if something is.

def _tensor(t, name, device, dtypes, ndim):
    """Checks t's kind; `device` is the index of the GPU that the call's tensors live on (-1: none)."""
    try:
        if t.dtype in dtypes and t.ndim == ndim and t.get_device() == device >= 0:
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.ndim != ndim:
        raise ValueError(f"{name}: {t.ndim} dimensions, not {ndim}")
    raise ValueError(f"{name} must live on the GPU, with the other tensors ({t.device})")


def _vector(t, name, device, length, dtype=torch.int32):
    _tensor(t, name, device, (dtype,), 1)
    if t.size(0) != length:
        raise ValueError(f"{name}: length {t.shape[0]} != {length}")
    if length > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t):
    """The index of the GPU that t lives on, -1 if on none (or no tensor: the checks say so)."""
    return t.get_device() if isinstance(t, torch.Tensor) else -1


def _shape(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


def _strides(t, name):
    """Strides without the last dimension's, which must be contiguous.  A dimension of one element has
    no stride of its own (torch may report any): 0."""
    *outer, last = t.stride()
    shape = t.shape
    if last != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if 1 in shape:
        return [s if n > 1 else 0 for s, n in zip(outer, shape)]
    return outer


def _empty(device, dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=torch.device("cuda", device))


_I32 = (torch.int32,)
_TOKENS = (torch.int32, torch.int64)
_CACHE = (torch.bfloat16, torch.float16)
_ANY = (torch.float32, torch.bfloat16, torch.float16)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda device: torch.cuda.current_stream(device).cuda_stream


def _call(fn, what, device, *args):
    """Calls the library on the current stream of `device`, which is made current if it is not."""
    if device == torch.cuda.current_device():
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st != OK:
        _raise(st, what)


class RoundSlots(NamedTuple):
    """What round_slots makes: row_start int32 [B + 1], slots int32 [N], positions int32 [N], masks int64 [N]
    (None without parents), counts int32 [2] (rows of the round, pages needed)."""
    row_start: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    masks: Optional[torch.Tensor]
    counts: torch.Tensor


def round_slots(cached: torch.Tensor, rows: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
                page_size: int, total_rows: int, parents: Optional[torch.Tensor] = None,
                free_head: Optional[torch.Tensor] = None, out: Optional[RoundSlots] = None) -> RoundSlots:
    """The slots of one round's rows in the paged cache, on the GPU (verify_round_slots).

    cached, rows    int32 [B]: tokens each request has in the cache, new rows it gets
    table           int32 [B, width] block table, updated in place: pages a request grows into are taken
                    from free_pages (int32 [F]) in request order, from place free_head (int32 [1] on
                    the GPU, default 0) on
    total_rows      N, the rows the round's buffers hold; rows behind the last request's get slot -1
    parents         int32 [N]: each drafted row's parent among its request's rows (-1: the committed
                    context), always a lower one; None: each request's rows are a chain
    out             buffers of an earlier call with the same sizes, written again
    counts[0] <= N and counts[1] <= the free pages tell that everything fitted; what did not has slot -1.
    """
    device = _device(table)
    _tensor(table, "table", device, _I32, 2)
    B, width = table.shape
    N = int(total_rows)
    if N < 0:
        raise ValueError("total_rows must not be negative")
    cp, rp = _vector(cached, "cached", device, B), _vector(rows, "rows", device, B)
    _tensor(free_pages, "free_pages", device, _I32, 1)
    F = free_pages.shape[0]
    if not free_pages.is_contiguous():
        raise ValueError("free_pages must be contiguous")
    if width > 1 and table.stride(1) != 1:
        raise ValueError("table: the last dimension must be contiguous")
    stride = table.stride(0) if B > 1 else width
    if stride < width:
        raise ValueError("table: rows overlap")
    hp = _vector(free_head, "free_head", device, 1) if free_head is not None else 0
    pp = _vector(parents, "parents", device, N) if parents is not None else 0
    if out is None:
        buf = _empty(device, torch.int32, B + 3 + 2 * N)
        out = RoundSlots(buf[N + N:N + N + B + 1], buf[:N], buf[N:N + N],
                         _empty(device, torch.int64, N) if parents is not None else None,
                         buf[N + N + B + 1:])
    elif (out.masks is None) != (parents is None):
        raise ValueError("out.masks must be given exactly when parents are")
    args = _SLOTS.pack(
        _SLOTS.size, cp, rp, table.data_ptr(), stride, free_pages.data_ptr(), hp, pp,
        _vector(out.row_start, "out.row_start", device, B + 1), _vector(out.slots, "out.slots", device, N),
        _vector(out.positions, "out.positions", device, N),
        _vector(out.masks, "out.masks", device, N, torch.int64) if out.masks is not None else 0,
        _vector(out.counts, "out.counts", device, 2), B, width, F, page_size, N, 0)
    _call(_load().verify_round_slots, "verify_round_slots", device, args)
    return out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                 inv_freq: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 q_out: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False) -> torch.Tensor:
    """Norm and rotary position of the query and key heads and the cache write (verify_qk_norm_rope).

    q, k, v            [T, heads, D], [T, kv_heads, D] twice: float32 or the cache's type, any row and head
                       strides of whole 16 bytes (slices of one projection, for instance)
    positions, slots   int32 [T]; a row with slot -1 (or past the cache) is skipped
    inv_freq           float32 [R / 2], R <= D rotated values: angle = position * inv_freq
    k_cache, v_cache   [pages, kv_heads, P, D], bfloat16 or float16, any strides of whole 16 bytes
    q_weight, k_weight float32 [D] norm weights; None: that head kind is not normed
    interleaved        rotates pairs (2i, 2i + 1) instead of (i, i + R/2)
    Returns q_out, [T, heads, D] of the cache's type (allocated if None; may be q itself).
    """
    device = _device(q)
    _tensor(q, "q", device, _ANY, 3)
    T, heads, D = q.shape
    one = (q.dtype,)
    _tensor(k, "k", device, one, 3)
    _tensor(v, "v", device, one, 3)
    kv_heads = k.shape[1]
    _shape(k, "k", (T, kv_heads, D))
    _shape(v, "v", (T, kv_heads, D))
    _tensor(k_cache, "k_cache", device, _CACHE, 4)
    pages, _, P, _ = k_cache.shape
    _shape(k_cache, "k_cache", (pages, kv_heads, P, D))
    _tensor(v_cache, "v_cache", device, (k_cache.dtype,), 4)
    _shape(v_cache, "v_cache", k_cache.shape)
    if q.dtype != torch.float32 and q.dtype != k_cache.dtype:
        raise TypeError(f"q, k, v: dtype {q.dtype} is neither float32 nor the cache's {k_cache.dtype}")
    if q_out is None:
        q_out = _empty(device, k_cache.dtype, T, heads, D)
    else:
        _tensor(q_out, "q_out", device, (k_cache.dtype,), 3)
        _shape(q_out, "q_out", q.shape)
    _tensor(inv_freq, "inv_freq", device, (torch.float32,), 1)
    half = inv_freq.shape[0]
    args = _ROPE.pack(
        _ROPE.size, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), _vector(positions, "positions", device, T), _vector(slots, "slots", device, T),
        _vector(inv_freq, "inv_freq", device, half, torch.float32),
        _vector(q_weight, "q_weight", device, D, torch.float32) if q_weight is not None else 0,
        _vector(k_weight, "k_weight", device, D, torch.float32) if k_weight is not None else 0,
        *_strides(q, "q"), *_strides(k, "k"), *_strides(v, "v"), *_strides(q_out, "q_out"),
        *_strides(k_cache, "k_cache"), *_strides(v_cache, "v_cache"), pages,
        T, heads, kv_heads, D, P, half, TYPE_CODES[q.dtype], TYPE_CODES[k_cache.dtype], int(bool(interleaved)), eps)
    _call(_load().verify_qk_norm_rope, "verify_qk_norm_rope", device, args)
    return q_out


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                   cached: torch.Tensor, row_start: torch.Tensor, out: Optional[torch.Tensor] = None,
                   masks: Optional[torch.Tensor] = None, max_rows: Optional[int] = None,
                   scale: Optional[float] = None) -> torch.Tensor:
    """Attention of each request's drafted rows over its paged cache (verify_tree_attention).

    q                  [T, heads, D], the cache's type; request b's rows are row_start[b] .. row_start[b+1] - 1
    k_cache, v_cache   [pages, kv_heads, P, D], bfloat16 or float16 (the rows' own keys and values are in it)
    table              int32 [B, width], cached int32 [B] (tokens before this round), row_start int32 [B + 1]
    masks              int64 [T]: bit i of a row's word lets it see row i of its request (round_slots); None:
                       row i sees rows 0..i
    max_rows           the most rows a request has, 1..64 (default min(T, 64)); rows past it are not computed
    scale              of the scores; default D ** -0.5
    Returns out, like q (allocated, as zeros, if None; may be q itself).  Rows that belong to no request
    are left as they were.
    """
    device = _device(q)
    _tensor(q, "q", device, _CACHE, 3)
    T, heads, D = q.shape
    one = (q.dtype,)
    _tensor(k_cache, "k_cache", device, one, 4)
    pages, kv_heads, P, _ = k_cache.shape
    _shape(k_cache, "k_cache", (pages, kv_heads, P, D))
    _tensor(v_cache, "v_cache", device, one, 4)
    _shape(v_cache, "v_cache", k_cache.shape)
    _tensor(table, "table", device, _I32, 2)
    B, width = table.shape
    if width > 1 and table.stride(1) != 1:
        raise ValueError("table: the last dimension must be contiguous")
    if out is None:
        out = _empty(device, q.dtype, T, heads, D).zero_()
    else:
        _tensor(out, "out", device, one, 3)
        _shape(out, "out", q.shape)
    if max_rows is None:
        max_rows = max(1, min(T, MAX_TREE_ROWS))
    lib = _load()
    args = _ATTENTION.pack(
        _ATTENTION.size, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(),
        _vector(cached, "cached", device, B), _vector(row_start, "row_start", device, B + 1),
        _vector(masks, "masks", device, T, torch.int64) if masks is not None else 0, out.data_ptr(),
        *_strides(q, "q"), *_strides(out, "out"), *_strides(k_cache, "k_cache"), *_strides(v_cache, "v_cache"),
        table.stride(0) if B > 1 else width, pages,
        T, B, heads, kv_heads, D, P, width, max_rows, TYPE_CODES[q.dtype], D ** -0.5 if scale is None else scale)
    need = lib.verify_tree_attention_workspace(args)
    if need < 0:
        _raise(need, "verify_tree_attention")
    work = _empty(device, torch.uint8, need) if need else None
    _call(lib.verify_tree_attention, "verify_tree_attention", device, args,
          work.data_ptr() if need else None, need)
    return out


class TokenLogprobs(NamedTuple):
    """What token_logprobs makes: logprobs float32 [T, N], entropy float32 [T], top_ids int32 [T, top],
    top_logprobs float32 [T, top]."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top: int = 0) -> TokenLogprobs:
    """Log probabilities of given tokens, entropy and top alternatives (verify_token_logprobs).

    logits   [T, V], float32, bfloat16 or float16, rows any distance apart
    tokens   [T, N] int32 or int64 (None: none); a token outside 0 .. V - 1 has log probability -inf
    top      alternatives per row, 0..min(V, 16), by descending logit, equal ones by ascending id
    """
    device = _device(logits)
    _tensor(logits, "logits", device, _ANY, 2)
    T, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits: the last dimension must be contiguous")
    N = 0
    if tokens is not None:
        _tensor(tokens, "tokens", device, _TOKENS, 2)
        N = tokens.shape[1]
        _shape(tokens, "tokens", (T, N))
        if not tokens.is_contiguous():
            raise ValueError("tokens must be contiguous")
    if not 0 <= top <= MAX_ALTERNATIVES or top > V:
        raise ValueError(f"top must be between 0 and {min(V, MAX_ALTERNATIVES)}")
    lib = _load()
    buf = _empty(device, torch.float32, T * (N + 1 + top))
    logprobs, entropy = buf[:T * N].view(T, N), buf[T * N:T * N + T]
    top_logprobs = buf[T * N + T:].view(T, top)
    top_ids = _empty(device, torch.int32, T, top)
    args = _LOGPROBS.pack(
        _LOGPROBS.size, logits.data_ptr(), tokens.data_ptr() if N else 0, logprobs.data_ptr() if N else 0,
        entropy.data_ptr(), top_ids.data_ptr(), top_logprobs.data_ptr(), logits.stride(0) if T > 1 else V,
        T, V, N, top, TYPE_CODES[logits.dtype], int(N > 0 and tokens.dtype == torch.int64))
    need = lib.verify_token_logprobs_workspace(args)
    if need < 0:
        _raise(need, "verify_token_logprobs")
    work = _empty(device, torch.uint8, need) if need else None
    _call(lib.verify_token_logprobs, "verify_token_logprobs", device, args, work.data_ptr() if need else None, need)
    return TokenLogprobs(logprobs, entropy, top_ids, top_logprobs)
