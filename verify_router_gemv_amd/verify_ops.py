"""Binding of the verify round's operators beside its MoE feed-forward (verify_ops.h).

    round_slots     block table, slot map, positions and tree masks from the requests' lengths
    qk_norm_rope    norm and rotary position of query and key heads, keys and values into the paged cache
    tree_attention  each request's tree of drafted rows over its paged cache (decode: a tree of one)
    token_logprobs  log probabilities of given tokens, entropy and top alternatives of logits rows

As with the MoE round's binding, tensors are checked (types, shapes, devices), raw device pointers passed
and status codes mapped to exceptions, here by the extension module _verify_ops (csrc/verify_binding.cpp);
what is computed is computed in the HIP library, and include/verify_ops.h has each call's definition and
limits.  All calls are asynchronous on the current stream of the tensors' device and may be captured into a
graph.  Outputs that are not given are allocated, as is the scratch memory (from torch's allocator, on that
stream).  They serve: no call records a gradient, whatever its inputs require.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import binding

MAX_TREE_ROWS = 64
MAX_ALTERNATIVES = 16

_module = None


def _native():
    """The extension module (raises if it is not built: there is no fallback path)."""
    global _module
    if _module is None:
        binding.load()
        try:
            from . import _verify_ops
        except ImportError as e:
            raise ImportError(f"{e}; run `python -m verify_router_gemv_amd.build`") from e
        _verify_ops.set_error(binding.MoeRoundError)
        _module = _verify_ops
    return _module


class RoundSlots(NamedTuple):
    """What round_slots makes: row_start int32 [B + 1], slots int32 [N], positions int32 [N], masks int64 [N]
    (None without parents), counts int32 [2] (rows of the round, pages needed)."""
    row_start: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    masks: Optional[torch.Tensor]
    counts: torch.Tensor


_NO_SLOTS = (None,) * 5


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
    made = _native().round_slots(cached, rows, table, free_pages, page_size, total_rows, parents, free_head,
                                 *(out if out is not None else _NO_SLOTS))
    return out if out is not None else RoundSlots(*made)


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
    return _native().qk_norm_rope(q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_out, q_weight, k_weight, eps,
                                  interleaved)


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
    return _native().tree_attention(q, k_cache, v_cache, table, cached, row_start, out, masks, max_rows, scale)


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
    return TokenLogprobs(*_native().token_logprobs(logits, tokens, top))
