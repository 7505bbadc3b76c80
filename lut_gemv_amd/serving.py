"""The operators of a serving step beside the weight products: those between a decoder
layer's products, and the step's tables before the layers and its sampling after them.

The arithmetic, its conventions and what each call does with indices outside
their range are stated at the entry points of ``include/lutgemm.h``. Tensors are
torch tensors in device memory, fp16 or bf16, checked and handed over by
``_binding.so`` (``csrc/binding.cpp``): ValueError for a wrong type, device or
shape, LutGemmError for numbers that an entry point refuses. Every call runs on the
current stream of the tensors' device and allocates its workspace in that
stream's order, so calls on different streams and captured graphs share nothing.
The operators serve; they have no gradients, and refuse tensors that need one.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["rotary_table", "qk_norm_rotate", "paged_attention", "adapters_add", "batch_tables",
           "shared_prefix_attention", "sample_tokens"]

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")

_ops = None


def _load():
    """The binding, bound once to the library's entry points."""
    global _ops
    from . import LutGemmError, lib
    L = lib()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built; run `python -m lut_gemv_amd.build`")
    from . import _binding
    names = ("lutgemm_qk_norm_rotate", "lutgemm_paged_attention",
             "lutgemm_paged_attention_workspace", "lutgemm_adapters_add",
             "lutgemm_adapters_workspace", "lutgemm_shared_attention",
             "lutgemm_shared_attention_workspace", "lutgemm_batch_tables",
             "lutgemm_batch_tables_workspace", "lutgemm_sample_tokens",
             "lutgemm_sample_tokens_workspace")
    _binding.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names), LutGemmError)
    _ops = _binding
    return _ops


def rotary_table(positions: int, rotary: int, base: float = 10000.0, device="cuda"):
    """The angles' table of :func:`qk_norm_rotate`: fp32 [positions][rotary], of position
    p the cosines and then the sines of p * base^(-2i/rotary), computed in 64 bits."""
    import torch
    if positions < 1 or rotary < 2 or rotary % 2:
        raise ValueError("positions must be >= 1 and rotary even and >= 2")
    turn = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(device)


def qk_norm_rotate(qkv, heads: int, kv_heads: int, positions=None, table=None, q_weight=None,
                   k_weight=None, eps: float = 1e-6, interleaved: bool = False, k_pages=None,
                   v_pages=None, slots=None, out=None):
    """Norms of queries and keys for each head, rotation by position, and the append of
    keys and values to the paged cache, in one pass (lutgemm_qk_norm_rotate).

    ``qkv`` [tokens][(heads + 2 kv_heads) head_dim], the fused projection's output;
    ``positions`` int64 [tokens]; ``table`` fp32 [positions][rotary]
    (:func:`rotary_table`), None for no rotation; ``q_weight``, ``k_weight`` [head_dim], None
    for no norm; ``k_pages``, ``v_pages`` [pages][page_size][kv_heads][head_dim], of any
    strides over the head dimension, and ``slots`` int64 [tokens], the cache slots of the
    tokens (one outside the cache is not written).
    Returns the queries [tokens][heads][head_dim] (in ``out`` if given, which may be
    ``qkv``'s own query part); without a cache, the queries and the keys
    [tokens][kv_heads][head_dim].
    """
    return (_ops or _load()).qk_norm_rotate(qkv, heads, kv_heads, positions, table, q_weight, k_weight,
                                            eps, interleaved, k_pages, v_pages, slots, out)


def paged_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts=None, max_q=None,
                    max_kv=None, scale=None, window: int = 0, out=None):
    """Attention of new tokens over a paged key/value cache (lutgemm_paged_attention).

    ``q`` [tokens][heads][head_dim]; ``k_pages``, ``v_pages``
    [pages][page_size][kv_heads][head_dim]; ``page_table`` int32 [seqs][width];
    ``kv_lens`` int32 [seqs], the keys of each sequence with its new tokens' own;
    ``q_starts`` int32 [seqs + 1], the first row of each sequence's new tokens and the end
    of the last (None: one new token each). ``max_q`` and ``max_kv``, the most new tokens and keys
    of one sequence, help to choose the launch (None: no bound known). ``scale``: None for
    head_dim ** -0.5; ``window``: the last so many keys only, 0 for all. Returns
    [tokens][heads][head_dim] (in ``out`` if given, which may be ``q``).
    """
    return (_ops or _load()).paged_attention(q, k_pages, v_pages, page_table, kv_lens, q_starts, max_q,
                                             max_kv, scale, window, out)


def adapters_add(y, x, a, b, ids, scales=None, out=None):
    """Low-rank adapters added to a projection's output (lutgemm_adapters_add):
    out_i = y_i + scales[ids_i] * b[ids_i] (a[ids_i] x_i).

    ``y`` [rows][N] and ``x`` [rows][K], the projection's output and input; ``a``
    [adapters][rank][K], ``b`` [adapters][N][rank]; ``ids`` int32 [rows], a row whose id is
    outside [0, adapters) keeps its y; ``scales`` fp32 [adapters] or None. Returns ``out``
    (a new tensor if None; it may be ``y``, but not overlap ``x`` or ``y`` otherwise).
    """
    return (_ops or _load()).adapters_add(y, x, a, b, ids, scales, out)


def shared_prefix_attention(q, k_pages, v_pages, prefix_table, prefix_lens, page_table, kv_lens,
                            q_starts=None, group_starts=None, max_q=None, max_kv=None, max_prefix=None,
                            scale=None, out=None):
    """Attention of new tokens of sequences that share long prefixes, each prefix read once
    for its whole group (lutgemm_shared_attention).

    ``prefix_table`` int32 [groups][width] and ``prefix_lens`` int32 [groups]: the pages and keys of
    the prefixes; ``group_starts`` int32 [groups + 1]: the first sequence of each group and the
    end of the last (None: one group of all). ``page_table`` and ``kv_lens`` are the keys
    behind the prefix, which the new tokens' own end; the other arguments are those of
    :func:`paged_attention`, ``max_prefix`` one more hint for the launch. Returns
    [tokens][heads][head_dim] (in ``out`` if given, which may be ``q``).
    """
    return (_ops or _load()).shared_prefix_attention(q, k_pages, v_pages, prefix_table, prefix_lens,
                                                     page_table, kv_lens, q_starts, group_starts, max_q,
                                                     max_kv, max_prefix, scale, out)


def batch_tables(change, kv_lens, page_table, page_size: int, tokens: int, free_pages=None,
                 free_range=None, offsets=None, in_place: bool = False):
    """One step's page tables, slots, positions and row ranges, made on the GPU
    (lutgemm_batch_tables).

    ``change`` int32 [seqs]: each sequence's new tokens, or minus the keys that it gives back
    (-kv_lens: all of them); ``kv_lens`` int32 [seqs], its keys before the step; ``page_table`` int32
    [seqs][width], to which the pages taken are added; ``tokens``: the rows of the step, at least
    as many as there are new tokens; ``free_pages`` int32 [capacity] with ``free_range`` int32 [2]
    (first, count), the ring of free pages (None: the table has all pages already);
    ``offsets`` int32 [seqs], added to the positions (the lengths of shared prefixes).
    Returns (positions, slots, kv_lens, q_starts, free_range): int64 [tokens] twice, as
    :func:`qk_norm_rotate` takes them, int32 [seqs] and [seqs + 1], as :func:`paged_attention`
    does, and the ring's new range (None without one). ``in_place``: the lengths and the range
    are written over those given, so that a captured step goes on from where it ended. A
    sequence that finds no room (rows, pages, width of its table row) keeps its length and gets no rows.
    """
    return (_ops or _load()).batch_tables(change, kv_lens, page_table, page_size, tokens, free_pages,
                                          free_range, offsets, in_place)


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """Next tokens drawn from logits by one random number a row (lutgemm_sample_tokens).

    ``logits`` [rows][vocab], fp16, bf16 or fp32; ``u`` fp32 [rows] in [0, 1); ``temperature``,
    ``top_p``, ``min_p`` fp32 [rows] and ``top_k`` int32 [rows], None for none: a temperature of 0 takes
    the largest logit, top_k <= 0, top_p >= 1 and min_p <= 0 filter nothing.
    Returns (tokens int64 [rows] (``out`` if given), their log-probabilities fp32 [rows]); -1 and NaN
    for a row that has no distribution.
    """
    return (_ops or _load()).sample_tokens(logits, u, temperature, top_k, top_p, min_p, out)
