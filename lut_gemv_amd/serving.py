"""The operators of a decoder layer beside its weight products.

Argument marshalling only, as in the package's other calls: the arithmetic, its
conventions and what each call does with indices outside their range are stated
at the entry points of ``include/lutgemm.h``. Tensors are torch tensors in device
memory, fp16 or bf16; every call runs on the current stream of the tensors'
device and allocates its workspace there, so calls on different streams and
captured graphs share nothing. The operators serve; they have no gradients.
"""
from __future__ import annotations

import ctypes
import functools
import struct

__all__ = ["rotary_table", "qk_norm_rotate", "paged_attention", "adapters_add"]

_HEADS = struct.Struct("@7if11q")
_ATTENTION = struct.Struct("@8ifi15q")
_ADAPTERS = struct.Struct("@6i3q")

_torch = None
_lib = None
_types = {}


def _load():
    """torch and the library, bound once."""
    global _torch, _lib
    import torch

    from . import lib
    _lib = lib()
    _types.update({torch.float16: 0, torch.bfloat16: 1})
    _torch = torch


def _raise(status: int, where: str):
    from . import LutGemmError
    raise LutGemmError(status, where)


def _type_of(t, what: str) -> int:
    kind = _types.get(t.dtype)
    if kind is None:
        raise ValueError(f"{what} must be fp16 or bf16, not {t.dtype}")
    return kind


def _like(t, ref, dims: int, what: str):
    """t: of ref's type, on its device, with so many dimensions, the last contiguous."""
    if t.dtype is not ref.dtype or t.device != ref.device or t.dim() != dims:
        raise ValueError(f"{what} must be a {dims}-dimensional {ref.dtype} tensor on {ref.device}")
    strides = t.stride()
    if strides[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    if 1 in t.shape:  # the stride of a single entry is never walked
        strides = tuple(0 if n == 1 else s for n, s in zip(t.shape, strides))
    return strides


def _index(t, dtype, ref, shape, what: str):
    if t.dtype is not dtype or t.device != ref.device or tuple(t.shape) != shape \
            or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on {ref.device}")
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name: str, described: bytes) -> int:
    # a function of the sizes alone
    out = ctypes.c_size_t()
    status = getattr(_lib, name)(described, ctypes.byref(out))
    if status:
        _raise(status, name)
    return out.value


def _call(device, name: str, described: bytes, args, workspace: str = ""):
    """One entry point on the current stream of `device`; `workspace` names its size query."""
    torch = _torch
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _call(device, name, described, args, workspace)
    stream = torch.cuda.current_stream(index).cuda_stream
    if workspace:
        need = _workspace_bytes(workspace, described)
        # allocated for this call in the stream's order: a graph being captured
        # keeps its own
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        status = getattr(_lib, name)(described, *args, ws.data_ptr() if need else None, need, stream)
    else:
        status = getattr(_lib, name)(described, *args, stream)
    if status:
        _raise(status, name)


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
    Returns the queries [tokens][heads][head_dim] (in ``out`` if given); without a
    cache, the queries and the keys [tokens][kv_heads][head_dim].
    """
    if _torch is None:
        _load()
    torch = _torch
    kind = _type_of(qkv, "qkv")
    if not qkv.is_cuda:
        raise ValueError("qkv must be on a GPU")
    heads, kv_heads = int(heads), int(kv_heads)
    qkv_strides = _like(qkv, qkv, 2, "qkv")
    tokens, width = qkv.shape
    parts = heads + 2 * kv_heads
    if heads < 1 or kv_heads < 1 or width % parts:
        raise ValueError(f"qkv's rows do not divide into {heads} + 2 x {kv_heads} heads")
    dim = width // parts
    rotary = limit = 0
    at = turns = None
    if table is not None:
        if table.dtype is not torch.float32 or table.dim() != 2 or not table.is_contiguous() \
                or table.device != qkv.device:
            raise ValueError(f"table must be a contiguous fp32 [positions][rotary] tensor on {qkv.device}")
        if positions is None:
            raise ValueError("a rotation needs the tokens' positions")
        limit, rotary = table.shape
        at, turns = _index(positions, torch.int64, qkv, (tokens,), "positions"), table.data_ptr()
    weights = [None, None]
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if q_weight is not None:
        weights = [_index(q_weight, qkv.dtype, qkv, (dim,), "q_weight"),
                   _index(k_weight, qkv.dtype, qkv, (dim,), "k_weight")]
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=qkv.dtype, device=qkv.device)
    else:
        _like(out, qkv, 3, "out")
        if tuple(out.shape) != (tokens, heads, dim) or (heads > 1 and out.stride(1) != dim):
            raise ValueError(f"out must be {[tokens, heads, dim]} with its heads side by side")
    if (k_pages is None) != (slots is None) or (v_pages is None) != (slots is None):
        raise ValueError("k_pages, v_pages and slots go together")
    if slots is None:
        keys = torch.empty((tokens, kv_heads, dim), dtype=qkv.dtype, device=qkv.device)
        described = _HEADS.pack(kind, heads, kv_heads, dim, rotary, int(bool(interleaved)), 1,
                                eps, tokens, limit, 0, qkv_strides[0], out.stride(0),
                                kv_heads * dim, 0, dim, 0, 0, 0)
        _call(qkv.device, "lutgemm_qk_norm_rotate", described,
              (qkv.data_ptr(), at, turns, *weights, out.data_ptr(), keys.data_ptr(), None, None))
        return out, keys
    ks, vs = _like(k_pages, qkv, 4, "k_pages"), _like(v_pages, qkv, 4, "v_pages")
    pages, page_size = k_pages.shape[:2]
    if tuple(k_pages.shape[2:]) != (kv_heads, dim) or k_pages.shape != v_pages.shape:
        raise ValueError(f"k_pages and v_pages must both be [pages][page_size][{kv_heads}][{dim}]")
    described = _HEADS.pack(kind, heads, kv_heads, dim, rotary, int(bool(interleaved)), page_size,
                            eps, tokens, limit, pages, qkv_strides[0], out.stride(0), *ks[:3],
                            *vs[:3])
    _call(qkv.device, "lutgemm_qk_norm_rotate", described,
          (qkv.data_ptr(), at, turns, *weights, out.data_ptr(), k_pages.data_ptr(),
           v_pages.data_ptr(), _index(slots, torch.int64, qkv, (tokens,), "slots")))
    return out


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
    [tokens][heads][head_dim] (in ``out`` if given).
    """
    if _torch is None:
        _load()
    torch = _torch
    kind = _type_of(q, "q")
    if not q.is_cuda:
        raise ValueError("q must be on a GPU")
    qs, ks, vs = _like(q, q, 3, "q"), _like(k_pages, q, 4, "k_pages"), _like(v_pages, q, 4, "v_pages")
    tokens, heads, dim = q.shape
    pages, page_size, kv_heads, kdim = k_pages.shape
    if kdim != dim or k_pages.shape != v_pages.shape:
        raise ValueError(f"k_pages and v_pages must both be [pages][page_size][kv_heads][{dim}]")
    if page_table.dtype is not torch.int32 or page_table.device != q.device \
            or page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table must be an int32 [seqs][width] tensor on {q.device}, "
                         "contiguous in its last dimension")
    seqs, width = page_table.shape
    lens = _index(kv_lens, torch.int32, q, (seqs,), "kv_lens")
    if q_starts is not None:
        starts = _index(q_starts, torch.int32, q, (seqs + 1,), "q_starts")
    elif tokens != seqs:
        raise ValueError(f"{tokens} tokens of {seqs} sequences need q_starts")
    else:
        starts, max_q = None, 1
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=q.dtype, device=q.device)
    elif tuple(out.shape) != (tokens, heads, dim):
        raise ValueError(f"out must be {[tokens, heads, dim]}")
    os = _like(out, q, 3, "out")
    described = _ATTENTION.pack(
        kind, heads, kv_heads, dim, page_size, seqs, width, window,
        dim ** -0.5 if scale is None else scale, 0, tokens, pages, page_table.stride(0),
        tokens if max_q is None else max_q, width * page_size if max_kv is None else max_kv,
        qs[0], qs[1], os[0], os[1], *ks[:3], *vs[:3])
    _call(q.device, "lutgemm_paged_attention", described,
          (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lens, starts,
           out.data_ptr()), "lutgemm_paged_attention_workspace")
    return out


def adapters_add(y, x, a, b, ids, scales=None, out=None):
    """Low-rank adapters added to a projection's output (lutgemm_adapters_add):
    out_i = y_i + scales[ids_i] * b[ids_i] (a[ids_i] x_i).

    ``y`` [rows][N] and ``x`` [rows][K], the projection's output and input; ``a``
    [adapters][rank][K], ``b`` [adapters][N][rank]; ``ids`` int32 [rows], a row whose id is
    outside [0, adapters) keeps its y; ``scales`` fp32 [adapters] or None. Returns ``out``
    (a new tensor if None; it may be ``y``).
    """
    if _torch is None:
        _load()
    torch = _torch
    kind = _type_of(x, "x")
    if not x.is_cuda:
        raise ValueError("x must be on a GPU")
    xs, ys = _like(x, x, 2, "x"), _like(y, x, 2, "y")
    rows, K = x.shape
    N = y.shape[1]
    if y.shape[0] != rows:
        raise ValueError(f"y has {y.shape[0]} rows, x {rows}")
    _like(a, x, 3, "a")
    count, rank, _ = a.shape
    if a.shape[2] != K or not a.is_contiguous():
        raise ValueError(f"a must be contiguous [adapters][rank][{K}]")
    _index(b, x.dtype, x, (count, N, rank), "b")
    if scales is not None:
        _index(scales, torch.float32, x, (count,), "scales")
    if out is None:
        out = torch.empty((rows, N), dtype=x.dtype, device=x.device)
    elif tuple(out.shape) != (rows, N):
        raise ValueError(f"out must be {[rows, N]}")
    os = _like(out, x, 2, "out")
    described = _ADAPTERS.pack(kind, rows, K, N, rank, count, xs[0], ys[0], os[0])
    _call(x.device, "lutgemm_adapters_add", described,
          (x.data_ptr(), y.data_ptr(), a.data_ptr(), b.data_ptr(),
           scales.data_ptr() if scales is not None else None,
           _index(ids, torch.int32, x, (rows,), "ids"), out.data_ptr()), "lutgemm_adapters_workspace")
    return out
