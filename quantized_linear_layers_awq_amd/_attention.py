"""The attention and cache calls.

As in ``_binding``, torch supplies memory and the stream, the C library
validates and launches.  The arguments are checked and converted by the native
module ``_calls`` (csrc/torch_calls.cpp), for these calls sit between two
linears of a decode step, where a few microseconds of host time count.  Sizes
come from the tensors' shapes.
"""

from __future__ import annotations

import torch

from ._binding import _check, _workspace, load_library

TF_TYPE_BF16, TF_TYPE_F16 = 0, 1

_calls = None


def _native():
    """The native module; raises where the library was never built."""
    global _calls
    if _calls is None:
        load_library()
        from . import _calls as native

        _calls = native
    return _calls


def _run(fn, call, like, stream, *args):
    """call(*args, stream handle) on `like`'s device: torch's current stream,
    or the given one.  Outputs are allocated on the launch stream, so that
    torch orders the memory's reuse with the call.  A call that needs a
    workspace and was given none (its last argument) gets the stream's."""
    index = like.get_device() if isinstance(like, torch.Tensor) else -1
    if index < 0:
        return call(*args, 0)  # refused there
    if stream is not None or torch._C._cuda_getDevice() != index:
        device = torch.device("cuda", index)
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(index)
        else:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        with torch.cuda.device(index), torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
            return _launch(fn, call, index, handle, args)
    return _launch(fn, call, index, torch._C._cuda_getCurrentRawStream(index), args)


def _launch(fn, call, index, handle, args):
    out = call(*args, handle)
    if type(out) is int:
        if out < 0:
            out = call(*args[:-1], _workspace(torch.device("cuda", index), handle, -out), handle)
        if type(out) is int:
            _check(out, fn)
    return out


def tf_kv_append(qkv, rope, seq, pos, tables, k_pages, v_pages, hq, q=None, stream=None):
    """Rotate the query and key heads of qkv [T][(hq + 2 Hkv) D] by their
    positions (rope fp32 [positions][D]: cosines, then sines) and store keys
    and values in the pages that tables [seqs][width] names for (seq, pos)
    int32 [T]; k_pages, v_pages [pages][Hkv][page][D] are written in place.
    Returns q [T][hq][D]."""
    return _run("tf_kv_append", _native().kv_append, qkv, stream, qkv, rope, seq, pos, tables, k_pages, v_pages, hq, q)


def tf_attn_decode_workspace_bytes(seqs: int, hq: int, hkv: int, d: int, longest: int) -> int:
    return int(load_library().tf_attn_decode_workspace_bytes(seqs, hq, hkv, d, longest))


def tf_attn_decode(q, k_pages, v_pages, tables, lens, longest, scale=None, out=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [seqs][Hq][D] (channels
    contiguous), over the first lens[s] tokens of its pages (lens int32 [seqs],
    at most `longest`).  scale defaults to D^-0.5.  Returns [seqs][Hq][D]."""
    return _run("tf_attn_decode", _native().attn_decode, q, stream, q, k_pages, v_pages, tables, lens, longest, scale, out,
                workspace)


def tf_attn_prefill_workspace_bytes(seqs: int, tokens: int, hq: int, hkv: int, d: int, longest: int, keys: int) -> int:
    return int(load_library().tf_attn_prefill_workspace_bytes(seqs, tokens, hq, hkv, d, longest, keys))


def tf_attn_prefill(q, k, v, cu_q, cu_k, longest, scale=None, out=None, workspace=None, stream=None):
    """Causal attention of packed prompts: q [T][Hq][D], k and v
    [keys][Hkv][D] (channels contiguous; parts of one fused QKV output will
    do), sequence s in rows cu_q[s] .. cu_q[s + 1] of q and cu_k[s] ..
    cu_k[s + 1] of k and v (int32 [seqs + 1]), its last token seeing every
    key.  `longest` bounds the new tokens of a sequence.  Keys are taken as they
    are: those of a QKV output are not rotated by tf_kv_append, whose rotated
    keys are in the pages (tf_attn_prefill_paged).  Returns [T][Hq][D]; rows of
    no sequence and past the bound are not written."""
    return _run("tf_attn_prefill", _native().attn_prefill, q, stream, q, k, v, cu_q, cu_k, longest, scale, out, workspace)


def tf_attn_prefill_paged(q, k_pages, v_pages, tables, cu_q, lens, longest, scale=None, out=None, workspace=None,
                          stream=None):
    """Causal attention of packed new tokens q [T][Hq][D] (sequence s in rows
    cu_q[s] .. cu_q[s + 1]) over the first lens[s] tokens of the sequences'
    pages, the new ones included.  Returns [T][Hq][D]; rows of no sequence and
    past the bound (`longest` new tokens) are not written."""
    return _run("tf_attn_prefill_paged", _native().attn_prefill_paged, q, stream, q, k_pages, v_pages, tables, cu_q, lens,
                longest, scale, out, workspace)


def tf_kv_fork_workspace_bytes(forks: int) -> int:
    return int(load_library().tf_kv_fork_workspace_bytes(forks))


def tf_kv_fork(cache, refs, tables, lens, parents, children, refs_out=None, tables_out=None, lens_out=None, status=None,
               workspace=None, stream=None):
    """Make sequence children[i] a copy of parents[i] (int32): full pages are
    shared, a partial page is copied into the lowest free one, in every plane
    of cache [planes][pages][Hkv][page][D].  refs [pages], tables
    [seqs][width], lens [seqs] are int32; their new state goes to the *_out
    tensors, or replaces the inputs where none is given.  Returns status, int32 [1]:
    0, or how many free pages were missing (then nothing is forked)."""
    return _run("tf_kv_fork", _native().kv_fork, cache, stream, cache, refs, tables, lens, parents, children, refs_out,
                tables_out, lens_out, status, workspace)


def tf_kv_compact_workspace_bytes(pages: int) -> int:
    return int(load_library().tf_kv_compact_workspace_bytes(pages))


def tf_kv_compact(cache, refs, tables, refs_out=None, tables_out=None, moved=None, workspace=None, stream=None):
    """Move the pages in use (refs > 0) of cache [planes][pages][Hkv][page][D]
    to the front of the pool, in every plane, and renumber tables; the new
    state goes to the *_out tensors, or replaces the inputs where none is given.
    Returns moved, int32 [pages]: where each page is now, -1 for free ones."""
    return _run("tf_kv_compact", _native().kv_compact, cache, stream, cache, refs, tables, refs_out, tables_out, moved,
                workspace)
