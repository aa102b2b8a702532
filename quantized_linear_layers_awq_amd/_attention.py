"""ctypes marshalling of the attention and cache calls (argument handling only).

As in ``_binding``: torch supplies memory and the stream, the C library
validates and launches.  Sizes come from the tensors' shapes; what the C side
cannot see -- types, devices, shapes that do not fit each other -- is checked
here.  These calls sit between two linears of a decode step, where a few
microseconds of host time count, so the checks are kept to attribute reads.
"""

from __future__ import annotations

import torch

from . import _binding
from ._binding import _check, _workspace, load_library

TF_TYPE_BF16, TF_TYPE_F16 = 0, 1
_TYPES = {torch.bfloat16: TF_TYPE_BF16, torch.float16: TF_TYPE_F16}
_I32 = torch.int32


def _lib():
    return _binding._lib or load_library()


def _type(t: torch.Tensor, fn: str, name: str) -> int:
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{fn}: {name} must be bfloat16 or float16 (got {t.dtype})") from None


def _same(fn: str, names, dtype, index: int, *tensors):
    """Tensors of `dtype` on device `index`, contiguous; `names` in their order, space-separated."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            i = next(i for i, u in enumerate(tensors) if u is t)
            raise ValueError(f"{fn}: {names.split()[i]} must be a contiguous {dtype} tensor on cuda:{index} "
                             f"(got {t.dtype} on {t.device}, strides {tuple(t.stride())})")


def _device(t: torch.Tensor, fn: str, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{fn}: {name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a device tensor (got {t.device})")
    return t.get_device()


class _On:
    """The device and stream of a call.  Outputs are allocated on the launch
    stream, so that torch orders the memory's reuse with the call; a call on
    another device than the current one switches to it."""

    __slots__ = ("index", "handle", "contexts")

    def __init__(self, index, stream):
        self.index = index
        self.contexts = ()
        if torch._C._cuda_getDevice() != index:
            self._enter(torch.cuda.device(index))
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(index)
        else:
            self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            self._enter(torch.cuda.stream(torch.cuda.ExternalStream(self.handle, device=torch.device("cuda", index))))

    def _enter(self, context):
        context.__enter__()
        self.contexts += (context,)

    def __enter__(self):
        return self

    def __exit__(self, *error):
        for context in reversed(self.contexts):
            context.__exit__(*error)


def _stride(t: torch.Tensor, fn: str, name: str):
    """(token stride, head stride) of [tokens][heads][D] with contiguous channels."""
    token, head, channel = t.stride()
    if channel != 1 and t.numel():
        raise ValueError(f"{fn}: the channels of {name} must be contiguous (strides {tuple(t.stride())})")
    tokens, heads, d = t.shape
    # the stride of an axis of one entry means nothing
    return (token if tokens > 1 else heads * d if token < d else token), (head if heads > 1 else d)


def _result(t, shape, like, index, fn, name):
    """The given output, checked, or a new one of `like`'s type and device."""
    return like.new_empty(shape) if t is None else _given(t, shape, like.dtype, index, fn, name)


def _given(t, shape, dtype, index, fn, name):
    _same(fn, name, dtype, index, t)
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must be {list(shape)} (got {list(t.shape)})")
    return t


def _pages(fn, k_pages, v_pages, tables):
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or tables.dim() != 2:
        raise ValueError(f"{fn}: k_pages and v_pages must be [pages][Hkv][page][D] of one shape, tables [seqs][width]")
    return k_pages.shape


def _need_workspace(workspace, on, nbytes, fn):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = _workspace(torch.device("cuda", on.index), on.handle, nbytes)
    elif workspace.get_device() != on.index or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous tensor on cuda:{on.index}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def tf_kv_append(qkv, rope, seq, pos, tables, k_pages, v_pages, hq, q=None, stream=None):
    """Rotate the query and key heads of qkv [T][(hq + 2 Hkv) D] by their
    positions (rope fp32 [positions][D]: cosines, then sines) and store keys
    and values in the pages that tables [seqs][width] names for (seq, pos)
    int32 [T]; k_pages, v_pages [pages][Hkv][page][D] are written in place.
    Returns q [T][hq][D]."""
    fn = "tf_kv_append"
    index = _device(qkv, fn, "qkv")
    kind = _type(qkv, fn, "qkv")
    _same(fn, "k_pages v_pages", qkv.dtype, index, k_pages, v_pages)
    _same(fn, "seq pos tables", _I32, index, seq, pos, tables)
    _same(fn, "rope", torch.float32, index, rope)
    pages, hkv, page, d = _pages(fn, k_pages, v_pages, tables)
    tokens, wide = seq.numel(), (hq + 2 * hkv) * d
    if qkv.shape != (tokens, wide) or (qkv.stride(1) != 1 and wide > 1 and tokens):
        raise ValueError(f"{fn}: qkv must be [{tokens}][{wide}] with contiguous channels")
    if pos.numel() != tokens or rope.dim() != 2 or rope.shape[1] != d:
        raise ValueError(f"{fn}: pos must have {tokens} entries, rope must be [positions][{d}]")
    with _On(index, stream) as on:
        q = _result(q, (tokens, hq, d), qkv, index, fn, "q")
        _check(_lib().tf_kv_append(kind, qkv.data_ptr(), qkv.stride(0) if tokens > 1 else wide, rope.data_ptr(),
                                   rope.shape[0], seq.data_ptr(), pos.data_ptr(), tokens, tables.data_ptr(),
                                   tables.shape[0], tables.shape[1], q.data_ptr(), k_pages.data_ptr(),
                                   v_pages.data_ptr(), pages, page, hq, hkv, d, on.handle), fn)
    return q


def tf_attn_decode_workspace_bytes(seqs: int, hq: int, hkv: int, d: int, longest: int) -> int:
    return int(load_library().tf_attn_decode_workspace_bytes(seqs, hq, hkv, d, longest))


def _scale(scale, d):
    return d ** -0.5 if scale is None else float(scale)


def tf_attn_decode(q, k_pages, v_pages, tables, lens, longest, scale=None, out=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [seqs][Hq][D] (channels
    contiguous), over the first lens[s] tokens of its pages (lens int32 [seqs],
    at most `longest`).  scale defaults to D^-0.5.  Returns [seqs][Hq][D]."""
    fn = "tf_attn_decode"
    index = _device(q, fn, "q")
    kind = _type(q, fn, "q")
    _same(fn, "k_pages v_pages", q.dtype, index, k_pages, v_pages)
    _same(fn, "tables lens", _I32, index, tables, lens)
    pages, hkv, page, d = _pages(fn, k_pages, v_pages, tables)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"{fn}: q must be [seqs][Hq][{d}]")
    seqs, hq, _ = q.shape
    if lens.numel() != seqs or tables.shape[0] != seqs:
        raise ValueError(f"{fn}: lens and tables must have {seqs} rows")
    token, head = _stride(q, fn, "q")
    lib = _lib()
    with _On(index, stream) as on:
        out = _result(out, (seqs, hq, d), q, index, fn, "out")
        ws, have = _need_workspace(workspace, on, lib.tf_attn_decode_workspace_bytes(seqs, hq, hkv, d, longest), fn)
        _check(lib.tf_attn_decode(kind, q.data_ptr(), token, head, k_pages.data_ptr(), v_pages.data_ptr(), pages, page,
                                  tables.data_ptr(), tables.shape[1], lens.data_ptr(), out.data_ptr(), seqs, hq, hkv, d,
                                  longest, _scale(scale, d), ws, have, on.handle), fn)
    return out


def tf_attn_prefill_workspace_bytes(seqs: int, tokens: int, hq: int, hkv: int, d: int, longest: int, keys: int) -> int:
    return int(load_library().tf_attn_prefill_workspace_bytes(seqs, tokens, hq, hkv, d, longest, keys))


def tf_attn_prefill(q, k, v, cu_q, cu_k, longest, scale=None, out=None, workspace=None, stream=None):
    """Causal attention of packed prompts: q [T][Hq][D], k and v
    [keys][Hkv][D] (channels contiguous; parts of one fused QKV output will
    do), sequence s in rows cu_q[s] .. cu_q[s + 1] of q and cu_k[s] ..
    cu_k[s + 1] of k and v (int32 [seqs + 1]), its last token seeing every
    key.  `longest` bounds the new tokens of a sequence.  Returns [T][Hq][D]."""
    fn = "tf_attn_prefill"
    index = _device(q, fn, "q")
    kind = _type(q, fn, "q")
    _same(fn, "cu_q cu_k", _I32, index, cu_q, cu_k)
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError(f"{fn}: q must be [T][Hq][D], k and v [keys][Hkv][D] of one shape")
    if k.dtype is not q.dtype or v.dtype is not q.dtype or k.get_device() != index or v.get_device() != index:
        raise ValueError(f"{fn}: q, k and v must have one type and device")
    seqs = cu_q.numel() - 1
    if seqs < 0 or cu_k.numel() != seqs + 1:
        raise ValueError(f"{fn}: cu_q and cu_k must have seqs + 1 entries")
    tokens, hq, d = q.shape
    keys, hkv, _ = k.shape
    qt, qh = _stride(q, fn, "q")
    kt, kh = _stride(k, fn, "k")
    vt, vh = _stride(v, fn, "v")
    lib = _lib()
    with _On(index, stream) as on:
        out = _result(out, (tokens, hq, d), q, index, fn, "out")
        ws, have = _need_workspace(workspace, on,
                                   lib.tf_attn_prefill_workspace_bytes(seqs, tokens, hq, hkv, d, longest, keys), fn)
        _check(lib.tf_attn_prefill(kind, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                                   cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(), seqs, tokens, keys, hq, hkv, d,
                                   longest, _scale(scale, d), ws, have, on.handle), fn)
    return out


def tf_attn_prefill_paged(q, k_pages, v_pages, tables, cu_q, lens, longest, scale=None, out=None, workspace=None,
                          stream=None):
    """Causal attention of packed new tokens q [T][Hq][D] (sequence s in rows
    cu_q[s] .. cu_q[s + 1]) over the first lens[s] tokens of the sequences'
    pages, the new ones included.  Returns [T][Hq][D]."""
    fn = "tf_attn_prefill_paged"
    index = _device(q, fn, "q")
    kind = _type(q, fn, "q")
    _same(fn, "k_pages v_pages", q.dtype, index, k_pages, v_pages)
    _same(fn, "tables cu_q lens", _I32, index, tables, cu_q, lens)
    pages, hkv, page, d = _pages(fn, k_pages, v_pages, tables)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"{fn}: q must be [T][Hq][{d}]")
    seqs, (rows, width) = lens.numel(), tables.shape
    if cu_q.numel() != seqs + 1 or rows != seqs:
        raise ValueError(f"{fn}: cu_q must have {seqs + 1} entries, tables {seqs} rows")
    tokens, hq, _ = q.shape
    token, head = _stride(q, fn, "q")
    lib = _lib()
    with _On(index, stream) as on:
        out = _result(out, (tokens, hq, d), q, index, fn, "out")
        ws, have = _need_workspace(workspace, on,
                                   lib.tf_attn_prefill_workspace_bytes(seqs, tokens, hq, hkv, d, longest, width * page), fn)
        _check(lib.tf_attn_prefill_paged(kind, q.data_ptr(), token, head, k_pages.data_ptr(), v_pages.data_ptr(),
                                         pages, page, tables.data_ptr(), width, cu_q.data_ptr(), lens.data_ptr(),
                                         out.data_ptr(), seqs, tokens, hq, hkv, d, longest, _scale(scale, d), ws, have,
                                         on.handle), fn)
    return out


def tf_kv_fork_workspace_bytes(forks: int) -> int:
    return int(load_library().tf_kv_fork_workspace_bytes(forks))


def tf_kv_compact_workspace_bytes(pages: int) -> int:
    return int(load_library().tf_kv_compact_workspace_bytes(pages))


def _pool(fn, cache, refs, tables):
    index = _device(cache, fn, "cache")
    if cache.dim() != 5 or cache.element_size() != 2 or not cache.is_contiguous():
        raise ValueError(f"{fn}: cache must be a contiguous 16-bit tensor [planes][pages][Hkv][page][D]")
    _same(fn, "refs tables", _I32, index, refs, tables)
    if refs.numel() != cache.shape[1] or tables.dim() != 2:
        raise ValueError(f"{fn}: refs must have {cache.shape[1]} entries, tables must be [seqs][width]")
    return index


def tf_kv_fork(cache, refs, tables, lens, parents, children, refs_out=None, tables_out=None, lens_out=None, status=None,
               workspace=None, stream=None):
    """Make sequence children[i] a copy of parents[i] (int32): full pages are
    shared, a partial page is copied into the lowest free one, in every plane
    of cache [planes][pages][Hkv][page][D].  refs [pages], tables
    [seqs][width], lens [seqs] are int32; their new state goes to the *_out
    tensors, or replaces the inputs where none is given.  Returns status, int32 [1]:
    0, or how many free pages were missing (then nothing is forked)."""
    fn = "tf_kv_fork"
    index = _pool(fn, cache, refs, tables)
    _same(fn, "lens parents children", _I32, index, lens, parents, children)
    if lens.numel() != tables.shape[0] or parents.numel() != children.numel():
        raise ValueError(f"{fn}: lens must have {tables.shape[0]} entries, parents and children equally many")
    planes, pages, hkv, page, d = cache.shape
    forks = parents.numel()
    lib = _lib()
    with _On(index, stream) as on:
        refs_out = refs if refs_out is None else _given(refs_out, refs.shape, _I32, index, fn, "refs_out")
        tables_out = tables if tables_out is None else _given(tables_out, tables.shape, _I32, index, fn, "tables_out")
        lens_out = lens if lens_out is None else _given(lens_out, lens.shape, _I32, index, fn, "lens_out")
        status = _result(status, (1,), refs, index, fn, "status")
        ws, have = _need_workspace(workspace, on, lib.tf_kv_fork_workspace_bytes(forks), fn)
        _check(lib.tf_kv_fork(cache.data_ptr(), planes, pages, hkv, page, d, refs.data_ptr(), tables.data_ptr(),
                              lens.data_ptr(), tables.shape[0], tables.shape[1], parents.data_ptr(),
                              children.data_ptr(), forks, refs_out.data_ptr(), tables_out.data_ptr(),
                              lens_out.data_ptr(), status.data_ptr(), ws, have, on.handle), fn)
    return status


def tf_kv_compact(cache, refs, tables, refs_out=None, tables_out=None, moved=None, workspace=None, stream=None):
    """Move the pages in use (refs > 0) of cache [planes][pages][Hkv][page][D]
    to the front of the pool, in every plane, and renumber tables; the new
    state goes to the *_out tensors, or replaces the inputs where none is given.
    Returns moved, int32 [pages]: where each page is now, -1 for free ones."""
    fn = "tf_kv_compact"
    index = _pool(fn, cache, refs, tables)
    planes, pages, hkv, page, d = cache.shape
    lib = _lib()
    with _On(index, stream) as on:
        refs_out = refs if refs_out is None else _given(refs_out, refs.shape, _I32, index, fn, "refs_out")
        tables_out = tables if tables_out is None else _given(tables_out, tables.shape, _I32, index, fn, "tables_out")
        moved = _result(moved, (pages,), refs, index, fn, "moved")
        ws, have = _need_workspace(workspace, on, lib.tf_kv_compact_workspace_bytes(pages), fn)
        _check(lib.tf_kv_compact(cache.data_ptr(), planes, pages, hkv, page, d, refs.data_ptr(), tables.data_ptr(),
                                 tables.shape[0], tables.shape[1], refs_out.data_ptr(), tables_out.data_ptr(),
                                 moved.data_ptr(), ws, have, on.handle), fn)
    return moved
