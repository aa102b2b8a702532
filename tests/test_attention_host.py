"""Refusals of the attention and cache calls, without a GPU: the C ABI with
addresses that are never followed, the binding with host tensors, workspace
sizes.  They only run where no GPU is visible, so that a validation bug gives
TF_ERR_HIP (no device) and never a launch."""

import inspect
import os
import re

import pytest
import torch

import quantized_linear_layers_awq_amd as tf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, _, ALIGN, SMALL, UNSUPPORTED, HIP = range(8)
P, WS = 1 << 20, 1 << 24  # 16- and 256-byte aligned

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="passes addresses that no device may follow")

APPEND = dict(type=0, qkv=P, qkv_token=6144, rope=P, rope_rows=100, seq=P, pos=P, T=4, tables=P, seqs=4, width=8, q=P,
              k_pages=P, v_pages=P, pages=32, page=16, Hq=32, Hkv=8, D=128, stream=0)
DECODE = dict(type=0, q=P, q_token=4096, q_head=128, k_pages=P, v_pages=P, pages=32, page=16, tables=P, width=8, lens=P,
              out=P, seqs=4, Hq=32, Hkv=8, D=128, longest=128, scale=0.1, workspace=0, ws_bytes=0, stream=0)
PREFILL = dict(type=0, q=P, q_token=6144, q_head=128, k=P, k_token=6144, k_head=128, v=P, v_token=6144, v_head=128, cu_q=P,
               cu_k=P, out=P, seqs=2, T=4000, keys=4000, Hq=32, Hkv=8, D=128, longest=2000, scale=0.1, workspace=0,
               ws_bytes=0, stream=0)
PAGED = dict(type=0, q=P, q_token=6144, q_head=128, k_pages=P, v_pages=P, pages=999, page=16, tables=P, width=8, cu_q=P,
             lens=P, out=P, seqs=2, T=4000, Hq=32, Hkv=8, D=128, longest=2000, scale=0.1, workspace=0, ws_bytes=0, stream=0)
FORK = dict(cache=P, planes=4, pages=64, Hkv=2, page=16, D=64, refs=P, tables=P, lens=P, seqs=8, width=5, parents=P,
            children=P, forks=3, refs_out=P, tables_out=P, lens_out=P, status=P, workspace=WS, ws_bytes=1 << 16, stream=0)
COMPACT = dict(cache=P, planes=4, pages=64, Hkv=2, page=16, D=64, refs=P, tables=P, seqs=8, width=5, refs_out=P,
               tables_out=P, moved=P, workspace=WS, ws_bytes=1 << 16, stream=0)
CALLS = dict(tf_kv_append=APPEND, tf_attn_decode=DECODE, tf_attn_prefill=PREFILL, tf_attn_prefill_paged=PAGED,
             tf_kv_fork=FORK, tf_kv_compact=COMPACT)


def call(name, **changes):
    base = CALLS[name]
    assert set(changes) <= set(base), set(changes) - set(base)
    return getattr(tf.load_library(), name)(*dict(base, **changes).values())


def test_argument_lists_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tilefuse_attention.h")).read(), flags=re.S)
    for name, base in CALLS.items():
        args = re.search(r"int %s\((.*?)\);" % name, text, re.S).group(1)
        assert [a.split()[-1].lstrip("*") for a in args.split(",")] == list(base), name
        assert len(getattr(tf.load_library(), name).argtypes) == len(base), name


NULLS = [(n, k) for n, base in CALLS.items() for k, v in base.items() if v in (P, WS)]


@needs_no_gpu
@pytest.mark.parametrize("name,arg", NULLS)
def test_null_and_misaligned_pointers(name, arg):
    assert call(name, **{arg: 0}) == NULL
    assert call(name, **{arg: CALLS[name][arg] + 2}) == ALIGN


BAD = [
    ("tf_kv_append", SHAPE, dict(T=-1)), ("tf_kv_append", SHAPE, dict(T=2**31)), ("tf_kv_append", SHAPE, dict(Hq=0)),
    ("tf_kv_append", SHAPE, dict(Hkv=0)), ("tf_kv_append", SHAPE, dict(Hq=65536)), ("tf_kv_append", SHAPE, dict(D=0)),
    ("tf_kv_append", SHAPE, dict(qkv_token=6143)), ("tf_kv_append", SHAPE, dict(seqs=-1)), ("tf_kv_append", SHAPE, dict(pages=0)),
    ("tf_kv_append", SHAPE, dict(width=0)), ("tf_kv_append", SHAPE, dict(rope_rows=-1)), ("tf_kv_append", SHAPE, dict(width=2**27)),
    ("tf_kv_append", ALIGN, dict(qkv_token=6148)), ("tf_kv_append", UNSUPPORTED, dict(D=120, qkv_token=8000)),
    ("tf_kv_append", UNSUPPORTED, dict(D=1040, qkv_token=10**6)), ("tf_kv_append", UNSUPPORTED, dict(page=24)),
    ("tf_kv_append", UNSUPPORTED, dict(page=8)), ("tf_kv_append", UNSUPPORTED, dict(page=2048)),
    ("tf_kv_append", UNSUPPORTED, dict(type=2)), ("tf_kv_append", UNSUPPORTED, dict(type=-1)),
    ("tf_attn_decode", UNSUPPORTED, dict(type=7)), ("tf_attn_decode", SHAPE, dict(Hq=30)), ("tf_attn_decode", SHAPE, dict(Hkv=0)),
    ("tf_attn_decode", UNSUPPORTED, dict(D=96, q_head=96)), ("tf_attn_decode", UNSUPPORTED, dict(D=256, q_head=256, q_token=8192)),
    ("tf_attn_decode", UNSUPPORTED, dict(Hq=1025, Hkv=1, q_token=1025 * 128)), ("tf_attn_decode", SHAPE, dict(seqs=-1)),
    ("tf_attn_decode", SHAPE, dict(seqs=65536)), ("tf_attn_decode", SHAPE, dict(longest=-1)),
    ("tf_attn_decode", SHAPE, dict(longest=2**30 + 1)), ("tf_attn_decode", SHAPE, dict(pages=2**31)),
    ("tf_attn_decode", SHAPE, dict(width=2**26 + 1)), ("tf_attn_decode", SHAPE, dict(q_token=127)),
    ("tf_attn_decode", SHAPE, dict(q_head=64)), ("tf_attn_decode", SHAPE, dict(q_token=2**26)),
    ("tf_attn_decode", ALIGN, dict(q_token=4100)), ("tf_attn_decode", ALIGN, dict(q_head=132)),
    ("tf_attn_decode", UNSUPPORTED, dict(scale=0.0)), ("tf_attn_decode", UNSUPPORTED, dict(scale=-1.0)),
    ("tf_attn_decode", UNSUPPORTED, dict(scale=float("nan"))), ("tf_attn_decode", UNSUPPORTED, dict(scale=float("inf"))),
    ("tf_attn_decode", UNSUPPORTED, dict(page=17)), ("tf_attn_decode", NULL, dict(longest=4096)),
    ("tf_attn_decode", SMALL, dict(longest=4096, workspace=WS, ws_bytes=64)),
    ("tf_attn_decode", ALIGN, dict(longest=4096, workspace=WS + 128, ws_bytes=1 << 40)),
    ("tf_attn_prefill", SHAPE, dict(longest=4001)), ("tf_attn_prefill", SHAPE, dict(longest=-1)),
    ("tf_attn_prefill", SHAPE, dict(T=2**30 + 1)), ("tf_attn_prefill", SHAPE, dict(keys=-1)),
    ("tf_attn_prefill", SHAPE, dict(keys=2**30 + 1)), ("tf_attn_prefill", SHAPE, dict(seqs=-2)),
    ("tf_attn_prefill", SHAPE, dict(seqs=2**30)), ("tf_attn_prefill", SHAPE, dict(k_token=64)),
    ("tf_attn_prefill", SHAPE, dict(v_head=0)), ("tf_attn_prefill", SHAPE, dict(v_token=2**26)),
    ("tf_attn_prefill", ALIGN, dict(k_head=129)), ("tf_attn_prefill", ALIGN, dict(v_token=6145)),
    ("tf_attn_prefill", UNSUPPORTED, dict(D=32)), ("tf_attn_prefill", SHAPE, dict(Hq=31)),
    ("tf_attn_prefill", UNSUPPORTED, dict(scale=float("inf"))), ("tf_attn_prefill", NULL, dict(longest=100, T=100, seqs=1)),
    ("tf_attn_prefill", SMALL, dict(longest=100, T=100, seqs=1, workspace=WS, ws_bytes=256)),
    ("tf_attn_prefill_paged", UNSUPPORTED, dict(page=48)), ("tf_attn_prefill_paged", SHAPE, dict(width=0)),
    ("tf_attn_prefill_paged", SHAPE, dict(width=2**27)), ("tf_attn_prefill_paged", SHAPE, dict(pages=0)),
    ("tf_attn_prefill_paged", SHAPE, dict(longest=2**31)), ("tf_attn_prefill_paged", UNSUPPORTED, dict(type=3)),
    ("tf_attn_prefill_paged", NULL, dict(longest=9, T=9, seqs=1, width=1000)),
    ("tf_kv_fork", SHAPE, dict(forks=-1)), ("tf_kv_fork", SHAPE, dict(planes=-1)), ("tf_kv_fork", SHAPE, dict(planes=65537)),
    ("tf_kv_fork", SHAPE, dict(forks=2**30)), ("tf_kv_fork", SHAPE, dict(pages=0)), ("tf_kv_fork", SHAPE, dict(page=0)),
    ("tf_kv_fork", SHAPE, dict(page=1025)), ("tf_kv_fork", SHAPE, dict(width=2**27)), ("tf_kv_fork", SHAPE, dict(seqs=-1)),
    ("tf_kv_fork", SHAPE, dict(Hkv=0)), ("tf_kv_fork", SHAPE, dict(Hkv=40000, page=1024, D=64)),
    ("tf_kv_fork", UNSUPPORTED, dict(D=12)), ("tf_kv_fork", SMALL, dict(ws_bytes=3)),
    ("tf_kv_fork", ALIGN, dict(workspace=WS + 16)), ("tf_kv_compact", SHAPE, dict(pages=2**31)),
    ("tf_kv_compact", SHAPE, dict(D=0)), ("tf_kv_compact", UNSUPPORTED, dict(D=4)), ("tf_kv_compact", SMALL, dict(ws_bytes=380)),
    ("tf_kv_compact", SHAPE, dict(seqs=2**31)), ("tf_kv_compact", SHAPE, dict(planes=10**6)),
]


@needs_no_gpu
@pytest.mark.parametrize("name,status,changes", BAD)
def test_refusals(name, status, changes):
    assert call(name, **changes) == status


@needs_no_gpu
@pytest.mark.parametrize("name,changes", [
    ("tf_kv_append", dict(T=0, qkv=0, seq=0)), ("tf_attn_decode", dict(seqs=0, q=0, lens=0)),
    ("tf_attn_prefill", dict(seqs=0, cu_q=0)), ("tf_attn_prefill", dict(T=0, longest=0, q=0)),
    ("tf_attn_prefill", dict(longest=0, out=0)), ("tf_attn_prefill_paged", dict(seqs=0, tables=0)),
    ("tf_attn_prefill_paged", dict(T=0, longest=0)),
])
def test_nothing_to_do(name, changes):
    assert call(name, **changes) == OK


@needs_no_gpu
@pytest.mark.parametrize("name", list(CALLS))
def test_valid_calls_reach_the_device(name):
    """The base arguments pass every check: without a device they end in TF_ERR_HIP."""
    assert call(name) == HIP


def test_workspace_sizes():
    assert tf.tf_attn_decode_workspace_bytes(4, 32, 8, 128, 512) == 0  # a workgroup per item
    shares = tf.tf_attn_decode_workspace_bytes(4, 32, 8, 128, 513)
    assert shares > 0 and shares == tf.tf_attn_decode_workspace_bytes(1, 8, 1, 128, 10**6)
    assert tf.tf_attn_decode_workspace_bytes(100, 40, 8, 128, 1024) == 0  # enough items
    assert tf.tf_attn_decode_workspace_bytes(4, 80, 2, 128, 4096) == pytest.approx(3 * shares, rel=0.01)  # 40 heads: 3 tiles of 16
    for bad in ((-1, 32, 8, 128, 4096), (4, 32, 7, 128, 4096), (4, 32, 8, 96, 4096), (4, 32, 8, 128, 2**31)):
        assert tf.tf_attn_decode_workspace_bytes(*bad) == 0
    assert tf.tf_attn_prefill_workspace_bytes(1, 8192, 32, 8, 128, 8192, 8192) == 0  # rows enough
    few = tf.tf_attn_prefill_workspace_bytes(1, 100, 32, 8, 128, 100, 8192)
    assert few % (100 * 32 * 130 * 4) == 0 and few // (100 * 32 * 130 * 4) in range(2, 17)
    assert tf.tf_attn_prefill_workspace_bytes(1, 100, 32, 8, 128, 100, 512) == 0  # two ranges at most
    assert tf.tf_attn_prefill_workspace_bytes(1, 100, 32, 8, 128, 101, 8192) == 0
    assert tf.tf_kv_fork_workspace_bytes(-1) == 0 and tf.tf_kv_fork_workspace_bytes(7) == 7 * 4 * 4
    assert tf.tf_kv_compact_workspace_bytes(9) == (1 + 3 * 4) * 4 and tf.tf_kv_compact_workspace_bytes(0) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    pages = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    for fn, args in ((tf.tf_kv_append, (t.view(4, -1), t, i, i, i.view(1, -1), pages, pages, 4)),
                     (tf.tf_attn_decode, (t, pages, pages, i.view(1, -1), i, 9)), (tf.tf_attn_prefill, (t, t, t, i, i, 4)),
                     (tf.tf_attn_prefill_paged, (t, pages, pages, i.view(1, -1), i, i, 4)),
                     (tf.tf_kv_fork, (pages[None], i, i.view(1, -1), i, i, i)), (tf.tf_kv_compact, (pages[None], i, i.view(1, -1)))):
        with pytest.raises(ValueError, match="device tensor"):
            fn(*args)
        with pytest.raises(TypeError, match="torch.Tensor"):
            fn(None, *args[1:])


def test_every_call_takes_a_stream_and_documents_itself():
    for name in CALLS:
        f = getattr(tf, name)
        assert "stream" in inspect.signature(f).parameters and f.__doc__
