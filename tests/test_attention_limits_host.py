"""The largest launches and scales of the attention and cache calls, without a
GPU: a launch has fewer than 2^32 threads, and a call past that is refused as a
shape before anything runs.  At the limit the arguments pass every check and end
in TF_ERR_HIP, for no device is there."""

import pytest

from test_attention_host import HIP, SHAPE, UNSUPPORTED, call, needs_no_gpu

MOST = (2**32 - 1) // 256  # workgroups of 256 threads


@needs_no_gpu
@pytest.mark.parametrize("name", ["tf_attn_prefill", "tf_attn_prefill_paged"])
def test_prefill_workgroups(name):
    # 63 blocks of 128 rows (2000 tokens, 4 heads of a group), 8 key-value heads
    seqs = MOST // (63 * 8)
    assert call(name, seqs=seqs) == HIP
    assert call(name, seqs=seqs + 1) == SHAPE
    # 256 prompts of up to 131072 tokens, 64 / 8 heads: one workgroup too many
    many = dict(Hq=64, Hkv=8, T=1 << 20, longest=131072, q_token=64 * 128)
    assert call(name, seqs=255, **many) == HIP
    assert call(name, seqs=256, **many) == SHAPE


@needs_no_gpu
def test_append_workgroups():
    # a workgroup for 4 tokens
    assert call("tf_kv_append", T=4 * MOST) == HIP
    assert call("tf_kv_append", T=4 * MOST + 1) == SHAPE


@needs_no_gpu
def test_fork_workgroups():
    """The copies are the second of two launches: were it refused by the
    runtime, the first would have changed the references already."""
    big = dict(seqs=1000, ws_bytes=1 << 40)
    forks = (MOST - 1000) // 65  # 64 planes' copies and the child's row
    assert call("tf_kv_fork", planes=64, forks=forks, **big) == HIP
    assert call("tf_kv_fork", planes=64, forks=forks + 1, **big) == SHAPE
    assert call("tf_kv_fork", forks=0, seqs=MOST) == HIP
    assert call("tf_kv_fork", forks=0, seqs=MOST + 1) == SHAPE
    assert call("tf_kv_fork", planes=2**62, forks=2) == SHAPE


@needs_no_gpu
@pytest.mark.parametrize("name", ["tf_attn_decode", "tf_attn_prefill", "tf_attn_prefill_paged"])
def test_scale_times_log2_e_is_finite(name):
    assert call(name, scale=2.3e38) == HIP and call(name, scale=1e-45) == HIP
    assert call(name, scale=2.4e38) == UNSUPPORTED and call(name, scale=3.4e38) == UNSUPPORTED
