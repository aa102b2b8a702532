"""The attention half of a layer's step as the header puts it together, against
64 bits from the unrotated QKV output on: append, then the prompts over the
pages, then single tokens."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip
from test_gpu_attention import _gen, _normal, _starts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _turn(x, angle):
    """x [n][heads][D] doubles, channels i and i + D / 2 turned by angle [n][D / 2]."""
    a, b = x.chunk(2, -1)
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _error(out, q, k, v, seen, scale, hkv, dtype):
    """out [n][Hq][D] against the definition on exact rotations: the largest
    error over its bound.  Beside the bound of the attention itself, the rotated
    queries and keys are rounded once and come from fp32 cosines, sines and
    products: each is off by e = h +
    2^-21 of the sum of its two products' sizes, at most sqrt(2) of the pair's
    length, so a score by 4 e S' with S' the scale times the product of the
    rows' lengths, and every weight by a factor of exp(8 e S') against the sum."""
    h = torch.finfo(dtype).eps / 2
    group, worst = q.shape[1] // hkv, 0.0
    for j in range(q.shape[1]):
        kk, vv = k[:, j // group], v[:, j // group]
        o, a, s = ref.attend(q[:, j], kk, vv, seen, scale)
        lengths = scale * q[:, j].norm(dim=1, keepdim=True) * kk.norm(dim=1).max()
        tol = ref.bound(o, a, s, q.shape[2], len(kk), dtype, float(vv.abs().max())) + a * torch.expm1(8 * (h + 2.0**-21) * lengths)
        worst = max(worst, float(((out[:, j].double() - o).abs() / tol).max()))
    return worst


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_append_then_attention_from_the_qkv_output_on(t):
    _, q_ = gpu_or_skip()
    hq, hkv, d, page, scale = 6, 2, 64, 16, 0.125
    lens, more = [70, 1, 133], 3
    g = _gen(71)
    total = [n + more for n in lens]
    tables, pages = ref.tables_for(total, page, g)
    tables = tables.to(DEV)
    kp, vp = (torch.full((pages, hkv, page, d), float("nan"), dtype=t, device=DEV) for _ in "kv")
    rate = 10000.0 ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    angle = torch.arange(max(total), device=DEV, dtype=torch.float64)[:, None] * rate
    rope = torch.cat([angle.cos(), angle.sin()], 1).float()
    fed = [_normal(g, (n, (hq + 2 * hkv) * d), t) for n in total]  # each sequence's QKV output

    def exact(s):
        x = fed[s].double().view(total[s], hq + 2 * hkv, d)
        turned = _turn(x[:, :hq + hkv], angle[:total[s]])
        return turned[:, :hq], turned[:, hq:], x[:, hq + hkv:]

    print("layer step: prompts", t, flush=True)
    qkv = torch.cat([f[:n] for f, n in zip(fed, lens)])
    kept = qkv.clone()
    seq, pos = [s for s, n in enumerate(lens) for _ in range(n)], [i for n in lens for i in range(n)]
    q = q_.tf_kv_append(qkv, rope, _ints(seq), _ints(pos), tables, kp, vp, hq)
    out = q_.tf_attn_prefill_paged(q, kp, vp, tables, _ints(_starts(lens)), _ints(lens), max(lens), scale)
    torch.cuda.synchronize()
    assert torch.equal(qkv, kept), "the QKV output is left as it was"
    at = _starts(lens)
    for s, n in enumerate(lens):
        qd, kd, vd = exact(s)
        seen, got = torch.arange(1, n + 1, device=DEV), out[at[s]:at[s + 1]]
        assert _error(got, qd[:n], kd[:n], vd[:n], seen, scale, hkv, t) <= 1.0
        if n > 1:  # the bound tells rotated keys from others
            plain = fed[s].double().view(total[s], -1, d)[:n, hq:hq + hkv]
            assert _error(got, qd[:n], plain, vd[:n], seen, scale, hkv, t) > 2.0
    for step in range(more):
        print("layer step: token", step, t, flush=True)
        now = [n + step + 1 for n in lens]
        qkv = torch.stack([f[n - 1] for f, n in zip(fed, now)])
        q = q_.tf_kv_append(qkv, rope, _ints(list(range(len(lens)))), _ints([n - 1 for n in now]), tables, kp, vp, hq)
        out = q_.tf_attn_decode(q, kp, vp, tables, _ints(now), max(now), scale)
        torch.cuda.synchronize()
        for s, n in enumerate(now):
            qd, kd, vd = exact(s)
            assert _error(out[s:s + 1], qd[n - 1:n], kd[:n], vd[:n], torch.tensor([n], device=DEV), scale, hkv, t) <= 1.0


def test_the_example_says_when_no_page_is_free():
    import importlib.util
    import os

    from conftest import ROOT

    gpu_or_skip()
    spec = importlib.util.spec_from_file_location("serve_decoder", os.path.join(ROOT, "examples", "serve_decoder.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cache = example.Cache(layers=1, pages=2, hkv=1, page=16, d=64, seqs=2, width=4)
    cache.reserve({0: 20})
    with pytest.raises(RuntimeError, match="no page is free"):
        cache.reserve({1: 1})
    # what was there before is as it was
    assert cache.lens.tolist() == [20, 0] and cache.refs.tolist() == [1, 1] and cache.tables[1].tolist() == [-1] * 4
