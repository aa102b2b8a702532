"""Scores so large that their rounding steps are whole powers of two: the
largest score's weight is 1 whatever its rounding, rows whose scores all are a
type's lowest value weigh their keys alike, and other rows beside them are as
ever."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip
from test_gpu_attention import _gen, _normal, _starts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _inputs(g, n, rows, d, t, size):
    """q [rows][4][D], k and v [n][1][D] of one key-value head.  Heads 0 and 1
    read channel 0 alone, whose products are exact in fp32: scores of up to
    +-size, 1/64 of it apart or equal.  Head 2 has scores of the lowest size
    only (channel 1), head 3 ordinary ones (the other channels)."""
    root = 2.0 ** (torch.tensor(size).log2().item() // 2)
    q = torch.zeros((rows, 4, d))
    q[:, 0, 0], q[:, 1, 0], q[:, 2, 1] = root, -root, root
    q[:, 3, 2:] = torch.randn((rows, d - 2), generator=g)
    k = torch.randn((n, 1, d), generator=g)
    k[..., 0] = (size / root) * (torch.randint(-32, 33, (n, 1), generator=g) / 64 + 1)
    k[..., 1] = -size / root * 1.5
    q, k = q.to(t).to(DEV), k.to(t).to(DEV)
    assert bool(torch.isfinite(k).all()) and bool(torch.isfinite(q).all())
    return q, k, _normal(g, (n, 1, d), t)


def _check(out, q, k, v, seen):
    """q, out [R][4][D]; k, v [n][D] doubles.  The first three heads' scores are exact, or equal: no error of theirs
    enters the bound."""
    for j in range(4):
        o, a, s = ref.attend(q[:, j].double(), k, v, seen, 1.0)
        ref.check(out[:, j], o, a, s if j == 3 else torch.zeros_like(s), len(k), float(v.abs().max()))


# 2^20 .. 2^32 for fp16, whose products end there; bf16 also far past a step of 2^8
SIZES = [("f16", 2.0**e * f) for e in (20, 22, 23, 24, 25, 26, 28, 30) for f in (1.0, 1.171875)]
SIZES += [("bf16", 2.0**e * f) for e in (20, 24, 28, 31, 32, 34, 40, 60, 100) for f in (1.0, 1.171875)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t,size", SIZES)
def test_large_scores(t, size, d):
    _, q_ = gpu_or_skip()
    page = 16
    print(f"large scores {t} {size:.3g} D {d}", flush=True)
    g = _gen(int(torch.tensor(size).log2()) + d)
    # a single token: a workgroup per item, shares
    for n in (1, 300, 3001):
        q, k, v = _inputs(g, n, 1, d, TYPES[t], size)
        tables, pages = ref.tables_for([n], page, g)
        kp, vp = (torch.zeros((pages, 1, page, d), dtype=TYPES[t], device=DEV) for _ in "kv")
        for x, p in ((k, kp), (v, vp)):
            for c in range(-(-n // page)):
                m = min(page, n - c * page)
                p[int(tables[0, c]), 0, :m] = x[c * page:c * page + m, 0]
        out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), _ints([n]), n, 1.0)
        torch.cuda.synchronize()
        _check(out, q, k[:, 0].double(), v[:, 0].double(), torch.tensor([n], device=DEV))
    # prompts: packed whole, and few rows over pages behind many keys, in ranges
    q, k, v = _inputs(g, 200, 200, d, TYPES[t], size)
    out = q_.tf_attn_prefill(q, k, v, _ints([0, 200]), _ints([0, 200]), 200, 1.0)
    torch.cuda.synchronize()
    _check(out, q, k[:, 0].double(), v[:, 0].double(), torch.arange(1, 201, device=DEV))
    n, new = 3001, 40
    q = _inputs(g, 1, new, d, TYPES[t], size)[0]
    k, v = (ref.gather(p, tables[0], n, 0) for p in (kp, vp))
    assert q_.tf_attn_prefill_workspace_bytes(1, new, 4, 1, d, new, tables.shape[1] * page) > 0
    out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(_starts([new])), _ints([n]), new, 1.0)
    torch.cuda.synchronize()
    _check(out, q, k, v, torch.arange(n - new + 1, n + 1, device=DEV))
