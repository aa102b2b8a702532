"""Prefill with all sequences side by side: a workgroup finds its sequence and
block by a search over the levels of blocks, one step of 64 levels or two.  The
sizes are checked against the rule that chooses this order, whole and with a
bound below the longest."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip
from test_gpu_attention import _check_prefill, _gen, _normal, _starts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _levels(seqs, heads, longest, keys):
    """Blocks of the longest sequence if the sequences run side by side (keys: of a sequence on average), else 0."""
    hq, hkv, d = heads
    blocks = -(-longest * (hq // hkv) // 128)
    fits = seqs * (hkv if hkv % 8 else hkv // 8) * keys * 4 * d <= 3 << 20
    return blocks if 1 < seqs <= 64 and hkv * seqs * blocks > 512 and fits else 0


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("lens,heads,bound", [
    # at most 64 levels: one step
    ([512, 513, 511, 1, 0, 300, 16, 17, 430, 128], (16, 2, 64), 460),
    # more: two steps, which the bound keeps
    ([600, 0, 17, 250, 430, 599, 1], (32, 2, 64), 519),
    # two steps, and one with the bound
    ([90, 545, 33, 0, 544, 64, 300, 1, 520], (32, 2, 64), 500),
])
def test_prefill_side_by_side(lens, heads, bound, paged, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    page, n = 16, len(lens)
    print(f"prefill side by side {t} paged={paged} {heads} {n} sequences", flush=True)
    g = _gen(sum(lens) + hq)
    cu = _starts(lens)
    q = _normal(g, (sum(lens), hq, d), t, 1.5)
    if paged:
        tables, pages = ref.tables_for(lens, page, g)
        kp, vp = (_normal(g, (pages, hkv, page, d), t) for _ in "kv")
        keys = tables.shape[1] * page

        def call(longest, **kw):
            return q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(cu), _ints(lens), longest, **kw)

        def keys_of(s, h):
            return ref.gather(kp, tables[s], lens[s], h), ref.gather(vp, tables[s], lens[s], h)
    else:
        k, v = (_normal(g, (sum(lens), hkv, d), t) for _ in "kv")
        keys = -(-sum(lens) // n)

        def call(longest, **kw):
            return q_.tf_attn_prefill(q, k, v, _ints(cu), _ints(cu), longest, **kw)

        def keys_of(s, h):
            return k[cu[s]:cu[s + 1], h].double(), v[cu[s]:cu[s + 1], h].double()
    whole, part = _levels(n, heads, max(lens), keys), _levels(n, heads, bound, keys)
    assert whole and part and (whole > 64, part > 64) == {460: (False, False), 519: (True, True), 500: (True, False)}[bound]
    out = call(max(lens))
    torch.cuda.synchronize()
    _check_prefill(q, keys_of, cu, lens, hkv, d ** -0.5, out)
    given = torch.full_like(q, 7.0)
    call(bound, out=given)
    torch.cuda.synchronize()
    for s, m in enumerate(lens):
        m = min(m, bound)
        assert torch.equal(given[cu[s]:cu[s] + m], out[cu[s]:cu[s] + m]) and bool((given[cu[s] + m:cu[s + 1]] == 7.0).all())
