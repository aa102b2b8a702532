"""Prompts over tables as wide as a model's longest context, with lengths far
below it: the work is planned for what the table can name, in up to 16 ranges of
keys of which most are empty, and gives what a table of the lengths' own width
gives."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip
from test_gpu_attention import _check_prefill, _gen, _normal, _starts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,nkeys,heads,page,context", [
    ([5], [5], (8, 1, 128), 16, 131072), ([1, 0, 3], [1, 0, 260], (28, 4, 128), 64, 131072),
    ([100, 64, 65, 1], [100, 64, 300, 1000], (8, 2, 64), 16, 32768), ([500], [500], (32, 8, 128), 128, 131072),
    # the batch would run side by side with tight tables, and does not with these
    ([600, 0, 17, 250, 430, 599, 1], [600, 0, 17, 250, 430, 599, 1], (32, 2, 64), 16, 131072),
])
def test_prefill_over_tables_far_wider_than_the_lengths(new, nkeys, heads, page, context, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    print(f"wide tables {t} {heads} new {new} keys {nkeys} context {context}", flush=True)
    g = _gen(sum(new) + 5 * sum(nkeys) + hq)
    wide, pages = ref.tables_for(nkeys, page, g, width=context // page, fill=2**31 - 1)
    tight = wide[:, :max(-(-n // page) for n in nkeys)].contiguous()
    cu = _starts(new)
    q = _normal(g, (sum(new), hq, d), t, 1.5)
    kp, vp = (_normal(g, (pages, hkv, page, d), t) for _ in "kv")
    few = hkv * sum(-(-n * (hq // hkv) // 128) for n in new) <= 100
    assert not few or q_.tf_attn_prefill_workspace_bytes(len(new), sum(new), hq, hkv, d, max(new), context) > 0
    for tables in (wide, tight):
        out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(cu), _ints(nkeys), max(new))
        torch.cuda.synchronize()
        _check_prefill(q, lambda s, h: (ref.gather(kp, tight[s], nkeys[s], h), ref.gather(vp, tight[s], nkeys[s], h)), cu, nkeys,
                       hkv, d ** -0.5, out)
