"""The stride of an axis of one entry means nothing: a single token's queries,
or a single key, taken out of a larger tensor."""

import pytest
import torch

from gpu_harness import gpu_or_skip
from test_gpu_attention import _gen, _normal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("stride", [2**26, 2**31, 100, 8193, 1])
def test_a_single_token_of_any_stride(stride):
    _, q_ = gpu_or_skip()
    hq, hkv, d, page, n = 8, 2, 64, 16, 40
    g = _gen(81)
    print("single token of stride", stride, flush=True)
    q, k, v = (_normal(g, (1, h, d), torch.bfloat16) for h in (hq, hkv, hkv))
    kp, vp = (_normal(g, (3, hkv, page, d), torch.bfloat16) for _ in "kv")
    t, cu, lens = _ints([[2, 0, 1]]), _ints([0, 1]), _ints([n])
    odd = [x.as_strided(x.shape, (stride, d, 1)) for x in (q, k, v)]

    def calls(q, k, v):
        return (q_.tf_attn_decode(q, kp, vp, t, lens, n), q_.tf_attn_prefill(q, k, v, cu, cu, 1),
                q_.tf_attn_prefill_paged(q, kp, vp, t, cu, lens, 1))

    for a, b in zip(calls(q, k, v), calls(*odd)):
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_the_last_token_of_a_long_prompt_decodes_in_place():
    """[1][T][Hq][D] with T Hq D = 2^26: the last token's queries are a view whose first stride is that."""
    _, q_ = gpu_or_skip()
    hq, hkv, d, page, n = 32, 8, 128, 64, 500
    g = _gen(82)
    every = torch.zeros((1, 16384, hq, d), dtype=torch.float16, device=DEV)
    every[0, -1] = _normal(g, (hq, d), torch.float16)
    last = every[:, -1]
    assert last.stride(0) == 2**26
    kp, vp = (_normal(g, (8, hkv, page, d), torch.float16) for _ in "kv")
    print("last token in place", flush=True)
    a, b = (q_.tf_attn_decode(x, kp, vp, _ints([list(range(8))]), _ints([n]), n) for x in (last, last.clone()))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
