"""Linears split over K and attention calls of two kernels, from several host
threads on one stream: they share that stream's workspace, and nothing comes
between the kernels of a call."""

import threading

import pytest
import torch

import attention_ref as ref
import synth
from gpu_harness import gpu_or_skip, linear_fn, repack, to_device
from test_gpu_attention import _gen, _normal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROUNDS = 60


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _linears(q_):
    for bits, M, K, N, G in ((4, 40, 4096, 512, 128), (4, 130, 4096, 256, 128), (8, 300, 1024, 456, 128)):
        c = synth.make_inputs(bits, M, K, N, G, seed=(91, bits, M, K))
        d = to_device(c, torch)
        p, fn = repack(c, d, q_), linear_fn(q_, bits, True)
        assert q_.tf_workspace_bytes(bits, True, M, K, N, G) > 0
        yield lambda fn=fn, x=d["x"], p=p, a=(K, N, G), **kw: fn(x, p, *a, **kw)


def _attention(q_):
    hq, hkv, d, page = 8, 2, 128, 16
    g = _gen(61)
    for lens in ([3000], [700, 5000]):
        tables, pages = ref.tables_for(lens, page, g)
        q = _normal(g, (len(lens), hq, d), torch.bfloat16)
        kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
        t, n = tables.to(DEV), _ints(lens)
        assert q_.tf_attn_decode_workspace_bytes(len(lens), hq, hkv, d, max(lens)) > 0
        yield lambda a=(q, kp, vp, t, n, max(lens)), **kw: q_.tf_attn_decode(*a, **kw)
        cu = _ints(list(range(len(lens) + 1)))
        assert q_.tf_attn_prefill_workspace_bytes(len(lens), len(lens), hq, hkv, d, 1, tables.shape[1] * page) > 0
        yield lambda a=(q, kp, vp, t, cu, n, 1), **kw: q_.tf_attn_prefill_paged(*a, **kw)


def test_linears_and_attention_of_several_threads_on_one_stream():
    _, q_ = gpu_or_skip()
    calls = [*_linears(q_), *_attention(q_)]
    print("linears and attention from threads on one stream", flush=True)
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors, stream = [[] for _ in calls], [], torch.cuda.current_stream()
    start = threading.Barrier(len(calls), timeout=60)

    def work(i):
        try:
            start.wait()
            for _ in range(ROUNDS):
                got[i].append(calls[i](stream=stream))
        except Exception as exc:  # reported by the main thread
            errors.append(exc)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    torch.cuda.synchronize()
    assert not errors and not any(t.is_alive() for t in threads), errors
    for i, (want, outs) in enumerate(zip(alone, got)):
        assert len(outs) == ROUNDS and all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs), f"call {i}"
