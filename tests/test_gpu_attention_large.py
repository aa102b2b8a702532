"""The attention and cache calls where offsets pass 32 bits and where a batch
has more sequences than a workgroup has threads."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip
from test_gpu_attention import _check_decode, _check_prefill, _gen, _normal, _starts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("heads,longest", [((2, 1, 64), 2500), ((6, 2, 128), 1400)])
def test_decode_of_many_sequences(heads, longest):
    """1300 sequences, most of them short, some empty, a few long: a thread
    takes several sequences, a share holds many."""
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    n, page = 1300, 16
    g = _gen(51)
    lens = torch.randint(0, 40, (n,), generator=g).tolist()
    for s, m in ((0, 0), (3, longest), (511, longest - 1), (512, 0), (777, 1025), (1298, longest), (1299, 0)):
        lens[s] = m
    tables, pages = ref.tables_for(lens, page, g)
    q = _normal(g, (n, hq, d), torch.bfloat16, 1.5)
    kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
    assert q_.tf_attn_decode_workspace_bytes(n, hq, hkv, d, longest) > 0
    print("decode many", heads, flush=True)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), _ints(lens), longest)
    torch.cuda.synchronize()
    pick = sorted({0, 3, 4, 510, 511, 512, 513, 776, 777, 778, 1297, 1298, 1299} | set(range(0, n, 13)))
    _check_decode(q[pick], kp, vp, tables[pick], [lens[s] for s in pick], d ** -0.5, out[pick])
    empty = [s for s in range(n) if lens[s] == 0]
    assert bool((out[empty] == 0).all())


def test_pages_past_32_bits():
    """A plane of 2.3e9 values: appending, decoding, prompts behind a cache,
    forking and compacting at pages near its end."""
    _, q_ = gpu_or_skip()
    _room(24)
    hq, hkv, d, page, pages = 8, 2, 128, 128, 70000
    g = _gen(52)
    planes = torch.zeros((2, pages, hkv, page, d), dtype=torch.bfloat16, device=DEV)
    kp, vp = planes[0], planes[1]
    assert kp.numel() > 2**31
    lens = [300, 129, 0]
    tables = torch.tensor([[69999, 5, 68000], [67000, 69998, -1], [-1, -1, -1]], dtype=torch.int32)
    for s, n in enumerate(lens):
        for c in range(-(-n // page)):
            for p in (kp, vp):
                p[int(tables[s, c])] = _normal(g, (hkv, page, d), torch.bfloat16)
    q = _normal(g, (3, hq, d), torch.bfloat16, 1.5)
    print("decode past 32 bits", flush=True)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), _ints(lens), 384)
    torch.cuda.synchronize()
    _check_decode(q, kp, vp, tables, lens, d ** -0.5, out)
    print("prefill past 32 bits", flush=True)
    new = [40, 129, 0]
    q = _normal(g, (169, hq, d), torch.bfloat16, 1.5)
    out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(_starts(new)), _ints(lens), 129)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (ref.gather(kp, tables[s], lens[s], h), ref.gather(vp, tables[s], lens[s], h)), _starts(new),
                   lens, hkv, d ** -0.5, out)
    print("append past 32 bits", flush=True)
    qkv = _normal(g, (2, (hq + 2 * hkv) * d), torch.bfloat16)
    rope = torch.cat([torch.ones(400, d // 2), torch.zeros(400, d // 2)], 1).to(DEV)  # no turn
    q_.tf_kv_append(qkv, rope, _ints([0, 1]), _ints([299, 130]), tables.to(DEV), kp, vp, hq)
    torch.cuda.synchronize()
    x = qkv.view(2, -1, d)
    assert torch.equal(kp[68000, :, 43], x[0, hq:hq + hkv]) and torch.equal(vp[68000, :, 43], x[0, hq + hkv:])
    assert torch.equal(kp[69998, :, 2], x[1, hq:hq + hkv]) and torch.equal(vp[69998, :, 2], x[1, hq + hkv:])
    print("fork and compact past 32 bits", flush=True)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[:67000] = 1  # the lowest free page is 67001
    refs[[67000, 68000, 69998, 69999]] = 1
    t, n = tables.to(DEV), _ints(lens)
    status = q_.tf_kv_fork(planes, refs, t, n, _ints([0]), _ints([2]))
    torch.cuda.synchronize()
    assert status.tolist() == [0] and t[2].tolist() == [69999, 5, 67001] and n.tolist() == [300, 129, 300]
    assert torch.equal(planes[:, 67001, :, :44], planes[:, 68000, :, :44]) and not bool(planes[:, 67001, :, 44:].any())
    kept = planes[:, 69999].clone()
    refs[:4000] = 0  # so that the last ones move
    refs[5] = 2
    q_.tf_kv_compact(planes, refs, t)
    torch.cuda.synchronize()
    live = int((refs > 0).sum())
    assert int(t.max()) < live and bool((refs[:live] > 0).all())
    assert torch.equal(planes[:, int(t[0, 0])], kept) and int(t[0, 1]) == 5


def test_strides_past_32_bits():
    """Packed prompts whose token strides put their last rows past 2^31 values."""
    _, q_ = gpu_or_skip()
    _room(8)
    hq, hkv, d, n, step = 4, 2, 64, 40, 60_000_000
    g = _gen(53)
    flat = torch.empty(step * (n - 1) + (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=DEV)
    assert flat.numel() > 2**31
    qkv = flat.as_strided((n, hq + 2 * hkv, d), (step, d, 1))
    qkv.copy_(_normal(g, (n, hq + 2 * hkv, d), torch.bfloat16))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    print("strides past 32 bits", flush=True)
    cu = _ints([0, n])
    out = q_.tf_attn_prefill(q, k, v, cu, cu, n)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (k[:, h].double(), v[:, h].double()), [0, n], [n], hkv, d ** -0.5, out)


def test_a_captured_layer_of_calls():
    """Append, decode in shares and a prompt in ranges captured together,
    replayed with new inputs between eager calls."""
    _, q_ = gpu_or_skip()
    hq, hkv, d, page = 8, 1, 128, 16
    lens, new = [3000, 900], [1, 1]
    g = _gen(54)
    tables, pages = ref.tables_for(lens, page, g)
    kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
    qkv = _normal(g, (2, (hq + 2 * hkv) * d), torch.bfloat16)
    rope = torch.randn((3000, d), generator=g).to(DEV)
    t, n, cu = tables.to(DEV), _ints(lens), _ints(_starts(new))
    seq, pos = _ints([0, 1]), _ints([2999, 899])
    assert q_.tf_attn_decode_workspace_bytes(2, hq, hkv, d, 3000) > 0
    assert q_.tf_attn_prefill_workspace_bytes(2, 2, hq, hkv, d, 1, tables.shape[1] * page) > 0

    def step():
        q = q_.tf_kv_append(qkv, rope, seq, pos, t, kp, vp, hq)
        return q, q_.tf_attn_decode(q, kp, vp, t, n, 3000), q_.tf_attn_prefill_paged(q, kp, vp, t, cu, n, 1)

    print("captured layer", flush=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    torch.cuda.synchronize()
    for it in range(4):
        qkv.copy_(torch.roll(qkv, 7, 1))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {it} differs"
        # a single new token of each sequence sees every key: both calls say the same, up to the roundings of p and o
        assert bool((got[1].float() - got[2].float()).abs().max() <= 2.0**-6)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("lens,heads", [
    # more workgroups than run at once, all sequences side by side: 75 levels of blocks, one and two steps of the search
    ([600, 0, 17, 250, 430], (32, 2, 64)), ([512, 513, 511, 1, 0, 300], (16, 2, 64)),
    # as many sequences as a wave has lanes, and one more, which run in turn
    ([1 + 7 * s % 41 for s in range(64)], (64, 8, 128)), ([1 + 7 * s % 41 for s in range(65)], (64, 8, 128)),
])
def test_prefill_of_many_blocks(lens, heads, paged, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    page = 16
    print(f"prefill many blocks {t} paged={paged} {heads} {len(lens)} sequences", flush=True)
    g = _gen(sum(lens) + hq)
    cu = _starts(lens)
    q = _normal(g, (sum(lens), hq, d), t, 1.5)
    if paged:
        tables, pages = ref.tables_for(lens, page, g)
        kp, vp = (_normal(g, (pages, hkv, page, d), t) for _ in "kv")
        out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(cu), _ints(lens), max(lens))

        def keys_of(s, h):
            return ref.gather(kp, tables[s], lens[s], h), ref.gather(vp, tables[s], lens[s], h)
    else:
        k, v = (_normal(g, (sum(lens), hkv, d), t) for _ in "kv")
        out = q_.tf_attn_prefill(q, k, v, _ints(cu), _ints(cu), max(lens))

        def keys_of(s, h):
            return k[cu[s]:cu[s + 1], h].double(), v[cu[s]:cu[s + 1], h].double()
    torch.cuda.synchronize()
    _check_prefill(q, keys_of, cu, lens, hkv, d ** -0.5, out)
    # a bound below the longest: its rows and no others change nothing
    bound, given = max(lens) // 2, torch.full_like(q, 7.0)
    if paged:
        q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), _ints(cu), _ints(lens), bound, out=given)
    else:
        q_.tf_attn_prefill(q, k, v, _ints(cu), _ints(cu), bound, out=given)
    torch.cuda.synchronize()
    for s, n in enumerate(lens):
        m = min(n, bound)
        assert torch.equal(given[cu[s]:cu[s] + m], out[cu[s]:cu[s] + m]) and bool((given[cu[s] + m:cu[s + 1]] == 7.0).all())
