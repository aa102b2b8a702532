"""Attention over a paged cache and over packed prompts, on the GPU against the
definition in 64 bits; bounds derived in attention_ref."""

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _normal(g, shape, t, gain=1.0):
    return (torch.randn(shape, generator=g) * gain).to(t).to(DEV)


def _check_decode(q, kp, vp, tables, lens, scale, out):
    hq, hkv = q.shape[1], kp.shape[1]
    rows = tables.cpu()
    for s, n in enumerate(lens):
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            k, v = ref.gather(kp, rows[s], n, h), ref.gather(vp, rows[s], n, h)
            seen = torch.full((hq // hkv,), n, device=DEV)
            o, a, big = ref.attend(q[s, heads].double(), k, v, seen, scale)
            ref.check(out[s, heads], o, a, big, n, float(v.nan_to_num(0, 0, 0).abs().max()) if n else 0.0)


DECODE = [
    # lengths, (Hq, Hkv, D), page: around the tiles of 16 and 32 keys, the round of 256, empty and single tokens
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], (32, 8, 128), 16),
    ([255, 256, 257, 511, 512], (28, 4, 128), 32),
    ([333], (32, 8, 128), 16),
    ([1, 0, 700], (8, 1, 128), 64),
    ([47, 300, 5], (12, 12, 64), 128),
    ([129, 1030], (71, 1, 64), 32),
    ([77, 600], (40, 2, 128), 16),
    ([530, 90], (48, 1, 128), 16),
    ([100, 900], (14, 2, 64), 1024),
    # split over the length and joined: ragged chunks, sequences that end before the last chunk
    ([5000, 0, 1, 1024, 513], (64, 8, 128), 64),
    ([20001], (14, 2, 64), 16),
    ([9000, 8192], (32, 32, 128), 16),
    ([3001, 2999], (71, 1, 64), 16),
]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("lens,heads,page", DECODE)
def test_decode(lens, heads, page, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    print(f"decode {t} {heads} page {page} lens {lens}", flush=True)
    g = _gen(len(lens) * 1000 + sum(lens) + hq)
    tables, pages = ref.tables_for(lens, page, g)
    q = _normal(g, (len(lens), hq, d), TYPES[t], 1.5)
    kp, vp = (_normal(g, (pages, hkv, page, d), TYPES[t]) for _ in "kv")
    dev = [torch.tensor(lens, dtype=torch.int32, device=DEV), tables.to(DEV)]
    out = q_.tf_attn_decode(q, kp, vp, dev[1], dev[0], max(lens), d ** -0.5)
    torch.cuda.synchronize()
    _check_decode(q, kp, vp, tables, lens, d ** -0.5, out)
    again = q_.tf_attn_decode(q, kp, vp, dev[1], dev[0], max(lens))
    assert torch.equal(out, again), "two runs differ"


def test_decode_reads_nothing_past_the_lengths():
    """Stale rows of a last page, spare pages and table entries past a length
    hold NaN, infinities and ids of no page; a strided q; a bound of the
    lengths well above them; an own scale."""
    _, q_ = gpu_or_skip()
    lens, (hq, hkv, d), page = [37, 0, 300, 16, 1500], (16, 4, 128), 32
    g = _gen(5)
    tables, pages = ref.tables_for(lens, page, g, width=60, fill=10**9)
    kp, vp = (torch.full((pages, hkv, page, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    vp[..., ::2] = float("inf")
    for s, n in enumerate(lens):
        for c in range(-(-n // page)):
            m = min(page, n - c * page)
            for p in (kp, vp):
                p[int(tables[s, c]), :, :m] = _normal(g, (hkv, m, d), torch.bfloat16)
    qkv = _normal(g, (len(lens), hq + 2 * hkv, d), torch.bfloat16)
    q = qkv[:, :hq]
    print("decode stale rows", flush=True)
    for longest in (1500, 1920, 60 * 32):
        out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), longest, 0.31)
        torch.cuda.synchronize()
        _check_decode(q, kp, vp, tables, lens, 0.31, out)


def test_decode_pages_that_do_not_exist_and_lengths_past_the_bound():
    """Ids outside the pool read as zeros; lengths are clamped to the bound and
    to what the table can name, negative ones to zero."""
    _, q_ = gpu_or_skip()
    lens, (hq, hkv, d), page = [200, 100, 64], (8, 2, 64), 16
    g = _gen(6)
    tables, pages = ref.tables_for(lens, page, g, width=13)
    tables[0, 3], tables[0, 7], tables[1, 0], tables[2, 2] = -1, pages, 2**31 - 1, -(2**31)
    q = _normal(g, (3, hq, d), torch.float16)
    kp, vp = (_normal(g, (pages, hkv, page, d), torch.float16) for _ in "kv")
    print("decode bad pages", flush=True)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), 208, 0.125)
    torch.cuda.synchronize()
    _check_decode(q, kp, vp, tables, lens, 0.125, out)
    print("decode long lengths", flush=True)
    claimed = torch.tensor([2**31 - 1, -7, 150], dtype=torch.int32, device=DEV)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), claimed, 10**6, 0.125)
    torch.cuda.synchronize()
    _check_decode(q, kp, vp, tables, [208, 0, 150], 0.125, out)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), claimed, 40, 0.125)
    torch.cuda.synchronize()
    _check_decode(q, kp, vp, tables, [40, 0, 40], 0.125, out)


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_decode_sharp_and_growing_scores(t):
    """Scores that grow along the cache by hundreds (the running maximum is
    replaced again and again), a single dominating key, and scores of the
    lowest value a type has."""
    _, q_ = gpu_or_skip()
    n, (hq, hkv, d), page = 3000, (8, 2, 128), 16
    g = _gen(7)
    tables, pages = ref.tables_for([n, n, n], page, g)
    q = _normal(g, (3, hq, d), TYPES[t])
    kp, vp = (_normal(g, (pages, hkv, page, d), TYPES[t]) for _ in "kv")
    q[0], q[2] = q[0].abs() + 0.5, 1.0
    for c in range(-(-n // page)):
        kp[int(tables[0, c])] = (kp[int(tables[0, c])].float() * 0.1 + 0.02 * c).to(TYPES[t])
    kp[int(tables[1, 100]), :, 3] = 30.0 * torch.sign(q[1, ::hq // hkv])
    kp[int(tables[2, 5])] = torch.finfo(TYPES[t]).min
    lens = torch.full((3,), n, dtype=torch.int32, device=DEV)
    print("decode sharp", t, flush=True)
    out = q_.tf_attn_decode(q, kp, vp, tables.to(DEV), lens, n, 0.5)
    torch.cuda.synchronize()
    if t == "f16":  # sums of 128 fp16 minima stay in fp32; bf16's overflow to -inf, weight zero either way
        _check_decode(q, kp, vp, tables, [n, n, n], 0.5, out)
    else:
        _check_decode(q[:2], kp, vp, tables[:2], [n, n], 0.5, out[:2])
        assert bool(torch.isfinite(out[2]).all())


def _check_prefill(q, keys_of, cu_q, nkeys, hkv, scale, out):
    hq = q.shape[1]
    group = hq // hkv
    for s, n in enumerate(nkeys):
        a0, a1 = cu_q[s], cu_q[s + 1]
        if a1 == a0:
            continue
        seen = (n - (a1 - a0) + 1 + torch.arange(a1 - a0, device=DEV)).clamp(0, n)
        for h in range(hkv):
            k, v = keys_of(s, h)
            for j in range(h * group, (h + 1) * group):
                o, a, big = ref.attend(q[a0:a1, j].double(), k, v, seen, scale)
                ref.check(out[a0:a1, j], o, a, big, n, float(v.nan_to_num(0, 0, 0).abs().max()) if n else 0.0)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


PREFILL = [
    # new tokens, earlier tokens, (Hq, Hkv, D), page
    ([1, 2, 3, 31, 32, 33], [0] * 6, (32, 8, 128), 16),
    ([63, 0, 64, 65, 1], [0] * 5, (28, 4, 128), 32),
    ([77], [0], (14, 2, 64), 16),
    ([127, 129, 128], [0] * 3, (12, 12, 64), 64),
    ([200], [0], (71, 1, 64), 16),
    ([300, 5], [0, 0], (8, 1, 128), 128),
    ([64, 100, 1, 17], [0, 333, 500, 16], (64, 8, 128), 16),
    ([33, 400], [1000, 15], (40, 8, 128), 1024),
    ([513], [300], (32, 32, 128), 16),
    ([1, 1, 1], [0, 63, 64], (16, 1, 64), 16),
]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("new,old,heads,page", PREFILL)
def test_prefill(new, old, heads, page, paged, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    print(f"prefill {t} paged={paged} {heads} page {page} new {new} old {old}", flush=True)
    g = _gen(sum(new) + 7 * sum(old) + hq)
    nkeys = [a + b for a, b in zip(new, old)]
    cu = _starts(new)
    cu_q = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if paged:
        q = _normal(g, (sum(new), hq, d), TYPES[t], 1.5)
        tables, pages = ref.tables_for(nkeys, page, g)
        kp, vp = (_normal(g, (pages, hkv, page, d), TYPES[t]) for _ in "kv")
        out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), cu_q, torch.tensor(nkeys, dtype=torch.int32, device=DEV),
                                       max(new))

        def keys_of(s, h):
            return ref.gather(kp, tables[s], nkeys[s], h), ref.gather(vp, tables[s], nkeys[s], h)
    else:
        # parts of fused outputs: token strides wider than the heads
        ck = _starts(nkeys)
        q = _normal(g, (sum(new), hq + 3, d), TYPES[t], 1.5)[:, 1:hq + 1]
        kv = _normal(g, (sum(nkeys), 2 * hkv + 1, d), TYPES[t])
        k, v = kv[:, :hkv], kv[:, hkv + 1:]
        out = q_.tf_attn_prefill(q, k, v, cu_q, torch.tensor(ck, dtype=torch.int32, device=DEV), max(new))

        def keys_of(s, h):
            return k[ck[s]:ck[s + 1], h].double(), v[ck[s]:ck[s + 1], h].double()
    torch.cuda.synchronize()
    _check_prefill(q, keys_of, cu, nkeys, hkv, d ** -0.5, out)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_hidden_infinities_do_not_spread(t, d):
    """NaN and infinities in keys and values: rows that see them show them, rows
    that do not are as if they were not there.  Also more queries than keys
    (rows that see nothing are zero) and head-major strides."""
    _, q_ = gpu_or_skip()
    new, nkeys, hq, hkv = [150, 40, 9], [150, 13, 200], 6, 2
    g = _gen(11)
    cu, ck = _starts(new), _starts(nkeys)
    q = _normal(g, (hq, sum(new), d), TYPES[t]).transpose(0, 1)
    k = _normal(g, (hkv, sum(nkeys), d), TYPES[t]).transpose(0, 1)
    v = _normal(g, (hkv, sum(nkeys), d), TYPES[t]).transpose(0, 1)
    inf = float("inf")
    v[100, 0, 3], v[120, 0, 3], v[100, 1, 5], v[130, 1, 5], v[149, 0, 7] = inf, -inf, -inf, float("nan"), inf
    v[ck[1] + 12, 1, 9], v[ck[2] + 195, 0, 0], v[ck[2] + 199, 1, 1] = float("nan"), inf, -inf
    print("prefill hidden infinities", t, d, flush=True)
    ints = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cu, ck)]
    out = q_.tf_attn_prefill(q, k, v, *ints, 150, 0.2)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (k[ck[s]:ck[s + 1], h].double(), v[ck[s]:ck[s + 1], h].double()), cu, nkeys, hkv, 0.2, out)
    # a NaN key: rows before it are untouched, bit for bit
    k2 = k.clone()
    k2[140, :, 0] = float("nan")
    bad = q_.tf_attn_prefill(q, k2, v, *ints, 150, 0.2)
    torch.cuda.synchronize()
    assert torch.equal(bad[:140].view(torch.int16), out[:140].view(torch.int16))
    assert bool(torch.isnan(bad[140:150]).all())


def test_prefill_clamps_what_the_device_tensors_claim():
    """Row and key offsets past the tensors are clamped; pages that do not
    exist read as zeros; tokens past the bound are not computed."""
    _, q_ = gpu_or_skip()
    hq, hkv, d, page = 4, 2, 64, 16
    g = _gen(12)
    q = _normal(g, (50, hq, d), torch.bfloat16)
    kv = _normal(g, (60, 2 * hkv, d), torch.bfloat16)
    k, v = kv[:, :hkv], kv[:, hkv:]
    print("prefill clamped offsets", flush=True)
    cu_q, cu_k = ([0, 20, 10**9], [0, 25, 2**31 - 1])
    out = q_.tf_attn_prefill(q, k, v, torch.tensor(cu_q, dtype=torch.int32, device=DEV),
                             torch.tensor(cu_k, dtype=torch.int32, device=DEV), 50)
    torch.cuda.synchronize()
    cu, ck = [0, 20, 50], [0, 25, 60]
    _check_prefill(q, lambda s, h: (k[ck[s]:ck[s + 1], h].double(), v[ck[s]:ck[s + 1], h].double()), cu, [25, 35], hkv,
                   d ** -0.5, out)
    print("prefill bad pages", flush=True)
    tables, pages = ref.tables_for([100], page, g, width=8)
    tables[0, 1], tables[0, 4], tables[0, 6] = -5, pages + 3, 2**31 - 1
    kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
    out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), torch.tensor([0, 50], dtype=torch.int32, device=DEV),
                                   torch.tensor([100], dtype=torch.int32, device=DEV), 50)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (ref.gather(kp, tables[0], 100, h), ref.gather(vp, tables[0], 100, h)), [0, 50], [100],
                   hkv, d ** -0.5, out)
    print("prefill rows past the bound", flush=True)
    given = torch.full((50, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), torch.tensor([0, 50], dtype=torch.int32, device=DEV),
                             torch.tensor([100], dtype=torch.int32, device=DEV), 12, out=given)
    torch.cuda.synchronize()
    assert bool((given[12:] == 7.0).all()) and not bool((given[:12] == 7.0).any())


def test_empty_calls():
    _, q_ = gpu_or_skip()
    t = torch.bfloat16
    kp = torch.zeros((3, 2, 16, 64), dtype=t, device=DEV)
    none = torch.zeros((0,), dtype=torch.int32, device=DEV)
    out = q_.tf_attn_decode(torch.zeros((0, 4, 64), dtype=t, device=DEV), kp, kp, none.view(0, 1)[:, :1].reshape(0, 1), none, 0)
    assert out.shape == (0, 4, 64)
    zero = torch.zeros((1,), dtype=torch.int32, device=DEV)
    out = q_.tf_attn_prefill(torch.zeros((0, 4, 64), dtype=t, device=DEV), kp[0, 0, :0].reshape(0, 2, 64), kp[0, 0, :0].reshape(0, 2, 64), zero, zero, 0)
    assert out.shape == (0, 4, 64)
    # queries without a key
    q = torch.ones((5, 4, 64), dtype=t, device=DEV)
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    out = q_.tf_attn_prefill(q, q[:0, :2], q[:0, :2], cu, torch.zeros_like(cu), 5)
    torch.cuda.synchronize()
    assert bool((out == 0).all())


def test_other_streams_and_graphs():
    """Calls on a stream of their own, given and current, and a captured decode
    step replayed between eager calls."""
    _, q_ = gpu_or_skip()
    lens, (hq, hkv, d), page = [3000, 70, 0, 900], (32, 8, 128), 16
    g = _gen(13)
    tables, pages = ref.tables_for(lens, page, g)
    q = _normal(g, (4, hq, d), torch.bfloat16)
    kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
    tables, n = tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    eager = q_.tf_attn_decode(q, kp, vp, tables, n, 3000)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    given = q_.tf_attn_decode(q, kp, vp, tables, n, 3000, stream=s)
    s.synchronize()
    assert torch.equal(given, eager)
    out = torch.empty_like(q)
    with torch.cuda.stream(s):
        q_.tf_attn_decode(q, kp, vp, tables, n, 3000, out=out)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            q_.tf_attn_decode(q, kp, vp, tables, n, 3000, out=out)
    torch.cuda.synchronize()
    for it in range(4):
        out.fill_(0)
        q.copy_(torch.roll(q, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q_.tf_attn_decode(q, kp, vp, tables, n, 3000)), f"replay {it} differs"
        torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_bound_below_the_new_tokens(d):
    """Rows up to the bound see the keys they see without it; the rest is not
    written.  Offsets of the lowest and highest value are clamped."""
    _, q_ = gpu_or_skip()
    hq, hkv = 6, 2
    g = _gen(21)
    qkv = _normal(g, (90, hq + 2 * hkv, d), torch.bfloat16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cu = torch.tensor([0, 70, 90], dtype=torch.int32, device=DEV)
    print("prefill bound", d, flush=True)
    want = q_.tf_attn_prefill(q, k, v, cu, cu, 70)
    given = torch.full((90, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    q_.tf_attn_prefill(q, k, v, cu, cu, 33, out=given)
    torch.cuda.synchronize()
    assert torch.equal(given[:33], want[:33]) and bool((given[33:70] == 7.0).all())
    assert torch.equal(given[70:], want[70:])
    low, high = -(2**31), 2**31 - 1
    odd = torch.tensor([low, 40, low, high, low], dtype=torch.int32, device=DEV)  # 0..40, none, 0..90, none
    given = torch.full((90, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    q_.tf_attn_prefill(q, k, v, odd[:3].contiguous(), odd[:3].contiguous(), 90, out=given)
    torch.cuda.synchronize()
    assert bool((given[40:] == 7.0).all())
    _check_prefill(q, lambda s, h: (k[:40, h].double(), v[:40, h].double()), [0, 40], [40], hkv, d ** -0.5, given)
    given = q_.tf_attn_prefill(q, k, v, odd[2:].contiguous(), odd[2:].contiguous(), 90)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (k[:, h].double(), v[:, h].double()), [0, 90], [90], hkv, d ** -0.5, given)


def test_fp16_keeps_the_small_weights_of_a_long_row():
    """One key of weight 1 and 40000 of weight about 2^-23, each too small for
    fp16 beside it but a part of 200 together."""
    _, q_ = gpu_or_skip()
    n, d, page = 40001, 64, 64
    pages = -(-n // page)
    kp = torch.zeros((pages, 1, page, d), dtype=torch.float16, device=DEV)
    vp = torch.ones_like(kp)
    q = torch.zeros((1, 1, d), dtype=torch.float16, device=DEV)
    q[..., 0], kp[0, 0, 0, 0], vp[0, 0, 0] = 1.0, 16.0, 0.0
    tables = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    print("small weights", flush=True)
    for out in (q_.tf_attn_decode(q, kp, vp, tables, lens, n, 1.0),
                q_.tf_attn_prefill_paged(q, kp, vp, tables, torch.tensor([0, 1], dtype=torch.int32, device=DEV), lens, 1, 1.0)):
        torch.cuda.synchronize()
        w = (n - 1) * torch.exp(torch.tensor(-16.0, dtype=torch.float64))
        want = float(w / (1 + w))
        # a weight is rounded to half of fp16's smallest step, 2^-25, against a maximum held at 2^7; the sum, one rounding
        tol = n * 2.0**-32 + 3 * 2.0**-11 * want
        assert bool(((out.double() - want).abs() <= tol).all()), (out.flatten()[:2].tolist(), want)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("new,nkeys,heads,page", [
    # few rows behind many keys: the keys are cut into ranges and joined
    ([1], [5000], (8, 1, 128), 16), ([37, 0, 5], [3001, 0, 700], (28, 4, 128), 64), ([130], [4097], (14, 2, 64), 16),
    ([400, 3], [1500, 4500], (8, 1, 128), 128), ([7, 9, 40], [7, 2, 2000], (71, 1, 64), 32), ([900], [900], (4, 2, 64), 16),
])
@pytest.mark.parametrize("paged", [False, True])
def test_prefill_ranges_of_keys(new, nkeys, heads, page, paged, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    print(f"prefill ranges {t} paged={paged} {heads} page {page} new {new} keys {nkeys}", flush=True)
    g = _gen(sum(new) + 3 * sum(nkeys) + hq)
    cu, ck = _starts(new), _starts(nkeys)
    cu_q = torch.tensor(cu, dtype=torch.int32, device=DEV)
    q = _normal(g, (sum(new), hq, d), TYPES[t], 1.5)
    if paged:
        tables, pages = ref.tables_for(nkeys, page, g)
        kp, vp = (_normal(g, (pages, hkv, page, d), TYPES[t]) for _ in "kv")
        assert q_.tf_attn_prefill_workspace_bytes(len(new), sum(new), hq, hkv, d, max(new), tables.shape[1] * page) > 0
        out = q_.tf_attn_prefill_paged(q, kp, vp, tables.to(DEV), cu_q, torch.tensor(nkeys, dtype=torch.int32, device=DEV), max(new))

        def keys_of(s, h):
            return ref.gather(kp, tables[s], nkeys[s], h), ref.gather(vp, tables[s], nkeys[s], h)
    else:
        k, v = (_normal(g, (sum(nkeys), hkv, d), TYPES[t]) for _ in "kv")
        need = q_.tf_attn_prefill_workspace_bytes(len(new), sum(new), hq, hkv, d, max(new), sum(nkeys))
        assert need > 0
        ws = torch.full((need // 4,), float("nan"), device=DEV)  # what it holds does not matter
        out = q_.tf_attn_prefill(q, k, v, cu_q, torch.tensor(ck, dtype=torch.int32, device=DEV), max(new), workspace=ws)
        small = ws[:-1]
        with pytest.raises(q_.TileFuseError, match="(?i)buffer|workspace|small"):
            q_.tf_attn_prefill(q, k, v, cu_q, torch.tensor(ck, dtype=torch.int32, device=DEV), max(new), workspace=small)

        def keys_of(s, h):
            return k[ck[s]:ck[s + 1], h].double(), v[ck[s]:ck[s + 1], h].double()
    torch.cuda.synchronize()
    _check_prefill(q, keys_of, cu, nkeys, hkv, d ** -0.5, out)


def test_prefill_infinities_past_a_range():
    """Infinities and NaN in values of every range, seen by some rows and not by others."""
    _, q_ = gpu_or_skip()
    n, new, hq, hkv, d = 2500, 60, 6, 2, 128
    g = _gen(31)
    q = _normal(g, (new, hq, d), torch.float16)
    k, v = (_normal(g, (n, hkv, d), torch.float16) for _ in "kv")
    for at, h, c, x in ((2490, 0, 3, "inf"), (2470, 1, 90, "-inf"), (2445, 1, 5, "nan"), (2499, 0, 127, "nan"), (2450, 0, 64, "inf")):
        v[at, h, c] = float(x)
    print("infinities past a range", flush=True)
    ints = [torch.tensor([0, x], dtype=torch.int32, device=DEV) for x in (new, n)]
    assert q_.tf_attn_prefill_workspace_bytes(1, new, hq, hkv, d, new, n) > 0
    out = q_.tf_attn_prefill(q, k, v, *ints, new, 0.2)
    torch.cuda.synchronize()
    _check_prefill(q, lambda s, h: (k[:, h].double(), v[:, h].double()), [0, new], [n], hkv, 0.2, out)


def test_threads_on_one_stream_share_its_workspace():
    """Calls of two kernels each from several host threads on the same stream:
    nothing comes between a call's kernels."""
    import threading

    _, q_ = gpu_or_skip()
    hq, hkv, d, page, rounds = 8, 2, 128, 16, 60
    g = _gen(41)
    cases = []
    for lens in ([3000], [700, 5000], [9000, 1, 2000], [1500] * 5):
        tables, pages = ref.tables_for(lens, page, g)
        q = _normal(g, (len(lens), hq, d), torch.bfloat16)
        kp, vp = (_normal(g, (pages, hkv, page, d), torch.bfloat16) for _ in "kv")
        cases.append((q, kp, vp, tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens)))
    print("threads on one stream", flush=True)
    alone = [q_.tf_attn_decode(*c) for c in cases]
    torch.cuda.synchronize()
    got, stream = [[] for _ in cases], torch.cuda.current_stream()

    def work(i):
        for _ in range(rounds):
            got[i].append(q_.tf_attn_decode(*cases[i], stream=stream))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    torch.cuda.synchronize()
    for want, outs in zip(alone, got):
        assert len(outs) == rounds and all(torch.equal(o, want) for o in outs)
