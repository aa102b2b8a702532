"""The paged cache on the GPU: rotating and storing tokens, forking and
compacting pages, against plain models in 64 bits and whole numbers."""

import random

import pytest
import torch

import attention_ref as ref
from gpu_harness import gpu_or_skip

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rope(rows, d):
    rate = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("heads,page,lens,mode", [
    ((32, 8, 128), 16, [1, 17, 400, 33], "step"),
    ((32, 8, 128), 64, [1, 17, 100, 33], "prompt"),
    ((28, 4, 128), 32, [300], "prompt"),
    ((14, 2, 64), 16, [5, 31, 2], "prompt"),
    ((71, 1, 64), 128, [3, 129], "prompt"),
    ((3, 1, 96), 16, [20, 1], "prompt"),
    ((2, 2, 16), 16, [9], "step"),
    ((5, 5, 256), 16, [40], "prompt"),
    ((32, 32, 128), 16, [700, 600], "prompt"),  # enough tokens that a wave takes all passes
])
def test_append(heads, page, lens, mode, t):
    _, q_ = gpu_or_skip()
    hq, hkv, d = heads
    print(f"append {t} {heads} page {page} {lens} {mode}", flush=True)
    g = torch.Generator()
    g.manual_seed(sum(lens) + hq + d)
    tables, pages = ref.tables_for(lens, page, g)
    seq = [i for i, n in enumerate(lens) for _ in range(n)] if mode == "prompt" else list(range(len(lens)))
    pos = [j for n in lens for j in range(n)] if mode == "prompt" else [n - 1 for n in lens]
    wide = (torch.randn((len(seq), (hq + 2 * hkv) * d + 8), generator=g)).to(TYPES[t]).to(DEV)
    qkv = wide[:, :-8]
    kp, vp = (torch.randn((pages, hkv, page, d), generator=g).to(TYPES[t]).to(DEV) for _ in "kv")
    k0, v0 = kp.clone(), vp.clone()
    rope = _rope(max(lens), d)
    q = q_.tf_kv_append(qkv, rope, _ints(seq), _ints(pos), tables.to(DEV), kp, vp, hq)
    torch.cuda.synchronize()
    x = qkv.double().view(-1, hq + 2 * hkv, d)
    turn = rope.double()[torch.tensor(pos)][:, None]
    c, s = turn[..., :d // 2], turn[..., d // 2:]
    a, b = x[..., :d // 2], x[..., d // 2:]
    y = torch.cat([a * c - b * s, b * c + a * s], -1)
    size = torch.cat([(a * c).abs() + (b * s).abs()] * 1 + [(b * c).abs() + (a * s).abs()], -1)
    # one rounding, two fp32 products and a sum; fp16's smallest step
    tol = torch.finfo(TYPES[t]).eps / 2 * y.abs() + 3 * 2.0**-24 * size * (1 + 2.0**-7) + 2.0**-25
    assert bool(((q.double() - y[:, :hq]).abs() <= tol[:, :hq]).all())
    touched = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    at = tables.to(DEV)[torch.tensor(seq), torch.tensor([p // page for p in pos])].long()
    row = torch.tensor([p % page for p in pos], device=DEV)
    touched[at, row] = True
    assert bool(((kp[at, :, row].double() - y[:, hq:hq + hkv]).abs() <= tol[:, hq:hq + hkv]).all())
    assert torch.equal(vp[at, :, row].view(torch.int16), qkv.reshape(-1, hq + 2 * hkv, d)[:, hq + hkv:].contiguous().view(torch.int16))
    keep = ~touched[:, None, :, None].expand_as(kp)
    assert torch.equal(kp[keep], k0[keep]) and torch.equal(vp[keep], v0[keep])


def test_append_skips_places_that_do_not_exist():
    _, q_ = gpu_or_skip()
    hq, hkv, d, page, pages = 2, 1, 32, 16, 4
    tables = _ints([[0, -1, 2], [9, 1, -(2**31)]])
    seq = [0, 0, 0, 1, 1, 1, -1, 2, 2**31 - 1, 0, 0, 1]
    pos = [0, 16, 40, 0, 20, 33, 3, 3, 3, -1, 48, 2**31 - 1]
    g = torch.Generator()
    g.manual_seed(3)
    qkv = torch.randn((len(seq), (hq + 2 * hkv) * d), generator=g).to(torch.bfloat16).to(DEV)
    kp, vp = (torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    print("append bad places", flush=True)
    q = q_.tf_kv_append(qkv, _rope(48, d), _ints(seq), _ints(pos), tables, kp, vp, hq)
    torch.cuda.synchronize()
    stored = {(0, 0): 0, (2, 8): 2, (1, 4): 4}  # (page, row): token
    x = qkv.view(-1, hq + 2 * hkv, d)
    for p in range(pages):
        for r in range(page):
            want = x[stored[p, r], -1] if (p, r) in stored else torch.zeros(d, dtype=torch.bfloat16, device=DEV)
            assert torch.equal(vp[p, 0, r], want), (p, r)
            assert bool((kp[p, 0, r] == 0).all()) == ((p, r) not in stored)
    turned = [i for i, n in enumerate(pos) if 0 <= n < 48]
    for i in range(len(pos)):
        assert bool((q[i] == 0).all()) == (i not in turned), i


def _state(rng, seqs, page, longest, gone, pages_more):
    lens = [0 if i in gone else rng.randint(1, longest) for i in range(seqs)]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + pages_more
    order = list(range(pages))
    rng.shuffle(order)
    width = max(need) + 2
    tables, refs, at = [], [0] * pages, 0
    for n in need:
        row = order[at:at + n]
        at += n
        for p in row:
            refs[p] = 1
        tables.append(row + [-1] * (width - n))
    return lens, tables, refs, pages


def _fork_model(cache, refs, tables, lens, parents, children, page):
    cache, refs, tables, lens = cache.clone(), list(refs), [list(r) for r in tables], list(lens)
    free = [p for p, r in enumerate(refs) if r == 0]
    size = [lens[p] for p in parents]
    want = [i for i, n in enumerate(size) if n % page]
    if len(want) > len(free):
        return cache, refs, tables, lens, len(want) - len(free)
    got = dict(zip(want, free))
    rows = []
    for i, p in enumerate(parents):
        full = size[i] // page
        row = tables[p][:full] + ([got[i]] if i in got else [])
        rows.append(row + [-1] * (len(tables[p]) - len(row)))
        for x in row:
            refs[x] += 1
        if i in got:
            r = size[i] % page
            cache[:, got[i], :, :r] = cache[:, tables[p][full], :, :r]
    for i, c in enumerate(children):
        tables[c], lens[c] = rows[i], size[i]
    return cache, refs, tables, lens, 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,page,longest,planes,heads,more,forks", [
    (6, 16, 100, 2, (2, 64), 9, 2), (24, 16, 900, 4, (8, 128), 60, 8), (5, 64, 64, 3, (1, 128), 3, 1),
    (4, 1, 7, 2, (2, 8), 20, 2), (40, 32, 300, 2, (4, 64), 3000, 20), (6, 16, 100, 2, (2, 64), 1, 3),
    (3, 16, 50, 2, (2, 64), 9, 0), (3000, 16, 20, 1, (1, 8), 9000, 1400),
])
def test_fork(seqs, page, longest, planes, heads, more, forks, in_place):
    _, q_ = gpu_or_skip()
    rng = random.Random(seqs * 100 + more)
    print(f"fork seqs {seqs} page {page} longest {longest} forks {forks} in place {in_place}", flush=True)
    children = list(range(seqs - forks, seqs))
    lens, tables, refs, pages = _state(rng, seqs, page, longest, set(children), more)
    rng.shuffle(children)
    parents = [rng.randrange(seqs - forks) for _ in children]
    cache = torch.randint(-30000, 30000, (planes, pages, heads[0], page, heads[1]), dtype=torch.int16).view(torch.bfloat16)
    dev = cache.to(DEV)
    state = [_ints(refs), _ints(tables), _ints(lens)]
    outs = state if in_place else [torch.empty_like(x) for x in state]
    kwargs = {} if in_place else dict(refs_out=outs[0], tables_out=outs[1], lens_out=outs[2])
    status = q_.tf_kv_fork(dev, *state, _ints(parents), _ints(children), **kwargs)
    torch.cuda.synchronize()
    want = _fork_model(cache.view(torch.int16), refs, tables, lens, parents, children, page)
    assert status.tolist() == [want[4]]
    assert outs[0].tolist() == want[1] and outs[1].tolist() == want[2] and outs[2].tolist() == want[3]
    assert torch.equal(dev.cpu().view(torch.int16), want[0])
    if not in_place:
        assert state[0].tolist() == refs and state[1].tolist() == tables


def test_fork_skips_pairs_that_do_not_exist():
    _, q_ = gpu_or_skip()
    cache = torch.arange(2 * 6 * 16 * 8, dtype=torch.int16, device=DEV).view(2, 6, 1, 16, 8).view(torch.float16)
    before = cache.clone()
    refs, tables, lens = _ints([1, 1, 0, 0, 1, 0]), _ints([[0, 1, -1], [4, 99, 7], [-1, -1, -1], [-1, -1, -1]]), _ints([20, 40, 0, -3])
    print("fork bad pairs", flush=True)
    status = q_.tf_kv_fork(cache, refs, tables, lens, _ints([-1, 9, 0, 1]), _ints([2, 3, 4, 3]))
    torch.cuda.synchronize()
    # the last pair alone exists; its partial page (id 7) does not, so its fresh page keeps what it held
    assert status.tolist() == [0] and lens.tolist() == [20, 40, 0, 40]
    assert tables.tolist() == [[0, 1, -1], [4, 99, 7], [-1, -1, -1], [4, 99, 2]]
    assert refs.tolist() == [1, 1, 1, 0, 2, 0]
    assert torch.equal(cache.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,page,longest,planes,heads,more,freed", [
    (6, 16, 100, 2, (2, 64), 9, 2), (40, 64, 1024, 2, (8, 128), 30, 16), (5, 64, 64, 3, (1, 128), 0, 0),
    (4, 1, 7, 2, (2, 8), 20, 3), (500, 16, 300, 1, (1, 8), 9000, 250), (3, 16, 50, 2, (2, 64), 9, 3),
])
def test_compact(seqs, page, longest, planes, heads, more, freed, in_place):
    _, q_ = gpu_or_skip()
    rng = random.Random(seqs * 10 + more)
    print(f"compact seqs {seqs} page {page} longest {longest} freed {freed} in place {in_place}", flush=True)
    lens, tables, refs, pages = _state(rng, seqs, page, longest, set(), more)
    for s in rng.sample(range(seqs), freed):
        for c, p in enumerate(tables[s]):
            if p >= 0:
                refs[p] = 0
                tables[s][c] = -1
    for p in range(0, pages, 7):  # shared pages
        refs[p] += refs[p] > 0
    tables[0][-1] = pages + 5  # no page of the pool
    cache = torch.randint(-30000, 30000, (planes, pages, heads[0], page, heads[1]), dtype=torch.int16)
    dev = cache.view(torch.float16).to(DEV)
    state = [_ints(refs), _ints(tables)]
    outs = state if in_place else [torch.empty_like(x) for x in state]
    moved = q_.tf_kv_compact(dev, *state, **({} if in_place else dict(refs_out=outs[0], tables_out=outs[1])))
    torch.cuda.synchronize()
    live = [p for p in range(pages) if refs[p] > 0]
    n = len(live)
    to = iter([p for p in range(n) if refs[p] == 0])
    where = {p: p if p < n else next(to) for p in live}
    want, want_refs = cache.clone(), [0] * pages
    for p, w in where.items():
        want[:, w] = cache[:, p]
        want_refs[w] = refs[p]
    assert moved.tolist() == [where.get(p, -1) for p in range(pages)]
    assert outs[0].tolist() == want_refs
    assert outs[1].tolist() == [[where.get(p, -1) for p in r] for r in tables]
    assert torch.equal(dev.cpu().view(torch.int16), want)


def test_pool_calls_under_a_graph():
    """Fork and compact captured together, replayed from the same state between
    eager calls."""
    _, q_ = gpu_or_skip()
    rng = random.Random(4)
    lens, tables, refs, pages = _state(rng, 8, 16, 90, {6, 7}, 12)
    cache0 = torch.randint(-30000, 30000, (2, pages, 2, 16, 64), dtype=torch.int16, device=DEV).view(torch.bfloat16)
    start = [cache0, _ints(refs), _ints(tables), _ints(lens)]
    cache, r, t, n = (x.clone() for x in start)
    parents, children = _ints([1, 3]), _ints([6, 7])
    status, moved = _ints([0]), torch.empty_like(r)

    def step():
        q_.tf_kv_fork(cache, r, t, n, parents, children, status=status)
        q_.tf_kv_compact(cache, r, t, moved=moved)

    def reset():
        for x, y in zip((cache, r, t, n), start):
            x.copy_(y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        eager = [x.clone() for x in (cache, r, t, n, moved)]
        reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for it in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((cache, r, t, n, moved), eager):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16)), f"replay {it} differs"
        reset()
        step()
        torch.cuda.synchronize()


def test_append_without_a_rotation_is_zero_whatever_the_heads_hold():
    _, q_ = gpu_or_skip()
    hq, hkv, d, page = 2, 1, 32, 16
    qkv = torch.full((3, (hq + 2 * hkv) * d), float("inf"), dtype=torch.bfloat16, device=DEV)
    qkv[1], qkv[2] = float("nan"), 1.0
    kp, vp = (torch.ones((2, hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    print("append without rotation", flush=True)
    q = q_.tf_kv_append(qkv, _rope(4, d), _ints([0, 0, 0]), _ints([4, 17, 3]), _ints([[0, 1]]), kp, vp, hq)
    torch.cuda.synchronize()
    assert bool((q[:2] == 0).all()) and bool((q[2] != 0).all())
    assert bool((kp[0, 0, 4] == 0).all()) and bool((kp[1, 0, 1] == 0).all())
    assert bool((vp[0, 0, 4] == float("inf")).all()) and bool(vp[1, 0, 1].isnan().all())
