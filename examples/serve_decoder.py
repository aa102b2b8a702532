"""A small W4A16 decoder served from a paged cache: random weights, a few
prompts of different lengths, new tokens one at a time, parallel samples of one
prompt, a freed sequence and a compacted pool.

    python examples/serve_decoder.py [--layers 4] [--steps 16]

Each layer runs RMS norm (torch) -> QKV linear -> tf_kv_append ->
tf_attn_prefill_paged or tf_attn_decode -> output linear, then RMS norm ->
[gate | up] linear with SiLU -> down linear.  At the end every sequence's
hidden states are run again from nothing, as one prompt over packed keys, and
compared with what the served steps gave.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_linear_layers_awq_amd as tf  # noqa: E402

DEV = "cuda"
GROUP = 128


def random_linear(g, k, n, gate_up=False):
    """A packed W4 linear of random codes whose weights have a standard deviation of about k^-0.5."""
    qweight = torch.randint(-2**31, 2**31 - 1, (k, n // 8), generator=g, dtype=torch.int64).to(torch.int32).to(DEV)
    qzeros = torch.full((k // GROUP, n // 8), 0x77777777, dtype=torch.int32, device=DEV)
    scales = ((torch.rand((k // GROUP, n), generator=g) + 0.5) * 0.22 * k ** -0.5).to(torch.bfloat16).to(DEV)
    repack = tf.tf_repack_w4_gate_up if gate_up else tf.tf_repack_w4
    return repack(qweight, qzeros, scales, k, n, GROUP), k, n


def rms_norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Cache:
    """The pool of pages of all layers and the table of the sequences in it.

    Pages are handed out on the host, which keeps a copy of refs and lengths;
    forking and compacting run on the device."""

    def __init__(self, layers, pages, hkv, page, d, seqs, width):
        self.planes = torch.zeros((2 * layers, pages, hkv, page, d), dtype=torch.bfloat16, device=DEV)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.tables = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=DEV)
        self.page = page

    def layer(self, i):
        return self.planes[2 * i], self.planes[2 * i + 1]

    def reserve(self, more):
        """Room for more[s] tokens of each sequence s; returns the sequence and position of each new token."""
        refs, tables, lens = self.refs.tolist(), self.tables.tolist(), self.lens.tolist()
        free = (p for p, r in enumerate(refs) if r == 0)
        seq, pos = [], []
        for s, n in more.items():
            for c in range(-(-lens[s] // self.page), -(-(lens[s] + n) // self.page)):
                tables[s][c] = next(free, None)
                if tables[s][c] is None:
                    raise RuntimeError("no page is free")
                refs[tables[s][c]] = 1
            seq += [s] * n
            pos += range(lens[s], lens[s] + n)
            lens[s] += n
        for to, values in ((self.refs, refs), (self.tables, tables), (self.lens, lens)):
            to.copy_(torch.tensor(values, dtype=torch.int32))
        return ints(seq), ints(pos)

    def free(self, s):
        """Give up a sequence: its pages lose a reference."""
        row = self.tables[s][:-(-int(self.lens[s]) // self.page)].long()
        self.refs.index_add_(0, row, torch.full_like(row, -1, dtype=torch.int32))
        self.tables[s], self.lens[s] = -1, 0

    def fork(self, parent, children):
        status = tf.tf_kv_fork(self.planes, self.refs, self.tables, self.lens, ints([parent] * len(children)), ints(children))
        if int(status):
            raise RuntimeError(f"{int(status)} pages short")

    def compact(self):
        tf.tf_kv_compact(self.planes, self.refs, self.tables)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Decoder:
    def __init__(self, layers, hidden, hq, hkv, d, inner, positions, seed=0):
        g = torch.Generator()
        g.manual_seed(seed)
        self.hq, self.hkv, self.d = hq, hkv, d
        self.layers = [dict(qkv=random_linear(g, hidden, (hq + 2 * hkv) * d), o=random_linear(g, hq * d, hidden),
                            gate_up=random_linear(g, hidden, 2 * inner, gate_up=True), down=random_linear(g, inner, hidden))
                       for _ in range(layers)]
        rate = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        angle = torch.arange(positions, dtype=torch.float64)[:, None] * rate
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)

    def run(self, x, attend):
        """x [T][hidden] through all layers; attend(layer, qkv) is the layer's attention, [T][Hq][D]."""
        for i, w in enumerate(self.layers):
            packed, k, n = w["qkv"]
            out = attend(i, tf.tf_gemm_w4a16(rms_norm(x), packed, k, n, GROUP))
            packed, k, n = w["o"]
            x = x + tf.tf_gemm_w4a16(out.view(len(x), -1), packed, k, n, GROUP)
            packed, k, n = w["gate_up"]
            y = tf.tf_gemm_w4a16_silu_mul(rms_norm(x), packed, k, n, GROUP)
            packed, k, n = w["down"]
            x = x + tf.tf_gemm_w4a16(y, packed, k, n, GROUP)
        return x

    def _append(self, cache, i, qkv, seq, pos):
        k_pages, v_pages = cache.layer(i)
        return tf.tf_kv_append(qkv, self.rope, seq, pos, cache.tables, k_pages, v_pages, self.hq), k_pages, v_pages

    def prefill(self, cache, prompts):
        """prompts: sequence -> its new tokens' hidden states, [n][hidden]; the whole batch at once."""
        new = {s: len(prompts[s]) if s in prompts else 0 for s in range(len(cache.lens))}
        seq, pos = cache.reserve({s: n for s, n in new.items() if n})
        starts = ints([0] + torch.tensor(list(new.values())).cumsum(0).tolist())

        def attend(i, qkv):
            q, k_pages, v_pages = self._append(cache, i, qkv, seq, pos)
            return tf.tf_attn_prefill_paged(q, k_pages, v_pages, cache.tables, starts, cache.lens, max(new.values()))

        x = self.run(torch.cat([prompts[s] for s in sorted(prompts)]), attend)
        return dict(zip(sorted(prompts), x.split([new[s] for s in sorted(prompts)])))

    def decode(self, cache, x, live):
        """One new token for each live sequence: x [live][hidden]."""
        seq, pos = cache.reserve({s: 1 for s in live})
        rows, longest = seq.long(), int(cache.lens.max())
        tables, lens = cache.tables[rows], cache.lens[rows]

        def attend(i, qkv):
            q, k_pages, v_pages = self._append(cache, i, qkv, seq, pos)
            return tf.tf_attn_decode(q, k_pages, v_pages, tables, lens, longest)

        return self.run(x, attend)

    def whole(self, x):
        """One sequence at once: append rotates its keys into scratch pages, which are gathered into packed
        ones (the QKV output itself keeps unrotated keys)."""
        n = len(x)
        cu = ints([0, n])
        pages = -(-n // 128)
        scratch = torch.zeros((2, pages, self.hkv, 128, self.d), dtype=torch.bfloat16, device=DEV)
        tables = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
        seq, pos = ints([0] * n), ints(list(range(n)))

        def attend(i, qkv):
            q = tf.tf_kv_append(qkv, self.rope, seq, pos, tables, scratch[0], scratch[1], self.hq)
            k, v = (p.transpose(1, 2).reshape(-1, self.hkv, self.d)[:n] for p in scratch)
            return tf.tf_attn_prefill(q, k, v, cu, cu, n)

        return self.run(x, attend)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--heads", type=int, nargs=3, default=(16, 4, 64), metavar=("HQ", "HKV", "D"))
    p.add_argument("--prompts", type=int, nargs="+", default=(300, 45, 128))
    p.add_argument("--samples", type=int, default=2, help="further samples of the first prompt")
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--page", type=int, default=16)
    a = p.parse_args(argv)
    hq, hkv, d = a.heads
    seqs, longest = len(a.prompts) + a.samples, max(a.prompts) + 2 * a.steps
    width = -(-longest // a.page)
    model = Decoder(a.layers, a.hidden, hq, hkv, d, 2 * a.hidden, longest)
    cache = Cache(a.layers, seqs * width, hkv, a.page, d, seqs, width)
    g = torch.Generator()
    g.manual_seed(1)

    def states(n):
        return torch.randn((n, a.hidden), generator=g).to(torch.bfloat16).to(DEV)

    # what goes in and what comes out, for the comparison at the end
    fed = {s: states(n) for s, n in enumerate(a.prompts)}
    got = model.prefill(cache, fed)
    print(f"prefill: {len(a.prompts)} prompts, {sum(a.prompts)} tokens")

    # further samples of the first prompt share its full pages
    children = list(range(len(a.prompts), seqs))
    if children:
        cache.fork(0, children)
        for c in children:
            fed[c], got[c] = fed[0], got[0]
        print(f"fork: {len(children)} samples, {int((cache.refs > 1).sum())} pages shared")

    def steps(live):
        for _ in range(a.steps):
            x = states(len(live))
            y = model.decode(cache, x, live)
            for i, s in enumerate(live):
                fed[s], got[s] = torch.cat([fed[s], x[i:i + 1]]), torch.cat([got[s], y[i:i + 1]])

    live = sorted(fed)
    steps(live)
    print(f"decode: {a.steps} tokens for each of {len(live)} sequences")
    if len(live) > 1:
        gone = live.pop(1)
        cache.free(gone)
    cache.compact()
    used = int((cache.refs > 0).sum())
    assert int(cache.tables.max()) < used
    print(f"compact: {used} pages in use, all at the front")
    steps(live)

    worst = 0.0
    for s in sorted(fed):
        want = model.whole(fed[s])
        worst = max(worst, float((got[s].float() - want.float()).norm() / want.float().norm()))
    print(f"served against whole sequences: relative difference {worst:.2e}")
    return worst


if __name__ == "__main__":
    # bf16 activations: a few roundings of 2^-9 per layer, which different batch sizes add in different orders
    sys.exit(0 if main() < 2e-2 else 1)
