// Attention of one new token per sequence over a paged key-value cache:
//
//   o[s][j] = sum_t softmax_t(scale q[s][j] . k[t]) v[t],  t < lens[s]
//
// for the G = Hq / Hkv query heads j of each key-value head.
//
// What bounds it: the cache is read once, 4 D bytes per token and key-value
// head against 4 G D operations, so HBM does.  The kernel is a stream of
// key tiles with the arithmetic hidden under it:
//  - A workgroup's W waves each take every W-th 32-key tile of its range on
//    their own: K goes from memory straight into MFMA operand registers, V
//    through the wave's own LDS buffer (row-major in, transposed out), the
//    next tile's loads in flight meanwhile.  No barrier before the end.
//  - Both products run on 16x16x32 MFMAs with the query heads as columns, so
//    the heads of a group share one read of the cache.
//  - Page ids of 32 tiles are fetched by one load per wave (a lane per
//    16-key run) and read out lane by lane, off the critical path.
//  - The waves' (m, l, O) are joined in LDS in wave order.
//  - Short caches: a workgroup per (sequence, key-value head, group of 16 NT
//    query heads), which writes the output.  Long ones: the keys of all
//    (sequence, head, group) items, in units of a few tiles, are laid end to
//    end and cut into equal shares, one per workgroup and compute unit,
//    so that ragged lengths leave no tail.  A workgroup finds its share from
//    a prefix sum of the lengths.  Items that lie whole in a share are
//    written; the others' fp32 partials are added by attn_join_kernel in
//    order.  No atomics.  The next item's first tile is on its way while an
//    item's waves are joined (73 sequences of up to 1827, 12 heads of 64: 49
//    us, and 59 without).
// Measured, with the reading rate of a plain stream at 7.0 TB/s: 16 contexts of
// up to 32768 tokens, 8 heads of 128 channels, 171 us (6.6 TB/s); one of 131072
// 87 us (6.2: the kernel alone runs at 6.6, the join takes 5 us); 48 ragged ones
// of up to 4096, 4 heads, 45 us (5.3); one of 333 tokens 6.5 us, which is the
// latency of the chain length, pages, keys, join.
#include "tf_attn.h"

namespace tf {

namespace {

constexpr int kTile = 32;
// Cache policy of the keys and values: streamed (nt), for they are read once a
// step and the next layer's displace them.  Against the default, four caches
// in turn: 16 contexts of up to 32768 tokens (1.12 GB) 174 us and 193, one of
// 131072 89 and 99; where one cache of 240 MB is read again and again and
// stays in the last-level cache, 48 and 44.
constexpr int kStream = 2;

template <int D> struct Stage {
    u32x4 k[2][D / 32]; // sub-tile of 16 keys, 32-channel step
    u32x4 v[2][D / 32]; // 16 rows as they lie in memory, 1 KiB per load
};

template <int D> constexpr int v_swz(int row) { return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3); }

// Where a workgroup's share begins: the sequence, its length, and the units of
// the sequences before it (of one item each; a unit is 2^unit_shift keys, and the
// launch keeps the units of all items below 2^31).
struct Start {
    int units; // of all sequences
    int before, seq, len;
};

__device__ __forceinline__ int units_of(const DecodeArgs &a, int len) { return (len + (1 << a.unit_shift) - 1) >> a.unit_shift; }

// Finds units, and the sequence that holds unit place(units) of them (none past
// the end: seq = seqs).  Every thread takes a strip of sequences.
template <int THREADS, typename Place> __device__ __forceinline__ Start find_start(const DecodeArgs &a, Place place)
{
    __shared__ int s_sum[THREADS / 64], s_found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int strip = (a.seqs + THREADS - 1) / THREADS;
    const int first = min(tid * strip, a.seqs), end = min(first + strip, a.seqs);
    int sum = 0, len = 0;
    for (int s = first; s < end; ++s) {
        len = clampi(a.lens[s], 0, a.longest);
        sum += units_of(a, len);
    }
    int in = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(in, d);
        in += lane >= d ? y : 0;
    }
    if (lane == 63)
        s_sum[wave] = in;
    if (tid == 0)
        s_found[0] = a.seqs;
    __syncthreads();
    int before = in - sum, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        const int x = s_sum[w];
        before += w < wave ? x : 0;
        all += x;
    }
    const int at = place(all);
    if (before <= at && at < before + sum) {
        int s = first;
        if (strip > 1) // the strip's sequence that holds it
            for (;; ++s) {
                len = clampi(a.lens[s], 0, a.longest);
                const int r = units_of(a, len);
                if (at < before + r)
                    break;
                before += r;
            }
        s_found[0] = s;
        s_found[1] = before;
        s_found[2] = len;
    }
    __syncthreads();
    return {all, __builtin_amdgcn_readfirstlane(s_found[1]), __builtin_amdgcn_readfirstlane(s_found[0]),
            __builtin_amdgcn_readfirstlane(s_found[2])};
}

// W waves; SHARES: equal shares of all keys, else one item of one sequence
template <int D, bool F16, int NT, int W, bool SHARES> __global__ __launch_bounds__(64 * W, 2) void attn_decode_kernel(DecodeArgs a)
{
    constexpr int kSteps = D / 32;   // MFMA steps over channels
    constexpr int kTiles = D / 16;   // 16-channel tiles of O^T
    constexpr int kRow = 2 * D;      // bytes of a row
    constexpr int kChunks = D / 8;   // 16-byte units of a row
    constexpr int kRowsPerLoad = 1024 / kRow;
    constexpr int kWaveBytes = kTile * kRow; // V of a tile; in the join, 16 heads of D floats
    static_assert(kWaveBytes == 16 * D * 4, "the join reuses the V buffers");
    __shared__ __attribute__((aligned(16))) uint8_t lds[W * kWaveBytes];
    __shared__ float s_m[W][16], s_l[W][16];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, n = lane & 15;
    const int items = a.cache.hkv * a.groups; // of a sequence
    uint8_t *const vbuf = lds + wave * kWaveBytes;

    // V in LDS: unit c of row r at r kRow + 16 (c ^ v_swz(r))
    const int wr_row = lane / kChunks, wr_unit = lane % kChunks;
    uint32_t tr[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int r = 4 * g + (n >> 2), c = 2 * t + ((n >> 1) & 1);
        tr[t] = r * kRow + 16 * (c ^ v_swz<D>(r)) + 8 * (n & 1);
    }
    const u32x4 ones = F16 ? u32x4{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u}
                           : u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

    const int page_mask = (1 << a.cache.page_shift) - 1;
    const int64_t page_elems = (int64_t)D << a.cache.page_shift;
    const uint32_t k_off = n * kRow + 16 * g, v_off = 16 * lane;

    // Keys c0 .. c1 - 1 of an item (all uniform).  The result goes to the output
    // (slot < 0) or to a slot of the partial results.
    struct Segment {
        int seq, item, c0, c1, slot;
    };
    // this wave's tiles of a segment: wave, wave + W, ...
    auto tiles_here = [&](const Segment &e) {
        const int tiles = (e.c1 - e.c0 + kTile - 1) / kTile;
        return tiles > wave ? (tiles - wave + W - 1) / W : 0;
    };
    // lane L: the page of 16-key run L % 2 of this wave's tile it0 + L / 2.  The
    // load does not wait for the length (c1), which may still be on its way.
    auto page_ids = [&](const Segment &e, int it0) {
        const int key = e.c0 + kTile * (wave + W * (it0 + (lane >> 1))) + 16 * (lane & 1);
        int id = -1;
        if (key < a.longest)
            id = a.cache.tables[(int64_t)e.seq * a.cache.width + (key >> a.cache.page_shift)];
        return key < e.c1 && id < a.cache.pages ? id : -1;
    };
    auto load = [&](const Segment &e, Stage<D> &st, int it, int ids) {
        const int key0 = e.c0 + kTile * (wave + W * it), h = e.item % a.cache.hkv;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const int key = key0 + 16 * sub;
            const int id = __builtin_amdgcn_readlane(ids, (2 * it + sub) & 63);
            const int rows = id < 0 ? 0 : rows_before(e.c1, key);
            const int64_t at = ((int64_t)max(id, 0) * a.cache.hkv + h) * page_elems + (int64_t)(key & page_mask) * D;
            const Rsrc kr = make_rsrc_n(a.cache.k + at, rows * kRow), vr = make_rsrc_n(a.cache.v + at, rows * kRow);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                st.k[sub][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(kr, k_off + 64 * s, 0, kStream));
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                st.v[sub][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(vr, v_off + 1024 * s, 0, kStream));
        }
    };
    u32x4 q[NT][kSteps]; // Q^T operands: column n is head 16 NT group + 16 nt + n
    auto load_q = [&](const Segment &e) {
        const int h = e.item % a.cache.hkv, row0 = e.item / a.cache.hkv * 16 * NT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = min(row0 + 16 * nt + n, a.G - 1);
            const uint16_t *p = a.q + e.seq * a.q_token + (int64_t)(h * a.G + r) * a.q_head + 8 * g;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                q[nt][s] = load16(p + 32 * s);
        }
    };

    f32x4 o[NT][kTiles], l[NT];
    float m[NT];
    auto compute = [&](const Segment &e, const Stage<D> &st, int it) {
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int r = 16 * sub + kRowsPerLoad * s + wr_row;
                *reinterpret_cast<u32x4 *>(vbuf + r * kRow + 16 * (wr_unit ^ v_swz<D>(r))) = st.v[sub][s];
            }
        const int key0 = e.c0 + kTile * (wave + W * it);
        u32x4 p[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            f32x4 x[2] = {};
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    x[sub] = mfma16x16x32<F16>(st.k[sub][s], q[nt][s], x[sub]);
            if (key0 + kTile > e.c1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (key0 + 16 * (i >> 2) + 4 * g + (i & 3) >= e.c1)
                        x[i >> 2][i & 3] = -INFINITY;
            }
            float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                              fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
            top = held_maximum<F16>(max_swap32(max_swap16(top)) * a.scale_log2);
            if (__builtin_amdgcn_ballot_w64(top - m[nt] > kRescaleSlack)) {
                const float to = fmaxf(m[nt], top), f = exp2_fast(m[nt] - to);
                m[nt] = to;
                l[nt] *= f;
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    o[nt][t] *= f;
            }
            float by = a.scale_log2;
            if (__builtin_amdgcn_ballot_w64(fabsf(m[nt]) >= kLargeScore)) { // rare
                x[0] *= by, x[1] *= by;
                by = 1.f;
            }
            // P rounds to the inputs' type, the operands' of the MFMA (error
            // against 64 bits 1.6e-3 in the plain fp32 form and 1.7e-3 here,
            // bf16, the output's rounding the most of both); the sum is taken
            // over the rounded values (a product with ones), so that rounding
            // cancels where a row's weight sits on few keys
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[nt][j] = pack_half_x2<F16>(exp2_fast(x[j >> 1][2 * (j & 1)] * by - m[nt]),
                                             exp2_fast(x[j >> 1][2 * (j & 1) + 1] * by - m[nt]));
            l[nt] = mfma16x16x32<F16>(ones, p[nt], l[nt]);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const u32x2 lo = lds_read_tr(vbuf + tr[t]), hi = lds_read_tr(vbuf + tr[t] + 16 * kRow);
            const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                o[nt][t] = mfma16x16x32<F16>(v, p[nt], o[nt][t]);
        }
    };

    // join the waves, 16 heads at a time
    auto finish = [&](const Segment &e) {
        const int h = e.item % a.cache.hkv, row0 = e.item / a.cache.hkv * 16 * NT;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int heads = min(16, a.G - row0 - 16 * nt);
            if (heads <= 0)
                break;
            __syncthreads();
            float *const mine_o = reinterpret_cast<float *>(lds + wave * kWaveBytes);
            if (n < heads) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t) // 4-float units, XORed by head: no bank conflicts
                    *reinterpret_cast<f32x4 *>(mine_o + n * D + 4 * ((4 * t + g) ^ n)) = o[nt][t];
                if (g == 0) {
                    s_m[wave][n] = m[nt];
                    s_l[wave][n] = l[nt][0];
                }
            }
            __syncthreads();
            for (int u = threadIdx.x; u < heads * (D / 2); u += 64 * W) {
                const int r = u / (D / 2), c = 2 * (u % (D / 2));
                float top = s_m[0][r];
#pragma unroll
                for (int w = 1; w < W; ++w)
                    top = fmaxf(top, s_m[w][r]);
                float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float f = exp2_fast(s_m[w][r] - top);
                    const float *const p = reinterpret_cast<const float *>(lds + w * kWaveBytes) + r * D + 4 * ((c >> 2) ^ r) + (c & 3);
                    sum += f * s_l[w][r];
                    x += f * p[0];
                    y += f * p[1];
                }
                if (e.slot < 0) {
                    const int64_t at = (int64_t)e.seq * a.cache.hkv * a.G + h * a.G + row0 + 16 * nt + r;
                    const float inv = sum == 0.f ? 1.f : 1.f / sum;
                    *reinterpret_cast<uint32_t *>(a.out + at * D + c) = pack_half_x2<F16>(x * inv, y * inv);
                } else {
                    const int64_t at = (int64_t)e.slot * 16 * NT + 16 * nt + r;
                    *reinterpret_cast<f32x2 *>(a.part + at * D + c) = f32x2{x, y};
                    if (c == 0)
                        *reinterpret_cast<f32x2 *>(a.stats + 2 * at) = f32x2{top, sum};
                }
            }
        }
    };

    // Segments one after the other: the pages of the next one's first tiles are
    // asked for before this one's tiles, its queries and its first tile before
    // this one's waves are joined.  next(e, f) names the segment after e.
    constexpr bool kTwoStages = D == 64 || NT == 1; // else the registers hold one, and the other waves cover its loads
    auto run = [&](Segment e, auto next) {
        Stage<D> now;
        int ids = page_ids(e, 0), mine = tiles_here(e);
        load_q(e);
        if (kTwoStages && mine > 0)
            load(e, now, 0, ids);
        for (;;) {
            Segment f;
            const bool more = next(e, f);
            const int ids_after = more ? page_ids(f, 0) : -1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt] = kLowest;
                l[nt] = f32x4{};
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    o[nt][t] = f32x4{};
            }
#pragma unroll 1
            for (int it = 0; it < mine; ++it) {
                if constexpr (kTwoStages) {
                    // the loads of one stage in flight while the other is
                    // computed; a copy of the stage costs less than a second
                    // copy of the code
                    if (((it + 1) & 31) == 0)
                        ids = page_ids(e, it + 1);
                    Stage<D> after = now;
                    if (it + 1 < mine)
                        load(e, after, it + 1, ids);
                    compute(e, now, it);
                    now = after;
                } else {
                    if (it && (it & 31) == 0)
                        ids = page_ids(e, it);
                    load(e, now, it, ids);
                    compute(e, now, it);
                }
            }
            if (more) {
                ids = ids_after;
                mine = tiles_here(f);
                load_q(f);
                if (kTwoStages && mine > 0)
                    load(f, now, 0, ids);
            }
            finish(e);
            if (!more)
                break;
            __syncthreads(); // the join has read the V buffers
            e = f;
        }
    };

    if constexpr (!SHARES) {
        const int seq = blockIdx.y, len = clampi(a.lens[seq], 0, a.longest);
        run(Segment{seq, (int)blockIdx.x, 0, __builtin_amdgcn_readfirstlane(len), -1}, [](const Segment &, Segment &) { return false; });
    } else {
        const int me = blockIdx.x;
        // sequences without keys have no units: their rows are zeroed here
        for (int s = me; s < a.seqs; s += gridDim.x)
            if (a.lens[s] <= 0 || a.longest == 0)
                for (int64_t u = threadIdx.x; u < (int64_t)a.cache.hkv * a.G * (D / 8); u += 64 * W)
                    reinterpret_cast<u32x4 *>(a.out)[(int64_t)s * a.cache.hkv * a.G * (D / 8) + u] = u32x4{};
        int per = 0;
        const Start from = find_start<64 * W>(a, [&](int all) {
            per = (all * items + (int)gridDim.x - 1) / (int)gridDim.x;
            return me * per / items;
        });
        const int end = min(from.units * items, (me + 1) * per); // in units of items
        int at = me * per, before = from.before, seq = from.seq, len = from.len;
        int spans = 0, first_item = 0, first_seq = 0;
        // the segment that begins at `at`, and the place after it
        auto take = [&](Segment &e) {
            while (at < end && seq < a.seqs) {
                const int r = units_of(a, len), in = at - before * items;
                if (in < r * items) {
                    const int item = in / r, off = in - item * r, n_units = min(r - off, end - at);
                    const bool begins = off == 0, ends = off + n_units == r;
                    e.seq = seq;
                    e.item = __builtin_amdgcn_readfirstlane(item);
                    e.c0 = __builtin_amdgcn_readfirstlane(off << a.unit_shift);
                    e.c1 = __builtin_amdgcn_readfirstlane(min(len, (off + n_units) << a.unit_shift));
                    e.slot = begins && ends ? -1 : 2 * me + begins;
                    if (begins && !ends) { // this share and those up to the item's last unit
                        spans = (at + r - 1) / per - me + 1;
                        first_seq = seq;
                        first_item = item;
                    }
                    at += n_units;
                    return true;
                }
                before += r;
                if (++seq < a.seqs)
                    len = __builtin_amdgcn_readfirstlane(clampi(a.lens[seq], 0, a.longest));
            }
            return false;
        };
        Segment first;
        if (take(first))
            run(first, [&](const Segment &, Segment &f) { return take(f); });
        if (threadIdx.x == 0) {
            a.spans[3 * me] = spans;
            a.spans[3 * me + 1] = first_seq;
            a.spans[3 * me + 2] = first_item;
        }
    }
}

// The item that begins in share blockIdx.x and ends in a later one, one of its
// query heads: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over its
// shares.  Groups of D / 4 lanes take every so many-th share each and are added
// in order; a handful of kilobytes per row, bound by latency.
template <int D, bool F16, int NT> __global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a)
{
    constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
    const int me = blockIdx.x, r = blockIdx.y;
    const int n = a.spans[3 * me], seq = a.spans[3 * me + 1], item = a.spans[3 * me + 2];
    const int h = item % a.cache.hkv, head = item / a.cache.hkv * 16 * NT + r;
    if (n == 0 || head >= a.G)
        return;
    // share i of the item: slot 1 of the first workgroup, slot 0 of the others
    auto row_of = [&](int i) { return (int64_t)(2 * (me + i) + (i == 0)) * 16 * NT + r; };
    float top = kLowest;
    for (int i = threadIdx.x & 63; i < n; i += 64)
        top = fmaxf(top, a.stats[2 * row_of(i)]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    const int c = 4 * (threadIdx.x % kLanes), group = threadIdx.x / kLanes;
    f32x4 x = {};
    float sum = 0.f;
#pragma unroll 4
    for (int i = group; i < n; i += kGroups) {
        const int64_t at = row_of(i);
        const float f = exp2_fast(a.stats[2 * at] - top);
        sum += f * a.stats[2 * at + 1];
        x += f * *reinterpret_cast<const f32x4 *>(a.part + at * D + c);
    }
    __shared__ __attribute__((aligned(16))) float s_x[kGroups][D];
    __shared__ float s_l[kGroups];
    *reinterpret_cast<f32x4 *>(&s_x[group][c]) = x;
    if (c == 0)
        s_l[group] = sum;
    __syncthreads();
    if ((int)threadIdx.x < D / 2) {
        const int e = 2 * threadIdx.x;
        float all = 0.f, u = 0.f, v = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            all += s_l[i];
            u += s_x[i][e];
            v += s_x[i][e + 1];
        }
        const float inv = all == 0.f ? 1.f : 1.f / all;
        const int64_t row = ((int64_t)seq * a.cache.hkv + h) * a.G + head;
        *reinterpret_cast<uint32_t *>(a.out + row * D + e) = pack_half_x2<F16>(u * inv, v * inv);
    }
}

template <int D, bool F16, int NT> hipError_t run(const DecodeArgs &a, const DecodePlan &p, hipStream_t st)
{
    if (p.shares == 0) {
        const dim3 grid(a.cache.hkv * a.groups, a.seqs);
        if (p.waves == 2)
            attn_decode_kernel<D, F16, NT, 2, false><<<grid, 128, 0, st>>>(a);
        else
            attn_decode_kernel<D, F16, NT, 8, false><<<grid, 512, 0, st>>>(a);
        return hipGetLastError();
    }
    attn_decode_kernel<D, F16, NT, 8, true><<<(unsigned)p.shares, 512, 0, st>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    attn_join_kernel<D, F16, NT><<<dim3((unsigned)p.shares, std::min(a.G, 16 * NT)), 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int D, bool F16> hipError_t run_d(const DecodeArgs &a, const DecodePlan &p, hipStream_t st)
{
    return p.nt == 1 ? run<D, F16, 1>(a, p, st) : p.nt == 2 ? run<D, F16, 2>(a, p, st) : run<D, F16, 3>(a, p, st);
}

} // namespace

// Query heads of a key-value head are covered by groups of nt tiles of 16, at
// most three, each of which reads the cache.  The registers of one tile and, of
// 64 channels, of all three (215) hold two stages; of 128, two tiles have one
// stage (244), and three, with one stage, spill 56 or 57 registers in shares.
// 32768 tokens at most: 32 contexts of 48/1 heads of 128 95 us (3.0 TB/s), 16 of
// 40/2 59 (4.8); of 64, 64 contexts of 48/1 66 (4.6), and of 71/1, two groups
// that fetch it twice, 110 (2.7).
// Equal shares cost a look for the share's start and the join.  A workgroup per
// item is quicker where an item is two tiles a wave at most (one sequence, 8
// heads: 7.7 us for 512 tokens, and 8.8 for 513 in shares; past that each tile a
// wave adds 2.1 us), and for caches of up to 1024 keys where the items fill the
// device twice (128 sequences of up to 900 tokens, 4 heads: 32 us, and 40);
// there the longest item, alone at the end, takes no more than some 20 us.
// Workgroups per item have two waves, of which four fit a compute unit, where
// there are many of them or few keys (128 sequences of up to 200, 8 heads: 14.2
// us, and 20.6 with eight waves; one of 64: 3.3 us, and 3.7), else eight (one of
// 333: 6.4 us, and 7.0 with two).
// Shares are cut at whole units: 8 tiles, one for each wave, where there are many
// items, so that the items of a sequence are cut at the same pages, which
// neighbouring workgroups then read together (20 sequences of up to 3000, 32
// heads: 83 us, and 126 in units of one tile); fewer where an item is spread over
// more than sixteen shares and a unit of 8 would leave shares empty or unequal (one
// sequence of 2048 tokens, 8 heads: 9.7 us in units of 2, 11.6 of 8; of 17911:
// 21.2 in units of 4, 23.0 of 8).
DecodePlan plan_decode(int64_t seqs, int64_t hkv, int64_t G, int64_t longest, int cus)
{
    DecodePlan p;
    const int64_t tiles = (G + 15) / 16;
    p.groups = (tiles + 2) / 3;
    p.nt = (tiles + p.groups - 1) / p.groups;
    const int64_t items = seqs * hkv * p.groups;
    const bool direct = longest <= 512 || (longest <= 1024 && items >= 2 * cus) ||
                        items * (longest / 64 + 1) >= (int64_t(1) << 30) - 2 * cus; // units are counted in 32 bits
    p.shares = direct ? 0 : cus;
    p.waves = longest <= 128 || items > cus ? 2 : 8;
    p.unit_shift = 16 * items >= cus ? 8 : items * ((longest + 63) / 64) > 2 * cus ? 7 : 6;
    return p;
}

hipError_t launch_attn_decode(const DecodeArgs &a, int D, bool f16, const DecodePlan &p, hipStream_t st)
{
    if (D == 64)
        return f16 ? run_d<64, true>(a, p, st) : run_d<64, false>(a, p, st);
    return f16 ? run_d<128, true>(a, p, st) : run_d<128, false>(a, p, st);
}

} // namespace tf
