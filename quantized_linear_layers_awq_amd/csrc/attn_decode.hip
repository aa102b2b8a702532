// Attention of one new token per sequence over a paged key-value cache:
//
//   o[s][j] = sum_t softmax_t(scale q[s][j] . k[t]) v[t],  t < lens[s]
//
// for the G = Hq / Hkv query heads j of each key-value head.
//
// What bounds it: the cache is read once, 4 D bytes per token and key-value
// head against 4 G D operations, so HBM does.  The kernel is a stream of
// key tiles with the arithmetic hidden under it:
//  - One workgroup of 8 waves per (chunk of keys, key-value head, sequence,
//    group of 16 NT query heads).  Each wave takes every eighth 32-key tile
//    of the chunk on its own: K goes from memory straight into MFMA operand
//    registers, V through the wave's own LDS buffer (row-major in, transposed
//    out), the next tile's loads in flight meanwhile.  No barrier before the
//    end.
//  - Both products run on 16x16x32 MFMAs with the query heads as columns, so
//    the heads of a group share one read of the cache.
//  - Page ids of 32 tiles are fetched by one load per wave (a lane per
//    16-key run) and read out lane by lane, off the critical path.
//  - The waves' (m, l, O) are joined in LDS in wave order.  With one chunk
//    the workgroup writes the output; otherwise it writes fp32 partials and
//    attn_join_kernel adds the chunks in order.  No atomics.
#include "tf_attn.h"

namespace tf {

namespace {

constexpr int kWaves = 8;
constexpr int kTile = 32;

template <int D> struct Stage {
    u32x4 k[2][D / 32]; // sub-tile of 16 keys, 32-channel step
    u32x4 v[2][D / 32]; // 16 rows as they lie in memory, 1 KiB per load
};

template <int D> constexpr int v_swz(int row) { return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3); }

template <int D, bool F16, int NT> __global__ __launch_bounds__(64 * kWaves, 2) void attn_decode_kernel(DecodeArgs a)
{
    constexpr int kSteps = D / 32;   // MFMA steps over channels
    constexpr int kTiles = D / 16;   // 16-channel tiles of O^T
    constexpr int kRow = 2 * D;      // bytes of a row
    constexpr int kChunks = D / 8;   // 16-byte units of a row
    constexpr int kRowsPerLoad = 1024 / kRow;
    constexpr int kWaveBytes = kTile * kRow; // V of a tile; in the join, 16 heads of D floats
    static_assert(kWaveBytes == 16 * D * 4, "the join reuses the V buffers");
    __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kWaveBytes];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, n = lane & 15;
    const int h = blockIdx.x % a.cache.hkv, group = blockIdx.x / a.cache.hkv;
    const int seq = blockIdx.y, split = blockIdx.z;
    const int len = clampi(a.lens[seq], 0, a.longest);
    const int c0 = split * a.chunk, c1 = min(len, c0 + a.chunk);
    if (c1 <= c0 && a.splits > 1)
        return; // the join reads only the chunks that a sequence has
    const int tiles = c1 > c0 ? (c1 - c0 + kTile - 1) / kTile : 0;
    const int row0 = group * 16 * NT; // first query head of the group here

    // Q^T operands: column n is head row0 + 16 nt + n
    u32x4 q[NT][kSteps];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = min(row0 + 16 * nt + n, a.G - 1);
        const uint16_t *p = a.q + seq * a.q_token + (int64_t)(h * a.G + r) * a.q_head + 8 * g;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[nt][s] = load16(p + 32 * s);
    }

    const int32_t *table = a.cache.tables + (int64_t)seq * a.cache.width;
    const int page_mask = (1 << a.cache.page_shift) - 1;
    const int64_t page_elems = (int64_t)D << a.cache.page_shift;
    uint8_t *const vbuf = lds + wave * kWaveBytes;

    // lane L: the page of 16-key run L % 2 of this wave's tile it0 + L / 2
    auto page_ids = [&](int it0) {
        const int key = c0 + kTile * (wave + kWaves * (it0 + (lane >> 1))) + 16 * (lane & 1);
        int id = -1;
        if (key < c1)
            id = table[key >> a.cache.page_shift];
        return id >= 0 && id < a.cache.pages ? id : -1;
    };
    const uint32_t k_off = n * kRow + 16 * g, v_off = 16 * lane;
    auto load = [&](Stage<D> &st, int it, int ids) {
        const int key0 = c0 + kTile * (wave + kWaves * it);
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const int key = key0 + 16 * sub;
            const int id = __builtin_amdgcn_readlane(ids, (2 * it + sub) & 63);
            const int rows = id < 0 ? 0 : rows_before(c1, key);
            const int64_t at = ((int64_t)max(id, 0) * a.cache.hkv + h) * page_elems + (int64_t)(key & page_mask) * D;
            const Rsrc kr = make_rsrc_n(a.cache.k + at, rows * kRow), vr = make_rsrc_n(a.cache.v + at, rows * kRow);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                st.k[sub][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(kr, k_off + 64 * s, 0, 0));
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                st.v[sub][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(vr, v_off + 1024 * s, 0, 0));
        }
    };

    f32x4 o[NT][kTiles] = {}, l[NT] = {};
    float m[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        m[nt] = kLowest;
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

    auto compute = [&](const Stage<D> &st, int it) {
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int r = 16 * sub + kRowsPerLoad * s + wr_row;
                *reinterpret_cast<u32x4 *>(vbuf + r * kRow + 16 * (wr_unit ^ v_swz<D>(r))) = st.v[sub][s];
            }
        const int key0 = c0 + kTile * (wave + kWaves * it);
        u32x4 p[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            f32x4 x[2] = {};
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    x[sub] = mfma16x16x32<F16>(st.k[sub][s], q[nt][s], x[sub]);
            if (key0 + kTile > c1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (key0 + 16 * (i >> 2) + 4 * g + (i & 3) >= c1)
                        x[i >> 2][i & 3] = -INFINITY;
            }
            float top = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])),
                              fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
            top = max_swap32(max_swap16(top)) * a.scale_log2 - kHeadroom<F16>;
            if (__builtin_amdgcn_ballot_w64(top > m[nt] + kRescaleSlack)) {
                const float to = fmaxf(m[nt], top), f = exp2_fast(m[nt] - to);
                m[nt] = to;
                l[nt] *= f;
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    o[nt][t] *= f;
            }
            // P rounds to the inputs' type for the MFMA; the sum is taken over the
            // rounded values (a product with ones), so that rounding cancels
            // where a row's weight sits on few keys
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[nt][j] = pack_half_x2<F16>(exp2_fast(x[j >> 1][2 * (j & 1)] * a.scale_log2 - m[nt]),
                                             exp2_fast(x[j >> 1][2 * (j & 1) + 1] * a.scale_log2 - m[nt]));
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

    // this wave's tiles: wave, wave + 8, ...; two stages, the loads of one in
    // flight while the other is computed
    const int mine = tiles > wave ? (tiles - wave + kWaves - 1) / kWaves : 0;
    if constexpr (D == 128 && NT > 1) {
        // more heads: the registers hold one stage beside the accumulators, and
        // the device's other waves cover its loads
        int ids = -1;
        for (int it = 0; it < mine; ++it) {
            if ((it & 31) == 0)
                ids = page_ids(it);
            Stage<D> s0;
            load(s0, it, ids);
            compute(s0, it);
        }
    } else if (mine > 0) {
        Stage<D> s0, s1;
        int ids = page_ids(0);
        load(s0, 0, ids);
        for (int it = 0; it < mine; it += 2) {
            if (it + 1 < mine)
                load(s1, it + 1, ids);
            compute(s0, it);
            if (it + 2 < mine) {
                if (((it + 2) & 31) == 0)
                    ids = page_ids(it + 2);
                load(s0, it + 2, ids);
            }
            if (it + 1 < mine)
                compute(s1, it + 1);
        }
    }

    // join the waves, 16 heads at a time
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int heads = min(16, a.G - row0 - 16 * nt);
        if (heads <= 0)
            break;
        __syncthreads();
        float *const mine_o = reinterpret_cast<float *>(lds + wave * kWaveBytes);
        if (n < heads) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                *reinterpret_cast<f32x4 *>(mine_o + n * D + 4 * ((4 * t + g) ^ n)) = o[nt][t]; // 4-float units, XORed
                                                                                               // by head: no bank conflicts
            if (g == 0) {
                s_m[wave][n] = m[nt];
                s_l[wave][n] = l[nt][0];
            }
        }
        __syncthreads();
        for (int u = threadIdx.x; u < heads * (D / 2); u += 64 * kWaves) {
            const int r = u / (D / 2), c = 2 * (u % (D / 2));
            float top = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                top = fmaxf(top, s_m[w][r]);
            float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = exp2_fast(s_m[w][r] - top);
                const float *const p = reinterpret_cast<const float *>(lds + w * kWaveBytes) + r * D + 4 * ((c >> 2) ^ r) + (c & 3);
                sum += f * s_l[w][r];
                x += f * p[0];
                y += f * p[1];
            }
            const int64_t at = (int64_t)seq * a.cache.hkv * a.G + h * a.G + row0 + 16 * nt + r;
            if (a.splits == 1) {
                const float inv = sum == 0.f ? 1.f : 1.f / sum;
                *reinterpret_cast<uint32_t *>(a.out + at * D + c) = pack_half_x2<F16>(x * inv, y * inv);
            } else {
                float *const part = a.part + (at * a.splits + split) * D + c;
                part[0] = x;
                part[1] = y;
                if (c == 0) {
                    a.stats[2 * (at * a.splits + split)] = top;
                    a.stats[2 * (at * a.splits + split) + 1] = sum;
                }
            }
        }
    }
}

// One query row per workgroup: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i
// over the row's chunks.  The four waves take every fourth chunk each and are
// added in wave order; a handful of kilobytes per row, bound by latency.
template <int D, bool F16> __global__ __launch_bounds__(256) void attn_join_kernel(DecodeArgs a)
{
    constexpr int kPer = D / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const int seq = (int)(row / (a.cache.hkv * a.G));
    const int len = clampi(a.lens[seq], 0, a.longest);
    const int n = (len + a.chunk - 1) / a.chunk;
    const float *const st = a.stats + 2 * row * a.splits;
    float top = kLowest;
    for (int i = lane; i < n; i += 64)
        top = fmaxf(top, st[2 * i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    float x[kPer] = {}, sum = 0.f;
#pragma unroll 8
    for (int i = wave; i < n; i += 4) {
        const float f = exp2_fast(st[2 * i] - top);
        const float *const p = a.part + (row * a.splits + i) * D + kPer * lane;
        sum += f * st[2 * i + 1];
#pragma unroll
        for (int c = 0; c < kPer; ++c)
            x[c] += f * p[c];
    }
    __shared__ float s_x[4][D], s_l[4];
#pragma unroll
    for (int c = 0; c < kPer; ++c)
        s_x[wave][kPer * lane + c] = x[c];
    if (lane == 0)
        s_l[wave] = sum;
    __syncthreads();
    if ((int)threadIdx.x < D / 2) {
        const int c = 2 * threadIdx.x;
        const float all = s_l[0] + s_l[1] + s_l[2] + s_l[3];
        const float inv = all == 0.f ? 1.f : 1.f / all;
        const float u = s_x[0][c] + s_x[1][c] + s_x[2][c] + s_x[3][c];
        const float v = s_x[0][c + 1] + s_x[1][c + 1] + s_x[2][c + 1] + s_x[3][c + 1];
        *reinterpret_cast<uint32_t *>(a.out + row * D + c) = pack_half_x2<F16>(u * inv, v * inv);
    }
}

template <int D, bool F16, int NT> hipError_t run(const DecodeArgs &a, int seqs, int groups, hipStream_t st)
{
    attn_decode_kernel<D, F16, NT><<<dim3(a.cache.hkv * groups, seqs, a.splits), 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
}

template <int D, bool F16> hipError_t run_d(const DecodeArgs &a, int seqs, int nt, int groups, hipStream_t st)
{
    hipError_t e = nt == 1   ? run<D, F16, 1>(a, seqs, groups, st)
                   : nt == 2 ? run<D, F16, 2>(a, seqs, groups, st)
                             : run<D, F16, 3>(a, seqs, groups, st);
    if (e != hipSuccess || a.splits == 1)
        return e;
    attn_join_kernel<D, F16><<<dim3((unsigned)(seqs * a.cache.hkv * a.G)), 256, 0, st>>>(a);
    return hipGetLastError();
}

} // namespace

// Query heads of a key-value head are covered by groups of nt tiles of 16, at
// most three (the accumulators of more do not fit the registers beside two
// stages).  The cache's length is cut into chunks so that the grid at the
// longest length fills the device a few times over, each chunk a whole
// number of rounds of the waves' tiles.
DecodePlan plan_decode(int64_t seqs, int64_t hkv, int64_t G, int64_t longest, int cus)
{
    DecodePlan p;
    const int64_t tiles = (G + 15) / 16;
    p.groups = (tiles + 2) / 3;
    p.nt = (tiles + p.groups - 1) / p.groups;
    const int64_t round = kWaves * kTile;
    const int64_t rounds = std::max<int64_t>(1, (longest + round - 1) / round);
    const int64_t have = std::max<int64_t>(1, seqs * hkv * p.groups), want = 4 * (int64_t)cus;
    int64_t splits = std::min(rounds, std::max<int64_t>(1, want / have));
    if (longest <= 2 * round)
        splits = 1;
    const int64_t per = (rounds + splits - 1) / splits;
    p.chunk = per * round;
    p.splits = (rounds + per - 1) / per;
    return p;
}

hipError_t launch_attn_decode(const DecodeArgs &a, int D, bool f16, int64_t seqs, const DecodePlan &p, hipStream_t st)
{
    const int s = (int)seqs, nt = (int)p.nt, gr = (int)p.groups;
    if (D == 64)
        return f16 ? run_d<64, true>(a, s, nt, gr, st) : run_d<64, false>(a, s, nt, gr, st);
    return f16 ? run_d<128, true>(a, s, nt, gr, st) : run_d<128, false>(a, s, nt, gr, st);
}

} // namespace tf
