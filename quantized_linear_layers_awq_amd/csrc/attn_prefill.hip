// Causal attention of packed prompts with grouped heads, over packed keys or
// over the pages of a cache that already holds earlier tokens:
//
//   o[i][j] = sum_t softmax_t(scale q[i][j] . k[t]) v[t],  t <= n - new + i
//
// for the new tokens i of a sequence whose n keys end with them, and the
// G = Hq / Hkv query heads j of a key-value head.  The last new token sees
// every key; a token that sees none (more queries than keys) gives zeros.
//
// What bounds it: 4 D operations per visible (token, key, head), on MFMAs;
// beside them one exponential per score, which the vector unit issues at a
// quarter of its rate -- for D = 128 about as long as the products take.
//  - The rows of one (sequence, key-value head) are its tokens times its G
//    heads, token-major, so heads that share keys share tiles of them for any
//    G, and a tile of rows spans few tokens (little waste at the diagonal).
//    A workgroup of 4 waves takes 128 rows, 32 per wave, one row per MFMA
//    column (32x32x16).
//  - K and V come in tiles of 64 keys by LDS-DMA, two buffers each, the next
//    tile's copies running while this one is computed: one barrier per tile.
//    Units of 16 bytes are XOR-swizzled by row on the way in, K so that 16
//    rows read at one channel fall into 16 bank groups, V so that the
//    transpose reads do.
//  - Wave w copies rows 16 w .. 16 w + 15, which lie in one page (pages hold a
//    multiple of 16 tokens): one page id per wave and tile.
//  - Workgroups are ordered with the last rows first (they see the most keys),
//    and with the key-value head fastest, so that an XCD's L2 serves the same
//    heads throughout.
#include "tf_attn.h"

namespace tf {

namespace {

constexpr int kWaves = 4;
constexpr int kRowsWave = 32;
constexpr int kRowsBlock = kWaves * kRowsWave;
constexpr int kKeys = 64;

template <int D> __device__ constexpr int k_swz(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D> __device__ constexpr int v_swz(int row) { return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3); }

// true where a 16-bit half has an exponent of all ones, at bit 15 / 31
template <bool F16> __device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w)
{
    return F16 ? ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

template <int D, bool F16, bool PAGED> __global__ __launch_bounds__(64 * kWaves, 2) void attn_prefill_kernel(PrefillArgs a)
{
    constexpr int kSteps = D / 16;          // MFMA steps over channels
    constexpr int kTiles = D / 32;          // 32-channel tiles of O^T
    constexpr int kRow = 2 * D;             // bytes of a row
    constexpr int kChunks = D / 8;          // 16-byte units of a row
    constexpr int kRowsPerDma = 1024 / kRow;
    constexpr int kDmas = 16 / kRowsPerDma; // of a wave's 16 rows
    constexpr int kBuf = kKeys * kRow;
    __shared__ __attribute__((aligned(16))) uint8_t lds[4 * kBuf]; // K, V, K, V
    __shared__ uint32_t s_bad[kWaves];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, n = lane & 31;
    const int h = blockIdx.x % a.hkv, seq = blockIdx.x / a.hkv;
    const int tile = gridDim.y - 1 - blockIdx.y;

    const int q0 = clampi(a.cu_q[seq], 0, a.tokens);
    const int all_new = max(clampi(a.cu_q[seq + 1], 0, a.tokens) - q0, 0);
    const int fresh = min(all_new, a.longest); // tokens past the bound are not computed
    const int64_t row0 = (int64_t)tile * kRowsBlock;
    const int64_t rows = (int64_t)fresh * a.G;
    if (row0 >= rows)
        return;
    int k0 = 0, keys;
    if constexpr (PAGED) {
        keys = clampi(a.lens[seq], 0, a.cache.width << a.cache.page_shift);
    } else {
        k0 = clampi(a.cu_k[seq], 0, a.keys);
        keys = max(clampi(a.cu_k[seq + 1], 0, a.keys) - k0, 0);
    }
    // keys visible to the first and the last token of the workgroup
    const int first = (int)(row0 / a.G);
    const int last = (int)((min(rows, row0 + kRowsBlock) - 1) / a.G);
    const int shift = keys - all_new + 1;
    const int seen_first = clampi(shift + first, 0, keys), seen_last = clampi(shift + last, 0, keys);
    const int tiles = (seen_last + kKeys - 1) / kKeys;

    // this lane's row: token and head
    const int64_t row = row0 + kRowsWave * wave + n;
    const int64_t row_in = min(row, rows - 1);
    const int token = (int)(row_in / a.G), head = h * a.G + (int)(row_in % a.G);
    const int seen = clampi(shift + token, 0, keys);
    u32x4 q[kSteps];
    {
        const uint16_t *p = a.q + (int64_t)(q0 + token) * a.q_token + (int64_t)head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[s] = load16(p + 16 * s);
    }

    // LDS-DMA of tile t into buffer b: unit u of row r lands at u ^ swz(r)
    const int32_t *const table = PAGED ? a.cache.tables + (int64_t)seq * a.cache.width : nullptr;
    const int d_row = lane / kChunks, d_unit = lane % kChunks;
    const int kstride = PAGED ? kRow : 2 * (int)a.k_token, vstride = PAGED ? kRow : 2 * (int)a.v_token;
    uint32_t k_voff[kDmas], v_voff[kDmas];
#pragma unroll
    for (int i = 0; i < kDmas; ++i) {
        const int r = kRowsPerDma * i + d_row; // within the wave's 16 rows
        k_voff[i] = r * kstride + 16 * (d_unit ^ k_swz<D>(r));
        v_voff[i] = r * vstride + 16 * (d_unit ^ v_swz<D>(r));
    }
    auto page_of = [&](int t) { // of the wave's rows of tile t; uniform
        const int key = kKeys * t + 16 * wave;
        return PAGED && key < keys ? table[key >> a.cache.page_shift] : -1;
    };
    auto fetch = [&](int t, int b, int page) {
        const int key = kKeys * t + 16 * wave;
        const int have = clampi(keys - key, 0, 16);
        Rsrc kr, vr;
        if constexpr (PAGED) {
            const bool ok = page >= 0 && page < a.cache.pages;
            const int64_t at = (((int64_t)(ok ? page : 0) * a.hkv + h) << a.cache.page_shift) + (key & ((1 << a.cache.page_shift) - 1));
            const uint32_t bytes = ok ? have * kRow : 0;
            kr = make_rsrc_n(a.cache.k + at * D, bytes);
            vr = make_rsrc_n(a.cache.v + at * D, bytes);
        } else {
            const int64_t at = k0 + min(key, max(keys - 1, 0));
            kr = make_rsrc_n(a.k + at * a.k_token + (int64_t)h * a.k_head, have ? (have - 1) * kstride + kRow : 0);
            vr = make_rsrc_n(a.v + at * a.v_token + (int64_t)h * a.v_head, have ? (have - 1) * vstride + kRow : 0);
        }
        uint8_t *const kb = lds + 2 * b * kBuf + 16 * wave * kRow, *const vb = kb + kBuf;
#pragma unroll
        for (int i = 0; i < kDmas; ++i)
            dma16(kr, k_voff[i], 0, kb + 1024 * i);
#pragma unroll
        for (int i = 0; i < kDmas; ++i)
            dma16(vr, v_voff[i], 0, vb + 1024 * i);
    };

    // LDS offsets of the operand reads
    uint32_t k_rd[kSteps], v_rd[kTiles];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
        k_rd[s] = n * kRow + 16 * ((2 * s + half) ^ k_swz<D>(n));
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
        const int r = 4 * half + ((lane & 15) >> 2);
        const int u = 4 * c + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        v_rd[c] = kBuf + r * kRow + 16 * (u ^ v_swz<D>(r)) + 8 * (lane & 1);
    }

    f32x16 o[kTiles] = {};
    float m = kLowest, l = 0.f;

    auto compute = [&](int t, const uint8_t *buf, bool masked, bool bad) {
        f32x16 x[2] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
                x[sub] = mfma32x32x16<F16>(*reinterpret_cast<const u32x4 *>(buf + k_rd[s] + 32 * kRow * sub), q[s], x[sub]);
        // row i of x[sub] is key 32 sub + 8 (i / 4) + 4 half + i % 4
        const int left = seen - kKeys * t - 4 * half; // visible keys from this lane's first on
        if (masked) {
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (32 * sub + 8 * (i >> 2) + (i & 3) >= left)
                        x[sub][i] = -INFINITY;
        }
        float top = x[0][0];
#pragma unroll
        for (int i = 1; i < 32; ++i)
            top = fmaxf(top, x[i >> 4][i & 15]);
        top = max_swap32(top) * a.scale_log2 - kHeadroom<F16>;
        if (__builtin_amdgcn_ballot_w64(top > m + kRescaleSlack)) {
            const float to = fmaxf(m, top), f = exp2_fast(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                o[c] *= f;
        }
        // P rounds to the inputs' type (nearest even) for the MFMA; the sum is
        // kept in fp32 over the unrounded values
        u32x4 p[4];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float e0 = exp2_fast(x[i >> 4][i & 15] * a.scale_log2 - m);
            const float e1 = exp2_fast(x[i >> 4][(i & 15) + 1] * a.scale_log2 - m);
            sum += e0 + e1;
            p[i >> 3][(i & 7) >> 1] = pack_half_x2<F16>(e0, e1);
        }
        l += sum;
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const u32x2 lo = lds_read_tr(buf + v_rd[c] + 16 * ks * kRow);
                const u32x2 hi = lds_read_tr(buf + v_rd[c] + (16 * ks + 8) * kRow);
                u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
                if (masked && bad) {
                    // An infinity or NaN in this tile of V, at a key that some rows
                    // may not see: 0 V would spoil them.  Multiply with V's finite
                    // values, and add each kind of non-finite value where a row
                    // sees one (counted by a product of truth values).
                    u32x4 vis;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = 16 * ks + 8 * (j >> 1) + 2 * (j & 1);
                        const uint32_t one = F16 ? 0x3C00u : 0x3F80u;
                        vis[j] = (key < left ? one : 0u) | (key + 1 < left ? one << 16 : 0u);
                    }
                    u32x4 fin = v;
#pragma unroll 1
                    for (int kind = 0; kind < 3; ++kind) {
                        u32x4 is = {};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                const uint32_t b = (v[j] >> e) & 0xFFFFu, inf = F16 ? 0x7C00u : 0x7F80u;
                                if (kind == 0 ? b == inf : kind == 1 ? b == (inf | 0x8000u) : (b & 0x7FFFu) > inf) {
                                    is[j] |= (F16 ? 0x3C00u : 0x3F80u) << e;
                                    fin[j] &= ~(0xFFFFu << e);
                                }
                            }
                        const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : NAN;
                        const f32x16 seen_of = mfma32x32x16<F16>(is, vis, f32x16{});
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[c][i] += seen_of[i] > 0.f ? add : 0.f;
                    }
                    o[c] = mfma32x32x16<F16>(fin, p[ks], o[c]);
                } else {
                    o[c] = mfma32x32x16<F16>(v, p[ks], o[c]);
                }
            }
    };

    if (tiles > 0) {
        fetch(0, 0, page_of(0));
        int next_page = page_of(1);
        for (int t = 0; t < tiles; ++t) {
            uint8_t *const buf = lds + 2 * (t & 1) * kBuf;
            const bool masked = kKeys * (t + 1) > seen_first;
            wait_vmcnt<0>(); // the wave's copies of tile t
            if (masked) {
                // does V of this tile hold anything but finite numbers?
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < kDmas; ++i) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(buf + kBuf + 16 * wave * kRow + 1024 * i + 16 * lane);
                    w |= nonfinite_halves<F16>(v[0]) | nonfinite_halves<F16>(v[1]) | nonfinite_halves<F16>(v[2]) |
                         nonfinite_halves<F16>(v[3]);
                }
                const bool any = __builtin_amdgcn_ballot_w64(w != 0) != 0;
                if (lane == 0)
                    s_bad[wave] = any;
                wait_lgkmcnt0();
            }
            lds_barrier(); // everybody's copies are there, and tile t - 1 is used up
            if (t + 1 < tiles)
                fetch(t + 1, (t + 1) & 1, next_page);
            next_page = page_of(t + 2);
            if (masked) {
                const bool bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
                if (__builtin_amdgcn_readfirstlane((int)bad))
                    compute(t, buf, true, true);
                else
                    compute(t, buf, true, false);
                if (t + 1 < tiles)
                    lds_barrier(); // s_bad is read before the next tile writes it
            } else {
                compute(t, buf, false, false);
            }
        }
    }

    l = sum_swap32(l);
    const float inv = l == 0.f ? 1.f : 1.f / l;
    if (row < rows) {
        uint16_t *const p = a.out + ((int64_t)(q0 + token) * a.hkv * a.G + head) * D + 4 * half;
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const u32x2 w = {pack_half_x2<F16>(o[c][i] * inv, o[c][i + 1] * inv),
                                 pack_half_x2<F16>(o[c][i + 2] * inv, o[c][i + 3] * inv)};
                *reinterpret_cast<u32x2 *>(p + 32 * c + 2 * i) = w;
            }
    }
}

template <int D, bool F16, bool PAGED> hipError_t run(const PrefillArgs &a, int64_t seqs, hipStream_t st)
{
    const int64_t tiles = ((int64_t)a.longest * a.G + kRowsBlock - 1) / kRowsBlock;
    attn_prefill_kernel<D, F16, PAGED><<<dim3((unsigned)(a.hkv * seqs), (unsigned)tiles), 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_attn_prefill(const PrefillArgs &a, int D, bool f16, bool paged, int64_t seqs, hipStream_t st)
{
    if (D == 64)
        return paged ? f16 ? run<64, true, true>(a, seqs, st) : run<64, false, true>(a, seqs, st)
               : f16 ? run<64, true, false>(a, seqs, st)
                     : run<64, false, false>(a, seqs, st);
    return paged ? f16 ? run<128, true, true>(a, seqs, st) : run<128, false, true>(a, seqs, st)
           : f16 ? run<128, true, false>(a, seqs, st)
                 : run<128, false, false>(a, seqs, st);
}

} // namespace tf
