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
constexpr int kKeys = 64;

template <int D> __device__ constexpr int k_swz(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D> __device__ constexpr int v_swz(int row) { return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3); }

// true where a 16-bit half has an exponent of all ones, at bit 15 / 31
template <bool F16> __device__ __forceinline__ uint32_t nonfinite_halves(uint32_t w)
{
    return F16 ? ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// acc + the sum of two packed probabilities, in fp32
template <bool F16> __device__ __forceinline__ float dot_ones(uint32_t w, float acc)
{
    if constexpr (F16)
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{(_Float16)1.f, (_Float16)1.f}, acc, false);
    else
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(s16x2, w), s16x2{0x3F80, 0x3F80}, acc, false);
}

template <int D, bool F16, bool PAGED, int RT> __global__ __launch_bounds__(64 * kWaves, RT == 2 ? 1 : 2) void attn_prefill_kernel(PrefillArgs a)
{
    constexpr int kSteps = D / 16;          // MFMA steps over channels
    constexpr int kTiles = D / 32;          // 32-channel tiles of O^T
    constexpr int kRow = 2 * D;             // bytes of a row
    constexpr int kChunks = D / 8;          // 16-byte units of a row
    constexpr int kRowsPerDma = 1024 / kRow;
    constexpr int kDmas = 16 / kRowsPerDma; // of a wave's 16 rows
    constexpr int kBuf = kKeys * kRow;
    constexpr int kRowsBlock = kWaves * 32 * RT;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[]; // K, K, V, V
    __shared__ uint32_t s_bad[2][kWaves];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, n = lane & 31;
    const int h = blockIdx.x % a.hkv, seq = blockIdx.x / a.hkv;
    const int block = gridDim.y - 1 - blockIdx.y;

    const int q0 = clampi(a.cu_q[seq], 0, a.tokens);
    const int all_new = max(clampi(a.cu_q[seq + 1], 0, a.tokens) - q0, 0);
    const int fresh = min(all_new, a.longest); // tokens past the bound are not computed
    const int64_t row0 = (int64_t)block * kRowsBlock;
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
    const int shift = keys - all_new + 1;
    const int seen_first = clampi(shift + (int)(row0 / a.G), 0, keys);
    const int seen_last = clampi(shift + (int)((min(rows, row0 + kRowsBlock) - 1) / a.G), 0, keys);
    const int tiles = (seen_last + kKeys - 1) / kKeys;
    const int whole = seen_first / kKeys; // tiles that every row sees whole

    // this lane's rows: token, head and visible keys
    int64_t row[RT], at_out[RT];
    int seen[RT];
    u32x4 q[RT][kSteps];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        row[r] = row0 + 32 * (RT * wave + r) + n;
        const int64_t in = min(row[r], rows - 1);
        const int token = (int)(in / a.G), head = h * a.G + (int)(in % a.G);
        seen[r] = clampi(shift + token, 0, keys);
        at_out[r] = ((int64_t)(q0 + token) * a.hkv * a.G + head) * D + 4 * half;
        const uint16_t *p = a.q + (int64_t)(q0 + token) * a.q_token + (int64_t)head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[r][s] = load16(p + 16 * s);
    }

    // LDS-DMA of tile t: unit u of row i lands at u ^ swz(i)
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
    auto fetch = [&](bool is_k, int t, int page) {
        const int key = kKeys * t + 16 * wave;
        const int have = clampi(keys - key, 0, 16);
        const uint16_t *base = PAGED ? (is_k ? a.cache.k : a.cache.v) : is_k ? a.k : a.v;
        Rsrc rs;
        if constexpr (PAGED) {
            const bool ok = page >= 0 && page < a.cache.pages;
            const int64_t at = (((int64_t)(ok ? page : 0) * a.hkv + h) << a.cache.page_shift) + (key & ((1 << a.cache.page_shift) - 1));
            rs = make_rsrc_n(base + at * D, ok ? have * kRow : 0);
        } else {
            const int64_t at = k0 + min(key, max(keys - 1, 0));
            rs = make_rsrc_n(base + at * (is_k ? a.k_token : a.v_token) + (int64_t)h * (is_k ? a.k_head : a.v_head),
                             have ? (have - 1) * (is_k ? kstride : vstride) + kRow : 0);
        }
        uint8_t *const to = lds + ((is_k ? 0 : 2) + (t & 1)) * kBuf + 16 * wave * kRow;
#pragma unroll
        for (int i = 0; i < kDmas; ++i)
            dma16(rs, is_k ? k_voff[i] : v_voff[i], 0, to + 1024 * i);
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
        v_rd[c] = 2 * kBuf + r * kRow + 16 * (u ^ v_swz<D>(r)) + 8 * (lane & 1);
    }

    f32x16 o[RT][kTiles] = {}, x[RT][2];
    float m[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        m[r] = kLowest, l[r] = 0.f;

    // element i of x[r][sub] is the score of key 64 t + 32 sub + 8 (i / 4) + 4 half + i % 4
    auto scores = [&](int t, f32x16 (&y)[RT][2]) {
        const uint8_t *const buf = lds + (t & 1) * kBuf;
#pragma unroll
        for (int r = 0; r < RT; ++r)
            y[r][0] = f32x16{}, y[r][1] = f32x16{};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const u32x4 k = *reinterpret_cast<const u32x4 *>(buf + k_rd[s] + 32 * kRow * sub);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    y[r][sub] = mfma32x32x16<F16>(k, q[r][s], y[r][sub]);
            }
    };
    auto hide = [&](int t, f32x16 (&y)[RT][2]) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int left = seen[r] - kKeys * t - 4 * half; // visible keys from this lane's first on
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (32 * (i >> 4) + 8 * ((i & 15) >> 2) + (i & 3) >= left)
                    y[r][i >> 4][i & 15] = -INFINITY;
        }
    };
    auto highest = [&](const f32x16 (&y)[RT][2], float (&top)[RT]) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float t0 = y[r][0][0], t1 = y[r][1][0];
#pragma unroll
            for (int i = 1; i < 15; i += 2) {
                t0 = fmaxf(fmaxf(t0, y[r][0][i]), y[r][0][i + 1]);
                t1 = fmaxf(fmaxf(t1, y[r][1][i]), y[r][1][i + 1]);
            }
            t0 = fmaxf(fmaxf(t0, y[r][0][15]), t1);
            top[r] = max_swap32(fmaxf(t0, y[r][1][15])) * a.scale_log2 - kHeadroom<F16>;
        }
    };
    auto raise = [&](const float (&top)[RT]) {
        bool grows = false;
#pragma unroll
        for (int r = 0; r < RT; ++r)
            grows |= top[r] > m[r] + kRescaleSlack;
        if (__builtin_amdgcn_ballot_w64(grows)) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float to = fmaxf(m[r], top[r]), f = exp2_fast(m[r] - to);
                m[r] = to;
                l[r] *= f;
#pragma unroll
                for (int c = 0; c < kTiles; ++c)
                    o[r][c] *= f;
            }
        }
    };
    // An infinity or NaN in V at a key that some rows do not see: 0 V would
    // spoil them.  Rows that see it take it here, lane by lane; then it is
    // zeroed in LDS.  Rare: one lane's 4 channels at a time.
    auto mend = [&](int t) {
        uint8_t *const buf = lds + (2 + (t & 1)) * kBuf;
#pragma unroll 1
        for (int key = 0; key < kKeys; ++key)
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) { // channels 32 c + 8 i + 4 half ..
                    const int unit = 4 * c + i;
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(buf + key * kRow + 16 * (unit ^ v_swz<D>(key)) + 8 * half);
                    if (nonfinite_halves<F16>(v[0]) | nonfinite_halves<F16>(v[1])) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t b = v[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
                            const bool odd = nonfinite_halves<F16>(b) != 0;
#pragma unroll
                            for (int r = 0; r < RT; ++r)
                                o[r][c][4 * i + e] += odd && kKeys * t + key < seen[r] ? half_bits_to_f32<F16>(b) : 0.f;
                        }
                    }
                }
        wait_lgkmcnt0();
        lds_barrier();
#pragma unroll 1
        for (int i = 0; i < kDmas; ++i) { // this wave's rows
            u32x4 *const p = reinterpret_cast<u32x4 *>(buf + 16 * wave * kRow + 1024 * i + 16 * lane);
            u32x4 v = *p;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t bad = nonfinite_halves<F16>(v[j]);
                v[j] &= ~((bad & 0x8000u ? 0xFFFFu : 0u) | (bad & 0x80000000u ? 0xFFFF0000u : 0u));
            }
            *p = v;
        }
        wait_lgkmcnt0();
        lds_barrier();
    };

    // Tile t: p from its scores x, while the products of the next tile's
    // scores run; then P V, while the next scores' maximum is taken.
    auto step = [&](int t, auto more, auto masked) {
        f32x16 y[RT][2];
        u32x4 p[RT][4];
        if constexpr (more)
            scores(t + 1, y);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const uint32_t w = pack_half_x2<F16>(exp2_fast(x[r][i >> 4][i & 15] * a.scale_log2 - m[r]),
                                                     exp2_fast(x[r][i >> 4][(i & 15) + 1] * a.scale_log2 - m[r]));
                p[r][i >> 3][(i & 7) >> 1] = w;
                l[r] = dot_ones<F16>(w, l[r]);
            }
        if constexpr (more && masked)
            hide(t + 1, y);
        float top[RT];
        if constexpr (more)
            highest(y, top);
        const uint8_t *const buf = lds + (t & 1) * kBuf;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                const u32x2 lo = lds_read_tr(buf + v_rd[c] + 16 * ks * kRow);
                const u32x2 hi = lds_read_tr(buf + v_rd[c] + (16 * ks + 8) * kRow);
                const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    o[r][c] = mfma32x32x16<F16>(v, p[r][ks], o[r][c]);
            }
        if constexpr (more) {
            raise(top);
#pragma unroll
            for (int r = 0; r < RT; ++r)
                x[r][0] = y[r][0], x[r][1] = y[r][1];
        }
    };

    if (tiles > 0) {
        fetch(true, 0, page_of(0));
        fetch(false, 0, page_of(0));
        fetch(true, 1, page_of(1));
        int next_page = page_of(1), far_page = page_of(2);
        wait_vmcnt<2 * kDmas>(); // the wave's copies of the first keys
        lds_barrier();
        scores(0, x);
        if (whole == 0)
            hide(0, x);
        float top[RT];
        highest(x, top);
        raise(top);
        // Before tile t: its values and the next tile's keys are there for
        // everybody, and the buffers of the values before and of its own keys
        // are used up.
        auto turn = [&](int t, auto check) {
            wait_vmcnt<0>();
            asm volatile("" ::: "memory"); // no read of LDS moves above the wait
            if constexpr (check) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < kDmas; ++i) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + (2 + (t & 1)) * kBuf + 16 * wave * kRow + 1024 * i + 16 * lane);
                    w |= nonfinite_halves<F16>(v[0]) | nonfinite_halves<F16>(v[1]) | nonfinite_halves<F16>(v[2]) |
                         nonfinite_halves<F16>(v[3]);
                }
                const bool any = __builtin_amdgcn_ballot_w64(w != 0) != 0;
                if (lane == 0)
                    s_bad[t & 1][wave] = any;
                wait_lgkmcnt0();
            }
            lds_barrier();
            if (t + 2 < tiles)
                fetch(true, t + 2, far_page);
            if (t + 1 < tiles)
                fetch(false, t + 1, next_page);
            next_page = far_page;
            far_page = page_of(t + 3);
            if constexpr (check) {
                const uint32_t bad = s_bad[t & 1][0] | s_bad[t & 1][1] | s_bad[t & 1][2] | s_bad[t & 1][3];
                if (__builtin_amdgcn_readfirstlane((int)bad))
                    mend(t);
            }
        };
        int t = 0;
        for (; t + 1 < whole && t + 1 < tiles; ++t) {
            turn(t, std::false_type{});
            step(t, std::true_type{}, std::false_type{});
        }
        for (; t + 1 < tiles; ++t) {
            turn(t, std::true_type{});
            step(t, std::true_type{}, std::true_type{});
        }
        turn(t, std::true_type{});
        step(t, std::false_type{}, std::true_type{});
    }

#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const float sum = sum_swap32(l[r]);
        const float inv = sum == 0.f ? 1.f : 1.f / sum;
        if (row[r] < rows) {
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const u32x2 w = {pack_half_x2<F16>(o[r][c][i] * inv, o[r][c][i + 1] * inv),
                                     pack_half_x2<F16>(o[r][c][i + 2] * inv, o[r][c][i + 3] * inv)};
                    *reinterpret_cast<u32x2 *>(a.out + at_out[r] + 32 * c + 2 * i) = w;
                }
        }
    }
}

template <int D, bool F16, bool PAGED> hipError_t run(const PrefillArgs &a, int64_t seqs, hipStream_t st)
{
    constexpr int RT = PF_RT;
    const int64_t tiles = ((int64_t)a.longest * a.G + 128 * RT - 1) / (128 * RT);
    attn_prefill_kernel<D, F16, PAGED, RT><<<dim3((unsigned)(a.hkv * seqs), (unsigned)tiles), 64 * kWaves, 8 * kKeys * D, st>>>(a);
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
