// Causal attention of packed prompts with grouped heads, over packed keys or
// over the pages of a cache that already holds earlier tokens:
//
//   o[i][j] = sum_t softmax_t(scale q[i][j] . k[t]) v[t],  t <= n - new + i
//
// for the new tokens i of a sequence whose n keys end with them, and the
// G = Hq / Hkv query heads j of a key-value head.  The last new token sees
// every key; a token that sees none (more queries than keys) gives zeros.
//
// What bounds it: 4 D operations per visible (token, key, head), on MFMAs, at
// the clock that the board's power limit leaves them; beside them one
// exponential per score and some four other vector instructions.
//  - The rows of one (sequence, key-value head) are its tokens times its G
//    heads, token-major, so heads that share keys share tiles of them for any
//    G, and a tile of rows spans few tokens (little waste at the diagonal).
//    A workgroup of 4 waves takes 128 rows, 32 per wave, one row per MFMA
//    column (32x32x16); two workgroups run on a compute unit, three for heads
//    of 64 channels (166 to 168 registers).  (64 rows a wave, one wave a SIMD,
//    halves the reads of LDS but left nothing to run in a wave's waits: 8192
//    tokens 655 us, and 512 so; 8 waves sharing the tiles of 256 rows: 503 for
//    those, but a third more where rows are few.)
//  - K and V come in tiles of 64 keys by LDS-DMA, two buffers each, the next
//    tile's copies running while this one is computed: one barrier per tile.
//    Units of 16 bytes are XOR-swizzled by row on the way in, K so that 16
//    rows read at one channel, V so that 4 rows of 64 bytes read by half a
//    wave fall on all 64 banks: no conflicts (by counter).
//  - The scores of the next tile are computed beside this tile's exponentials,
//    its maximum beside the products with V.
//  - Wave w copies rows 16 w .. 16 w + 15, which lie in one page (pages hold a
//    multiple of 16 tokens): one page id per wave and tile.
//  - Workgroups that run side by side share keys and values in their XCD's L2:
//    sequences and groups of heads follow one another where not all of them fit
//    (four sequences of up to 6000 tokens, 64/8 heads: 601 us, and 1029 side by
//    side); where they do, all run side by side, the blocks that see the most
//    keys first, and no workgroup starts for a block that a shorter sequence
//    does not have (7 prompts of up to 1553, 32/8 heads: 120 us, and 142 with
//    those).
//  - Few rows behind many keys: the keys are cut into ranges and joined.
// Measured: one prompt of 8192 tokens, 32/8 heads of 128, 510 to 520 us by the
// board (1055 to 1080 TFLOP/s; a library product of 8192 x 8192 matrices runs at 1116, of
// 16384 at 1348) at 1.81 to 1.87 GHz, where the power limit holds the clock.  MFMAs
// are busy 56 % of its cycles, the vector unit issues in 45 %: together 101 %, they
// seldom run beside each other.  With 64 channels, as many exponentials for
// half the products, 298 us (923 TFLOP/s): MFMAs 46 %, vector issue 66 %.
// Neither is full alone, and the waves spend 42 and 46 % of their time waiting
// to issue.  A copy of the loop without maximum, exponentials and sum takes 457
// and 228 (1205 TFLOP/s both).  71/1 heads of 64, 3 prompts of up to 2048: 107
// us (735).
#include "tf_attn.h"

namespace tf {

namespace {

constexpr int kWaves = 4;
constexpr int kKeys = 64;
constexpr int kMinRange = 4;   // tiles of a range of keys, at least
constexpr int kMaxSplits = 16; // ranges
constexpr int64_t kSlots = 512; // workgroups that run at a time, two a compute unit (of 64 channels 768 would)
constexpr int64_t kL2Share = 3 << 20; // bytes of an XCD's 4 MiB for the keys and values in use

// tiles of a range when the keys of a sequence are cut into `splits`
__device__ __forceinline__ int prefill_range(int keys, int splits)
{
    return splits == 1 ? 1 << 30 : max(kMinRange, ((keys + kKeys - 1) / kKeys + splits - 1) / splits);
}

template <int D> __device__ constexpr int k_swz(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D> __device__ constexpr int v_swz(int row) { return D == 128 ? 4 * (row & 3) : 4 * ((row >> 1) & 1); }

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

template <int D, bool F16, bool PAGED> __global__ __launch_bounds__(64 * kWaves, 2) void attn_prefill_kernel(PrefillArgs a)
{
    constexpr int kSteps = D / 16;          // MFMA steps over channels
    constexpr int kTiles = D / 32;          // 32-channel tiles of O^T
    constexpr int kRow = 2 * D;             // bytes of a row
    constexpr int kChunks = D / 8;          // 16-byte units of a row
    constexpr int kRowsPerDma = 1024 / kRow;
    constexpr int kDmas = 16 / kRowsPerDma; // of a wave's 16 rows
    constexpr int kBuf = kKeys * kRow;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[]; // K, K, V, V
    __shared__ uint32_t s_bad[2][kWaves];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, n = lane & 31;
    int seq, h, block;
    if (a.all_blocks) {
        // only the blocks that there are, last ones first, each level's
        // sequences side by side: lane s holds the number of sequence s
        const int turn = blockIdx.x / a.hkv;
        h = blockIdx.x % a.hkv;
        int mine = 0;
        if (lane < a.seqs) {
            const int from = clampi(a.cu_q[lane], 0, a.tokens), to = clampi(a.cu_q[lane + 1], 0, a.tokens);
            mine = (int)(((int64_t)clampi(to - from, 0, a.longest) * a.G + kPrefillRows - 1) / kPrefillRows);
        }
        // blocks at level b (lane's own b) and above
        auto from_level = [&](int b) {
            int sum = 0;
            for (int s = 0; s < a.seqs; ++s)
                sum += max(__builtin_amdgcn_readlane(mine, s) - b, 0);
            return sum;
        };
        // the highest level that counts more than `turn` blocks from it on,
        // 64 levels at a time
        int low = 0;
        for (int step = a.steps; step > 0; step >>= 6) {
            const uint64_t past = __builtin_amdgcn_ballot_w64(from_level(low + step * lane) > turn);
            if (past == 0)
                return; // no such block
            low += step * (63 - __builtin_clzll(past));
        }
        block = low;
        const int rank = turn - __builtin_amdgcn_readfirstlane(from_level(block + 1)); // among the level's sequences
        const uint64_t there = __builtin_amdgcn_ballot_w64(mine > block);
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(there >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)there, 0));
        seq = __builtin_ctzll(__builtin_amdgcn_ballot_w64(mine > block && before == rank));
    } else {
        // sequence, group of heads, block of rows (last ones first), head (fastest)
        const int groups = a.hkv / a.heads_by, each = a.blocks * a.heads_by;
        const int rest = blockIdx.x % each, group = blockIdx.x / each;
        seq = group / groups;
        h = group % groups * a.heads_by + rest % a.heads_by;
        block = a.blocks - 1 - rest / a.heads_by;
    }

    const int q0 = clampi(a.cu_q[seq], 0, a.tokens);
    const int all_new = max(clampi(a.cu_q[seq + 1], 0, a.tokens) - q0, 0);
    const int fresh = min(all_new, a.longest); // tokens past the bound are not computed
    const int64_t row0 = (int64_t)block * kPrefillRows;
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
    const int seen_last = clampi(shift + (int)((min(rows, row0 + kPrefillRows) - 1) / a.G), 0, keys);
    const int whole = seen_first / kKeys; // tiles that every row sees whole
    // this workgroup's tiles: t0 .. tiles - 1
    const int all_tiles = (seen_last + kKeys - 1) / kKeys, per = prefill_range(keys, a.splits);
    const int split = blockIdx.y, t0 = split * per, tiles = min(all_tiles, t0 + per);
    if (split > 0 && t0 >= all_tiles)
        return; // the join reads only the ranges that a block has

    // this lane's row: token, head and visible keys
    const int64_t row = row0 + 32 * wave + n, row_in = min(row, rows - 1);
    const int token = (int)(row_in / a.G), head = h * a.G + (int)(row_in % a.G);
    const int seen = clampi(shift + token, 0, keys);
    const int64_t row_out = (int64_t)(q0 + token) * a.hkv * a.G + head;
    u32x4 q[kSteps];
    {
        const uint16_t *p = a.q + (int64_t)(q0 + token) * a.q_token + (int64_t)head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            q[s] = load16(p + 16 * s);
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
    // The pages of this wave's rows of 64 tiles, a lane per tile, in one load;
    // a tile's page is read out of its lane, so that it is uniform.
    int ids = -1;
    auto pages_from = [&](int t) {
        if constexpr (PAGED) {
            const int key = kKeys * ((t & ~63) + lane) + 16 * wave;
            ids = key < keys ? table[key >> a.cache.page_shift] : -1;
            ids = ids < a.cache.pages ? ids : -1;
        }
    };
    auto page_of = [&](int t) {
        if constexpr (PAGED)
            return __builtin_amdgcn_readlane(ids, t & 63);
        else
            return 0;
    };
    // Where this wave's rows of the next tile to fetch lie (packed: tiles are
    // fetched in order), or where this head's rows of page 0 lie (paged).
    const uint8_t *k_next, *v_next;
    const int64_t page_bytes = (int64_t)a.hkv * kRow << a.cache.page_shift;
    if constexpr (PAGED) {
        const int64_t at = ((int64_t)h << a.cache.page_shift) * kRow;
        k_next = reinterpret_cast<const uint8_t *>(a.cache.k) + at;
        v_next = reinterpret_cast<const uint8_t *>(a.cache.v) + at;
    } else {
        const int64_t key = k0 + (int64_t)kKeys * t0 + 16 * wave;
        k_next = reinterpret_cast<const uint8_t *>(a.k + key * a.k_token + (int64_t)h * a.k_head);
        v_next = reinterpret_cast<const uint8_t *>(a.v + key * a.v_token + (int64_t)h * a.v_head);
    }
    auto fetch = [&](bool is_k, int t, int page) {
        const int key = kKeys * t + 16 * wave;
        const int have = rows_before(keys, key), stride = is_k ? kstride : vstride;
        const uint8_t *&next = is_k ? k_next : v_next;
        Rsrc rs;
        if constexpr (PAGED) {
            const int64_t at = max(page, 0) * page_bytes + (key & ((1 << a.cache.page_shift) - 1)) * kRow;
            rs = make_rsrc_n(next + at, page < 0 ? 0 : have * kRow);
        } else {
            rs = make_rsrc_n(next, have ? (have - 1) * stride + kRow : 0);
            next += (int64_t)kKeys * stride;
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

    f32x16 o[kTiles] = {}, x[2];
    float m = kLowest, l = 0.f;

    // element i of y[sub] is the score of key 64 t + 32 sub + 8 (i / 4) + 4 half + i % 4
    auto scores = [&](int t, f32x16 (&y)[2]) {
        const uint8_t *const buf = lds + (t & 1) * kBuf;
        y[0] = f32x16{}, y[1] = f32x16{};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
                y[sub] = mfma32x32x16<F16>(*reinterpret_cast<const u32x4 *>(buf + k_rd[s] + 32 * kRow * sub), q[s], y[sub]);
    };
    auto hide = [&](int t, f32x16 (&y)[2]) {
        const int left = seen - kKeys * t - 4 * half; // visible keys from this lane's first on
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * (i >> 4) + 8 * ((i & 15) >> 2) + (i & 3) >= left)
                y[i >> 4][i & 15] = -INFINITY;
    };
    auto highest = [&](const f32x16 (&y)[2]) {
        float t0 = y[0][0], t1 = y[1][0];
#pragma unroll
        for (int i = 1; i < 15; i += 2) {
            t0 = fmaxf(fmaxf(t0, y[0][i]), y[0][i + 1]);
            t1 = fmaxf(fmaxf(t1, y[1][i]), y[1][i + 1]);
        }
        t0 = fmaxf(fmaxf(t0, y[0][15]), t1);
        return held_maximum<F16>(max_swap32(fmaxf(t0, y[1][15])) * a.scale_log2);
    };
    float by; // what the scores x are still to be multiplied with
    auto raise = [&](float top) {
        if (__builtin_amdgcn_ballot_w64(top - m > kRescaleSlack)) {
            const float to = fmaxf(m, top), f = exp2_fast(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
                o[c] *= f;
        }
        by = a.scale_log2;
        if (__builtin_amdgcn_ballot_w64(fabsf(m) >= kLargeScore)) { // rare
            x[0] *= by, x[1] *= by;
            by = 1.f;
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
                            o[c][4 * i + e] += odd && kKeys * t + key < seen ? half_bits_to_f32<F16>(b) : 0.f;
                        }
                    }
                }
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
        lds_barrier();
    };

    // Tile t: p from its scores x, while the products of the next tile's
    // scores run; then P V, while the next scores' maximum is taken.  p rounds
    // to the inputs' type, for MFMA operands of 16 bits are what V is read in;
    // a second product with what the rounding leaves would double P V.  It
    // moves the error against 64 bits from 1.7e-3 of the plain fp32 form to at
    // most 1.8e-3 (bf16; the output's own rounding is the most of both).  The sum
    // is taken over the rounded p, so that their rounding cancels where a row's
    // weight sits on few keys.
    auto step = [&](int t, auto more, auto masked) {
        f32x16 y[2];
        u32x4 p[4];
        if constexpr (more)
            scores(t + 1, y);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const uint32_t w = pack_half_x2<F16>(exp2_fast(x[i >> 4][i & 15] * by - m),
                                                 exp2_fast(x[i >> 4][(i & 15) + 1] * by - m));
            p[i >> 3][(i & 7) >> 1] = w;
            l = dot_ones<F16>(w, l);
        }
        float top = 0.f;
        if constexpr (more) {
            if constexpr (masked)
                hide(t + 1, y);
            top = highest(y);
        }
        const uint8_t *const buf = lds + (t & 1) * kBuf;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
                const u32x2 lo = lds_read_tr(buf + v_rd[c] + 16 * ks * kRow);
                const u32x2 hi = lds_read_tr(buf + v_rd[c] + (16 * ks + 8) * kRow);
                o[c] = mfma32x32x16<F16>(u32x4{lo[0], lo[1], hi[0], hi[1]}, p[ks], o[c]);
            }
        if constexpr (more) {
            x[0] = y[0], x[1] = y[1];
            raise(top);
        }
    };

    if (tiles > t0) {
        pages_from(t0);
        fetch(true, t0, page_of(t0));
        fetch(false, t0, page_of(t0));
        if (((t0 + 1) & 63) == 0)
            pages_from(t0 + 1);
        int next_page = page_of(t0 + 1);
        fetch(true, t0 + 1, next_page);
        wait_vmcnt<2 * kDmas>(); // the wave's copies of the first keys
        lds_barrier();
        scores(t0, x);
        if (t0 >= whole)
            hide(t0, x);
        raise(highest(x));
        // Before tile t: its values and the next tile's keys are there for
        // everybody, and the buffers of the values before and of its own keys
        // are used up: every wave's reads of them have returned (their products
        // need not have run).
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
            }
            lds_barrier();
            if (t + 1 < tiles)
                fetch(false, t + 1, next_page);
            if (t + 2 < tiles) {
                if (((t + 2) & 63) == 0)
                    pages_from(t + 2);
                next_page = page_of(t + 2);
                fetch(true, t + 2, next_page);
            }
            if constexpr (check) {
                const uint32_t bad = s_bad[t & 1][0] | s_bad[t & 1][1] | s_bad[t & 1][2] | s_bad[t & 1][3];
                if (__builtin_amdgcn_readfirstlane((int)bad))
                    mend(t);
            }
        };
        int t = t0;
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

    const float sum = sum_swap32(l);
    if (row >= rows)
        return;
    if (a.splits > 1) {
        const int64_t at = row_out * a.splits + split;
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<f32x4 *>(a.part + at * D + 32 * c + 2 * i + 4 * half) =
                    f32x4{o[c][i], o[c][i + 1], o[c][i + 2], o[c][i + 3]};
        if (half == 0) {
            a.stats[2 * at] = m;
            a.stats[2 * at + 1] = sum;
        }
        return;
    }
    const float inv = sum == 0.f ? 1.f : 1.f / sum;
    uint16_t *const p = a.out + row_out * D + 4 * half;
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<u32x2 *>(p + 32 * c + 2 * i) = u32x2{pack_half_x2<F16>(o[c][i] * inv, o[c][i + 1] * inv),
                                                                   pack_half_x2<F16>(o[c][i + 2] * inv, o[c][i + 3] * inv)};
}

// Few rows and many keys: the ranges of a row's keys joined,
// o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i, a lane for 4 channels.
// Bound by the latency of reading a row's partial results.
template <int D, bool F16, bool PAGED> __global__ __launch_bounds__(256) void attn_prefill_join_kernel(PrefillArgs a)
{
    constexpr int kLanes = D / 4, kRows = 256 / kLanes;
    const int h = blockIdx.x % a.hkv, seq = blockIdx.x / a.hkv;
    const int q0 = clampi(a.cu_q[seq], 0, a.tokens);
    const int all_new = max(clampi(a.cu_q[seq + 1], 0, a.tokens) - q0, 0);
    const int64_t rows = (int64_t)min(all_new, a.longest) * a.G;
    int keys;
    if constexpr (PAGED) {
        keys = clampi(a.lens[seq], 0, a.cache.width << a.cache.page_shift);
    } else {
        const int k0 = clampi(a.cu_k[seq], 0, a.keys);
        keys = max(clampi(a.cu_k[seq + 1], 0, a.keys) - k0, 0);
    }
    const int shift = keys - all_new + 1, per = prefill_range(keys, a.splits);
    const int c = 4 * (threadIdx.x % kLanes);
    for (int64_t row = (int64_t)blockIdx.y * kRows + threadIdx.x / kLanes; row < rows; row += (int64_t)gridDim.y * kRows) {
        const int64_t last = min(rows, row / kPrefillRows * kPrefillRows + kPrefillRows) - 1; // of the row's block
        const int tiles = (clampi(shift + (int)(last / a.G), 0, keys) + kKeys - 1) / kKeys;
        const int n = max(1, (tiles + per - 1) / per);
        const int64_t at = (q0 + row / a.G) * a.hkv * a.G + h * a.G + row % a.G;
        const float *const st = a.stats + 2 * at * a.splits;
        const float *const part = a.part + at * a.splits * D + c;
        float top = st[0];
        for (int i = 1; i < n; ++i)
            top = fmaxf(top, st[2 * i]);
        f32x4 x = {};
        float sum = 0.f;
        for (int i = 0; i < n; ++i) {
            const float f = exp2_fast(st[2 * i] - top);
            sum += f * st[2 * i + 1];
            x += f * *reinterpret_cast<const f32x4 *>(part + (int64_t)i * D);
        }
        const float inv = sum == 0.f ? 1.f : 1.f / sum;
        *reinterpret_cast<u32x2 *>(a.out + at * D + c) = u32x2{pack_half_x2<F16>(x[0] * inv, x[1] * inv),
                                                               pack_half_x2<F16>(x[2] * inv, x[3] * inv)};
    }
}

template <int D, bool F16, bool PAGED> hipError_t run(const PrefillArgs &a, int64_t seqs, hipStream_t st)
{
    const dim3 grid((unsigned)(a.hkv * (a.all_blocks ? a.all_blocks : a.blocks * seqs)), (unsigned)a.splits);
    attn_prefill_kernel<D, F16, PAGED><<<grid, 64 * kWaves, 8 * kKeys * D, st>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || a.splits == 1)
        return e;
    const int64_t rows = (int64_t)a.longest * a.G, each = 1024 / D;
    attn_prefill_join_kernel<D, F16, PAGED>
        <<<dim3((unsigned)(a.hkv * seqs), (unsigned)std::min<int64_t>((rows + each - 1) / each, 32768)), 256, 0, st>>>(a);
    return hipGetLastError();
}

} // namespace

// Few row blocks: the keys of a sequence are cut into ranges, so that the
// device is filled (two workgroups a compute unit), and joined.  A workgroup
// takes some 5 us and 1.2 us a tile alone on a compute unit (2 beside another),
// the join 4 to 8 us, so it pays only where there are several ranges to a block
// and a range has some tiles: 1931 new tokens behind 6261, 8 heads on one, 121
// blocks: 148 us whole, 91 in two ranges, 78 in four; but 1000 tokens, 32/8
// heads, 256 blocks: 23 us whole, 34 in two, and 500 tokens, 128 blocks: 15 us
// whole, 19 in two.
int plan_prefill_splits(int64_t seqs, int64_t T, int64_t hkv, int64_t G, int64_t longest, int64_t keys, int cus)
{
    const int64_t blocks = hkv * std::min(seqs * prefill_blocks(longest, G), T * G / kPrefillRows + seqs);
    const int64_t ranges = (keys + kKeys * kMinRange - 1) / (kKeys * kMinRange);
    if (blocks > cus / 2 || ranges < 4)
        return 1;
    return (int)std::min<int64_t>({2 * (int64_t)cus / blocks, ranges, kMaxSplits});
}

hipError_t launch_attn_prefill(PrefillArgs a, int D, bool f16, bool paged, int64_t seqs, hipStream_t st)
{
    a.blocks = (int)prefill_blocks(a.longest, a.G);
    // An XCD runs the workgroups whose number is its own modulo 8: with 8 heads
    // those of one head.  Where the keys and values of all sequences and heads
    // that it meets fit its L2 (a sequence taken to have the mean number of
    // keys, or for pages what its table can name), all run side by side, the
    // blocks with the most keys first.  Else one sequence after the other, in
    // groups of as many heads as fit; so too where all workgroups run at once,
    // for the search costs 0.4 us.
    const int64_t keys = paged ? (int64_t)a.cache.width << a.cache.page_shift : (a.keys + seqs - 1) / seqs;
    const int64_t pair = std::max<int64_t>(1, keys * 4 * D);
    const int64_t most = std::min(seqs * a.blocks, (int64_t)a.tokens * a.G / kPrefillRows + seqs);
    const bool side = seqs > 1 && seqs <= 64 && a.hkv * seqs * a.blocks > kSlots && seqs * (a.hkv % 8 ? a.hkv : a.hkv / 8) * pair <= kL2Share;
    a.all_blocks = side ? (int)most : 0;
    a.steps = 1;
    while (64 * (int64_t)a.steps < a.blocks)
        a.steps *= 64;
    a.heads_by = (int)std::min<int64_t>(a.hkv, 8 * std::max<int64_t>(1, kL2Share / pair));
    while (a.hkv % a.heads_by)
        --a.heads_by;
    if (D == 64)
        return paged ? f16 ? run<64, true, true>(a, seqs, st) : run<64, false, true>(a, seqs, st)
               : f16 ? run<64, true, false>(a, seqs, st)
                     : run<64, false, false>(a, seqs, st);
    return paged ? f16 ? run<128, true, true>(a, seqs, st) : run<128, false, true>(a, seqs, st)
           : f16 ? run<128, true, false>(a, seqs, st)
                 : run<128, false, false>(a, seqs, st);
}

} // namespace tf
