// The paged key-value cache: rotating and writing new tokens, and giving
// pages to forks or moving them together.  All of it moves bytes: the floor
// of each kernel is what it has to read and write once.
#include "tf_attn.h"

namespace tf {

namespace {

// ---------------------------------------------------------------------------
// append: channels i and i + D/2 of a query or key head are a pair, turned by
// the position's angle: (a, b) -> (a cos - b sin, b cos + a sin), in fp32,
// rounded once.  Values are copied.  A lane holds 8 channels of the first
// half and their 8 partners, so a wave covers 64 / (D / 16) heads per pass
// with the position's cosines and sines kept in registers over its passes.
// HBM-bound for many tokens: 10639 of 32/8 heads of 128 channels take 46 us
// (5.8 TB/s, read and written; a plain copy runs at 4.7), with the input
// streamed, and 55 without; streaming the outputs too gives 49, and the
// attention reads them next.  For few tokens it is a chain of dependent loads
// (position, table, row), so each pass then gets a wave of its own: 16 tokens
// 3.2 us on the device.

template <bool F16> __device__ __forceinline__ float half_lo(uint32_t w) { return half_bits_to_f32<F16>(w & 0xFFFFu); }
template <bool F16> __device__ __forceinline__ float half_hi(uint32_t w)
{
    if constexpr (F16)
        return half_bits_to_f32<true>(w >> 16);
    else
        return __uint_as_float(w & 0xFFFF0000u);
}

template <bool F16> __global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int passes_each)
{
    const int lane = threadIdx.x & 63;
    const int64_t token = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (token >= a.tokens)
        return;
    const int half = a.D / 2, units = half / 8; // units of 8 channels per half head
    const int per = 64 / units;                 // heads per pass
    const int unit = lane % units, sub = lane / units;
    const int heads = a.hq + 2 * a.hkv;
    const int pos = a.pos[token], seq = a.seq[token];
    const bool turns = pos >= 0 && pos < a.rope_rows;
    // the row of the cache, if the sequence, position and page all exist
    int page = -1;
    if (seq >= 0 && seq < a.seqs && pos >= 0 && (pos >> a.page_shift) < a.width)
        page = a.tables[(int64_t)seq * a.width + (pos >> a.page_shift)];
    const bool stored = page >= 0 && page < a.pages;
    float cs[8] = {}, sn[8] = {};
    if (turns) {
        const f32x4 *const r = reinterpret_cast<const f32x4 *>(a.rope + (int64_t)pos * a.D + 8 * unit);
        const f32x4 c0 = r[0], c1 = r[1];
        const f32x4 *const t = reinterpret_cast<const f32x4 *>(a.rope + (int64_t)pos * a.D + half + 8 * unit);
        const f32x4 s0 = t[0], s1 = t[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = c0[i];
            cs[4 + i] = c1[i];
            sn[i] = s0[i];
            sn[4 + i] = s1[i];
        }
    }
    const int64_t row = ((int64_t)(stored ? page : 0) * a.hkv << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    const uint16_t *const in = a.qkv + token * a.qkv_token + 8 * unit;
    const int first = blockIdx.y * passes_each * per, end = min(heads, first + passes_each * per);
#pragma unroll 2
    for (int head = first + sub; head < end; head += per) {
        if (sub >= per)
            break; // lanes past a whole number of heads (D / 16 no power of two)
        u32x4 lo = load16_stream(in + (int64_t)head * a.D), hi = load16_stream(in + (int64_t)head * a.D + half);
        if (head < a.hq + a.hkv) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // without a rotation the head is zero, whatever it held
                const uint32_t xs = turns ? lo[i] : 0u, ys = turns ? hi[i] : 0u;
                const float x0 = half_lo<F16>(xs), x1 = half_hi<F16>(xs);
                const float y0 = half_lo<F16>(ys), y1 = half_hi<F16>(ys);
                const float c0 = cs[2 * i], c1 = cs[2 * i + 1], s0 = sn[2 * i], s1 = sn[2 * i + 1];
                lo[i] = pack_half_x2<F16>(x0 * c0 - y0 * s0, x1 * c1 - y1 * s1);
                hi[i] = pack_half_x2<F16>(y0 * c0 + x0 * s0, y1 * c1 + x1 * s1);
            }
        }
        uint16_t *out;
        if (head < a.hq) {
            out = a.q + (token * a.hq + head) * a.D;
        } else {
            if (!stored)
                continue;
            const bool is_k = head < a.hq + a.hkv;
            const int64_t kv = head - a.hq - (is_k ? 0 : a.hkv);
            out = (is_k ? a.k : a.v) + (row + (kv << a.page_shift)) * a.D;
        }
        *reinterpret_cast<u32x4 *>(out + 8 * unit) = lo;
        *reinterpret_cast<u32x4 *>(out + 8 * unit + half) = hi;
    }
}

// ---------------------------------------------------------------------------
// pool bookkeeping

constexpr int kScan = 1024; // threads of the scanning workgroup
constexpr int kCells = 8;   // pages per thread and step

// exclusive prefix sum of x over the workgroup's threads; *total gets the sum
__device__ __forceinline__ int scan_exclusive(int x, int *total, int *shared)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int in = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(in, d);
        if (lane >= d)
            in += y;
    }
    __syncthreads(); // shared is free again
    if (lane == 63)
        shared[wave] = in;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kScan / 64; ++w) {
        const int s = shared[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + in - x;
}

// The fork's plan, laid out in the workspace: for each child the page its
// partial page comes from (-1: none) and goes to, and its length.
struct ForkPlan {
    int32_t *from, *to, *size;
};
__device__ __forceinline__ ForkPlan fork_plan(const PoolArgs &a) { return {a.plan, a.plan + a.forks, a.plan + 2 * a.forks}; }

__device__ __forceinline__ int parent_length(const PoolArgs &a, int p)
{
    return clampi(a.lens[p], 0, a.width * a.page);
}

// One workgroup: ranks the children that need a page (prefix sum), finds the
// free pages of those ranks in ascending order (prefix sum over refs <= 0),
// copies refs.  Latency-bound; 8192 pages per step.
__global__ __launch_bounds__(kScan) void kv_fork_plan_kernel(PoolArgs a)
{
    __shared__ int shared[kScan / 64];
    __shared__ int s_page_of[kScan];
    const ForkPlan plan = fork_plan(a);
    const int tid = threadIdx.x;
    int need = 0;
    int r[kCells]; // the first step's references, on their way while the ranks are found
    auto read_refs = [&](int p0) {
#pragma unroll
        for (int j = 0; j < kCells; ++j) {
            const int p = p0 + kCells * tid + j;
            r[j] = p < a.pages ? a.refs[p] : 1;
        }
    };
    read_refs(0);
    for (int i0 = 0; i0 < a.forks; i0 += kScan) {
        const int i = i0 + tid;
        int size = -1, from = -1;
        if (i < a.forks) {
            const int p = a.parents[i], c = a.children[i];
            if (p >= 0 && p < a.seqs && c >= 0 && c < a.seqs) {
                size = parent_length(a, p);
                if (size % a.page)
                    from = a.tables[(int64_t)p * a.width + size / a.page];
            }
        }
        const bool wants = size > 0 && size % a.page;
        int all;
        const int rank = need + scan_exclusive(wants, &all, shared);
        need += all;
        if (i < a.forks) {
            plan.size[i] = size;
            plan.from[i] = wants ? from : -1;
            plan.to[i] = wants ? -2 - rank : -1; // a rank until its page is found
        }
    }
    // ranks are found again below by the page's own rank: page_of[rank], in
    // LDS where they fit
    int32_t *const page_of = need <= kScan ? s_page_of : a.plan + 3 * a.forks;
    int have = 0;
    for (int p0 = 0; p0 < a.pages; p0 += kScan * kCells) {
        if (p0)
            read_refs(p0);
        int count = 0;
#pragma unroll
        for (int j = 0; j < kCells; ++j)
            count += r[j] <= 0;
        int all, rank = scan_exclusive(count, &all, shared) + have;
        have += all;
#pragma unroll
        for (int j = 0; j < kCells; ++j) {
            const int p = p0 + kCells * tid + j;
            if (p >= a.pages)
                break;
            const bool free = r[j] <= 0;
            if (a.refs_out != a.refs)
                a.refs_out[p] = r[j];
            if (free && rank < need)
                page_of[rank] = p;
            rank += free;
        }
    }
    __syncthreads();
    const int missing = max(0, need - have);
    if (tid == 0)
        a.told[0] = missing;
    for (int i = tid; i < a.forks; i += kScan) {
        const int to = plan.to[i];
        if (missing)
            plan.size[i] = -1; // nothing is forked
        else if (to <= -2) {
            const int page = page_of[-2 - to];
            plan.to[i] = page;
            a.refs_out[page] = 1;
        }
    }
}

// Table rows and lengths (workgroups past the copies), references of shared
// pages (whole numbers added atomically: any order gives the same), and the
// partial pages: workgroup (child, plane) copies the used rows of each head.
__global__ __launch_bounds__(256) void kv_fork_kernel(PoolArgs a, int copies)
{
    const ForkPlan plan = fork_plan(a);
    const int tid = threadIdx.x;
    int b = blockIdx.x;
    if (b < copies) {
        const int i = b % a.forks;
        const int64_t plane = b / a.forks;
        const int size = plan.size[i], from = plan.from[i], to = plan.to[i];
        if (size <= 0 || to < 0)
            return;
        const bool there = from >= 0 && from < a.pages; // a page that does not exist reads as zeros
        const int64_t page_elems = (int64_t)a.page * a.D;
        const int units = (size % a.page) * a.D / 8; // 16-byte units of a head
        const uint16_t *src = a.cache + (plane * a.pages + (there ? from : to)) * a.hkv * page_elems;
        uint16_t *dst = a.cache + (plane * a.pages + to) * a.hkv * page_elems;
        auto at = [&](int u) { return (u / units) * page_elems + 8 * (u % units); };
        int u = tid;
        for (; u + 3 * 256 < units * a.hkv; u += 4 * 256) { // four loads in flight
            u32x4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = there ? load16(src + at(u + 256 * i)) : u32x4{};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<u32x4 *>(dst + at(u + 256 * i)) = x[i];
        }
        for (; u < units * a.hkv; u += 256)
            *reinterpret_cast<u32x4 *>(dst + at(u)) = there ? load16(src + at(u)) : u32x4{};
        return;
    }
    b -= copies;
    if (b < a.forks) { // a child's row and its shared pages
        const int size = plan.size[b];
        if (size < 0)
            return;
        const int p = a.parents[b], c = a.children[b], full = size / a.page;
        for (int col = tid; col < a.width; col += 256) {
            int page = -1;
            if (col < full) {
                page = a.tables[(int64_t)p * a.width + col];
                if (page >= 0 && page < a.pages)
                    atomicAdd(a.refs_out + page, 1);
            } else if (col == full && size % a.page) {
                page = plan.to[b];
            }
            a.tables_out[(int64_t)c * a.width + col] = page;
        }
        if (tid == 0)
            a.lens_out[c] = size;
        return;
    }
    // the other sequences keep their rows
    const int s = b - a.forks;
    int child = 0;
    for (int i = tid; i < a.forks; i += 256)
        child |= a.children[i] == s && plan.size[i] >= 0;
    if (__syncthreads_or(child))
        return;
    if (a.tables_out != a.tables)
        for (int col = tid; col < a.width; col += 256)
            a.tables_out[(int64_t)s * a.width + col] = a.tables[(int64_t)s * a.width + col];
    if (tid == 0)
        a.lens_out[s] = a.lens[s];
}

// Compacting: with L pages live, the k-th live page at or past L moves into
// the k-th dead page before L (there are as many of one as of the other, at
// most half the pool).  One workgroup counts, ranks both kinds, lists the
// pairs, and writes refs_out and the map; every cell of refs is read by the
// thread that writes it, so refs_out may be refs.
struct CompactPlan {
    int32_t *count, *from, *to, *refs;
};
__device__ __forceinline__ CompactPlan compact_plan(const PoolArgs &a)
{
    const int most = a.pages / 2;
    return {a.plan, a.plan + 1, a.plan + 1 + most, a.plan + 1 + 2 * most};
}

__global__ __launch_bounds__(kScan) void kv_compact_plan_kernel(PoolArgs a)
{
    __shared__ int shared[kScan / 64];
    const CompactPlan plan = compact_plan(a);
    const int tid = threadIdx.x;
    int live = 0;
    for (int p0 = 0; p0 < a.pages; p0 += kScan * kCells) {
        int n = 0, all;
#pragma unroll
        for (int j = 0; j < kCells; ++j) {
            const int p = p0 + kCells * tid + j;
            n += p < a.pages && a.refs[p] > 0;
        }
        scan_exclusive(n, &all, shared);
        live += all;
    }
    int movers = 0, holes = 0;
    for (int p0 = 0; p0 < a.pages; p0 += kScan * kCells) {
        int r[kCells], nm = 0, nh = 0, am, ah;
#pragma unroll
        for (int j = 0; j < kCells; ++j) {
            const int p = p0 + kCells * tid + j;
            r[j] = p < a.pages ? a.refs[p] : 0;
            nm += r[j] > 0 && p >= live;
            nh += r[j] <= 0 && p < live;
        }
        int m = movers + scan_exclusive(nm, &am, shared), h = holes + scan_exclusive(nh, &ah, shared);
        movers += am;
        holes += ah;
#pragma unroll
        for (int j = 0; j < kCells; ++j) {
            const int p = p0 + kCells * tid + j;
            if (p >= a.pages)
                break;
            const bool alive = r[j] > 0, front = p < live;
            if (alive && !front) {
                plan.refs[m] = r[j];
                plan.from[m++] = p;
            }
            if (!alive && front)
                plan.to[h++] = p;
            a.told[p] = alive && front ? p : -1; // movers below
            a.refs_out[p] = alive && front ? r[j] : 0;
        }
    }
    if (tid == 0)
        plan.count[0] = movers;
    __syncthreads();
    for (int k = tid; k < movers; k += kScan) {
        a.told[plan.from[k]] = plan.to[k];
        a.refs_out[plan.to[k]] = plan.refs[k];
    }
}

// The pages themselves, in steps of 16 KiB spread over the workgroups, and
// the tables.  A copy: 1.17 GB of page moves take 207 us (5.6 TB/s, read and
// written), streamed past the caches over many short workgroups; with the
// default policy and 2048 workgroups of 32 KiB steps 236.
__global__ __launch_bounds__(256) void kv_compact_kernel(PoolArgs a, int blocks, int chunks)
{
    const CompactPlan plan = compact_plan(a);
    const int movers = plan.count[0];
    const int tid = threadIdx.x;
    const int64_t page_units = (int64_t)a.hkv * a.page * a.D / 8;
    const int64_t per = (page_units + chunks - 1) / chunks;
    const int64_t work = (int64_t)movers * a.planes * chunks;
    for (int64_t w = blockIdx.x; w < work; w += blocks) {
        const int c = (int)(w % chunks);
        const int64_t rest = w / chunks;
        const int k = (int)(rest % movers);
        const int64_t plane = rest / movers;
        const u32x4 *const src = reinterpret_cast<const u32x4 *>(a.cache) + (plane * a.pages + plan.from[k]) * page_units;
        u32x4 *const dst = reinterpret_cast<u32x4 *>(a.cache) + (plane * a.pages + plan.to[k]) * page_units;
        const int64_t end = min(page_units, (c + 1) * per);
        int64_t u = c * per + tid;
        for (; u + 3 * 256 < end; u += 4 * 256) {
            u32x4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = __builtin_nontemporal_load(src + u + 256 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_nontemporal_store(x[i], dst + u + 256 * i);
        }
        for (; u < end; u += 256)
            dst[u] = src[u];
    }
    const int64_t all = (int64_t)blocks * 256, me = (int64_t)blockIdx.x * 256 + tid;
    const int64_t cells = (int64_t)a.seqs * a.width;
    for (int64_t i = me; i < cells; i += all) {
        const int p = a.tables[i];
        a.tables_out[i] = p >= 0 && p < a.pages ? a.told[p] : -1;
    }
}

} // namespace

hipError_t launch_kv_append(const AppendArgs &a, bool f16, hipStream_t st)
{
    const int units = a.D / 16, per = 64 / units;
    const int passes = (a.hq + 2 * a.hkv + per - 1) / per;
    const int64_t blocks = ((int64_t)a.tokens + 3) / 4;
    // few tokens: one pass per wave
    const int each = blocks * passes <= 2048 ? 1 : passes;
    const dim3 grid((unsigned)blocks, (unsigned)((passes + each - 1) / each));
    if (f16)
        kv_append_kernel<true><<<grid, 256, 0, st>>>(a, each);
    else
        kv_append_kernel<false><<<grid, 256, 0, st>>>(a, each);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const PoolArgs &a, hipStream_t st)
{
    kv_fork_plan_kernel<<<1, kScan, 0, st>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    const int copies = (int)(a.planes * a.forks);
    if (copies + a.forks + a.seqs == 0)
        return hipSuccess;
    kv_fork_kernel<<<copies + a.forks + a.seqs, 256, 0, st>>>(a, copies);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const PoolArgs &a, hipStream_t st)
{
    kv_compact_plan_kernel<<<1, kScan, 0, st>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    // 16 KiB of a page-plane per step of a workgroup; at most half the pages move
    const int64_t bytes = (int64_t)a.hkv * a.page * a.D * 2;
    const int chunks = (int)std::max<int64_t>(1, (bytes + 16383) / 16384);
    const int64_t most = std::max<int64_t>(a.planes * chunks * (a.pages / 2), ((int64_t)a.seqs * a.width + 255) / 256);
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(16384, most));
    kv_compact_kernel<<<blocks, 256, 0, st>>>(a, blocks, chunks);
    return hipGetLastError();
}

} // namespace tf
