// C ABI of the attention and cache calls: argument validation on the host
// (before any HIP call), then the launches on the caller's stream.  The
// declarations and their documentation live in include/tilefuse_attention.h.
#include "tilefuse_attention.h"

#include <cmath>

#include "tf_attn.h"

namespace {

constexpr int64_t kIntLimit = int64_t(1) << 31;
constexpr int64_t kKeyLimit = int64_t(1) << 30; // key numbers, and a few tiles past the last, are 32-bit
constexpr int64_t kStrideLimit = int64_t(1) << 26; // 16 rows of a strided tensor within 31-bit byte offsets
constexpr int64_t kGridYZ = 65535; // sequences of a decode call, a grid axis
constexpr int kMaxGroup = 1024;
constexpr int64_t kMaxWorkgroups = ((int64_t(1) << 32) - 1) / 256; // a launch has fewer than 2^32 threads, these kernels' workgroups 256

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// log2 of the page size, or -1: a power of two from 16 to 1024
int page_shift(int64_t page)
{
    for (int s = 4; s <= 10; ++s)
        if (page == int64_t(1) << s)
            return s;
    return -1;
}

bool count_ok(int64_t n, int64_t low) { return n >= low && n < kIntLimit; }

// Heads and channels of an attention call.
int check_heads(int type, int64_t Hq, int64_t Hkv, int64_t D)
{
    if (type != TF_TYPE_BF16 && type != TF_TYPE_F16)
        return TF_ERR_UNSUPPORTED;
    if (Hq < 1 || Hkv < 1 || Hq >= 65536 || Hq % Hkv || D < 1)
        return TF_ERR_SHAPE;
    if ((D != 64 && D != 128) || Hq / Hkv > kMaxGroup)
        return TF_ERR_UNSUPPORTED;
    return TF_OK;
}

int check_paged(const uint16_t *k, const uint16_t *v, int64_t pages, int64_t page, const int32_t *tables, int64_t width)
{
    if (!count_ok(pages, 1) || !count_ok(width, 1))
        return TF_ERR_SHAPE;
    const int shift = page_shift(page);
    if (shift < 0)
        return TF_ERR_UNSUPPORTED;
    if (width > kKeyLimit >> shift)
        return TF_ERR_SHAPE;
    if (!k || !v || !tables)
        return TF_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(tables, 4))
        return TF_ERR_ALIGN;
    return TF_OK;
}

// A [rows][heads][D] tensor read in 16-byte units: strides in elements.
int check_strided(const void *p, int64_t token, int64_t head, int64_t heads, int64_t D)
{
    if (token < D || (heads > 1 && head < D) || token >= kStrideLimit || head >= kStrideLimit || head < 0)
        return TF_ERR_SHAPE;
    if (!p)
        return TF_ERR_NULL;
    return aligned(p, 16) && token % 8 == 0 && (heads == 1 || head % 8 == 0) ? TF_OK : TF_ERR_ALIGN;
}

constexpr float kLog2E = 1.4426950408889634f;

// the kernels multiply with scale log2(e)
bool scale_ok(float s) { return std::isfinite(s * kLog2E) && s > 0.f; }

// Rows of a decode call's partial results, and its workspace: the rows, their
// maxima and sums, three numbers per share.
int64_t decode_part_rows(const tf::DecodePlan &p) { return p.shares * 2 * 16 * p.nt; }
size_t decode_ws(int64_t D, const tf::DecodePlan &p)
{
    return (size_t)(decode_part_rows(p) * (D + 2) + 3 * p.shares) * sizeof(float);
}

int check_decode_sizes(int type, int64_t seqs, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest)
{
    if (int st = check_heads(type, Hq, Hkv, D))
        return st;
    return seqs >= 0 && seqs <= kGridYZ && seqs * Hq < kIntLimit && longest >= 0 && longest <= kKeyLimit ? TF_OK : TF_ERR_SHAPE;
}

int check_ws(const void *ws, size_t have, size_t need)
{
    if (!need)
        return TF_OK;
    if (!ws)
        return TF_ERR_NULL;
    if (!aligned(ws, 256))
        return TF_ERR_ALIGN;
    return have < need ? TF_ERR_BUFFER_TOO_SMALL : TF_OK;
}

// Floats of the partial results of a prefill call of valid sizes.
int64_t prefill_part_floats(int64_t T, int64_t Hq, int64_t D, int splits) { return splits > 1 ? T * Hq * splits * (D + 2) : 0; }

int prefill(int type, tf::PrefillArgs &a, int64_t Hq, int64_t D, bool paged, int64_t seqs, int64_t keys, void *ws,
            size_t ws_bytes, void *stream)
{
    a.seqs = (int)seqs;
    a.splits = tf::plan_prefill_splits(seqs, a.tokens, a.hkv, a.G, a.longest, keys, tf::device_cus());
    const int64_t floats = prefill_part_floats(a.tokens, Hq, D, a.splits);
    if (int st = check_ws(ws, ws_bytes, (size_t)floats * sizeof(float)))
        return st;
    a.part = static_cast<float *>(ws);
    a.stats = floats ? a.part + (int64_t)a.tokens * Hq * a.splits * D : nullptr;
    return tf::launch_attn_prefill(a, (int)D, type == TF_TYPE_F16, paged, seqs, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? TF_OK
               : TF_ERR_HIP;
}

// Sizes of a prefill call.
int check_prefill_sizes(int type, int64_t seqs, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest, int64_t keys)
{
    if (int st = check_heads(type, Hq, Hkv, D))
        return st;
    if (!count_ok(seqs, 0) || T < 0 || T > kKeyLimit || longest < 0 || longest > T || keys < 0 || keys > kKeyLimit)
        return TF_ERR_SHAPE;
    // workgroups along the grid's first axis, at most (ranges of keys are its second)
    const int64_t blocks = std::max<int64_t>(1, tf::prefill_blocks(longest, Hq / Hkv)) * Hkv; // of a sequence: < 2^50
    return seqs && blocks > kMaxWorkgroups / seqs ? TF_ERR_SHAPE : TF_OK;
}

// What both prefill calls ask of their queries.
int check_queries(const uint16_t *q, int64_t q_token, int64_t q_head, const int32_t *cu_q, const uint16_t *out, int64_t Hq,
                  int64_t D)
{
    if (!cu_q || !out)
        return TF_ERR_NULL;
    if (!aligned(cu_q, 4) || !aligned(out, 16))
        return TF_ERR_ALIGN;
    return check_strided(q, q_token, q_head, Hq, D);
}

int check_pool(uint16_t *cache, int64_t planes, int64_t pages, int64_t Hkv, int64_t page, int64_t D, const int32_t *refs,
               const int32_t *tables, int64_t seqs, int64_t width, const int32_t *refs_out, const int32_t *tables_out,
               const int32_t *told)
{
    if (planes < 0 || planes > 65536 || !count_ok(pages, 1) || Hkv < 1 || Hkv >= 65536 || page < 1 || page > 1024 || D < 1 ||
        D > 65536 || seqs < 0 || seqs >= kIntLimit || !count_ok(width, 1) || width >= kIntLimit / page ||
        (Hkv * page * D) >= kIntLimit)
        return TF_ERR_SHAPE;
    if (D % 8)
        return TF_ERR_UNSUPPORTED;
    if ((planes && !cache) || !refs || !refs_out || !told || (seqs && (!tables || !tables_out)))
        return TF_ERR_NULL;
    if (!aligned(cache, 16) || !aligned(refs, 4) || !aligned(tables, 4) || !aligned(refs_out, 4) || !aligned(tables_out, 4) ||
        !aligned(told, 4))
        return TF_ERR_ALIGN;
    return TF_OK;
}

size_t fork_ws(int64_t forks) { return forks > 0 ? (size_t)forks * 4 * sizeof(int32_t) : 0; }
size_t compact_ws(int64_t pages) { return (size_t)(1 + 3 * (pages / 2)) * sizeof(int32_t); }

} // namespace

extern "C" {

int tf_kv_append(int type, const uint16_t *qkv, int64_t qkv_token, const float *rope, int64_t rope_rows,
                 const int32_t *seq, const int32_t *pos, int64_t T, const int32_t *tables, int64_t seqs, int64_t width,
                 uint16_t *q, uint16_t *k_pages, uint16_t *v_pages, int64_t pages, int64_t page, int64_t Hq,
                 int64_t Hkv, int64_t D, void *stream)
{
    if (type != TF_TYPE_BF16 && type != TF_TYPE_F16)
        return TF_ERR_UNSUPPORTED;
    if (T < 0 || T > 4 * kMaxWorkgroups || Hq < 1 || Hkv < 1 || Hq >= 65536 || Hkv >= 65536 || D < 1 || !count_ok(seqs, 0) ||
        !count_ok(rope_rows, 0) || qkv_token < (Hq + 2 * Hkv) * D) // a workgroup has a wave for each of 4 tokens
        return TF_ERR_SHAPE;
    if (D % 16 || D > 1024)
        return TF_ERR_UNSUPPORTED;
    if (T == 0)
        return TF_OK;
    if (!qkv || !rope || !seq || !pos || !q)
        return TF_ERR_NULL;
    if (!aligned(qkv, 16) || qkv_token % 8 || !aligned(rope, 16) || !aligned(seq, 4) || !aligned(pos, 4) || !aligned(q, 16))
        return TF_ERR_ALIGN;
    if (int st = check_paged(k_pages, v_pages, pages, page, tables, width))
        return st;
    tf::AppendArgs a;
    a.qkv = qkv;
    a.qkv_token = qkv_token;
    a.rope = rope;
    a.rope_rows = (int)rope_rows;
    a.seq = seq;
    a.pos = pos;
    a.tables = tables;
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    a.tokens = (int)T;
    a.seqs = (int)seqs;
    a.width = (int)width;
    a.pages = (int)pages;
    a.hq = (int)Hq;
    a.hkv = (int)Hkv;
    a.D = (int)D;
    a.page_shift = page_shift(page);
    return tf::launch_kv_append(a, type == TF_TYPE_F16, static_cast<hipStream_t>(stream)) == hipSuccess ? TF_OK : TF_ERR_HIP;
}

size_t tf_attn_decode_workspace_bytes(int64_t seqs, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest)
{
    if (check_decode_sizes(TF_TYPE_BF16, seqs, Hq, Hkv, D, longest) != TF_OK || seqs == 0)
        return 0;
    const tf::DecodePlan p = tf::plan_decode(seqs, Hkv, Hq / Hkv, longest, tf::device_cus());
    return decode_ws(D, p);
}

int tf_attn_decode(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k_pages,
                   const uint16_t *v_pages, int64_t pages, int64_t page, const int32_t *tables, int64_t width,
                   const int32_t *lens, uint16_t *out, int64_t seqs, int64_t Hq, int64_t Hkv, int64_t D,
                   int64_t longest, float scale, void *workspace, size_t ws_bytes, void *stream)
{
    if (int st = check_decode_sizes(type, seqs, Hq, Hkv, D, longest))
        return st;
    if (!scale_ok(scale))
        return TF_ERR_UNSUPPORTED;
    if (seqs == 0)
        return TF_OK;
    if (!lens || !out)
        return TF_ERR_NULL;
    if (!aligned(lens, 4) || !aligned(out, 16))
        return TF_ERR_ALIGN;
    if (int st = check_strided(q, q_token, q_head, Hq, D))
        return st;
    if (int st = check_paged(k_pages, v_pages, pages, page, tables, width))
        return st;
    const tf::DecodePlan p = tf::plan_decode(seqs, Hkv, Hq / Hkv, longest, tf::device_cus());
    if (int st = check_ws(workspace, ws_bytes, decode_ws(D, p)))
        return st;
    tf::DecodeArgs a = {};
    a.q = q;
    a.q_token = q_token;
    a.q_head = q_head;
    a.cache = {k_pages, v_pages, tables, (int)pages, (int)Hkv, page_shift(page), (int)width};
    a.lens = lens;
    a.out = out;
    a.part = static_cast<float *>(workspace);
    if (p.shares) {
        a.stats = a.part + decode_part_rows(p) * D;
        a.spans = reinterpret_cast<int32_t *>(a.stats + 2 * decode_part_rows(p));
    }
    a.seqs = (int)seqs;
    a.G = (int)(Hq / Hkv);
    a.groups = (int)p.groups;
    a.unit_shift = (int)p.unit_shift;
    a.longest = (int)std::min<int64_t>(longest, width * page);
    a.scale_log2 = scale * kLog2E;
    return tf::launch_attn_decode(a, (int)D, type == TF_TYPE_F16, p, static_cast<hipStream_t>(stream)) == hipSuccess
               ? TF_OK
               : TF_ERR_HIP;
}

size_t tf_attn_prefill_workspace_bytes(int64_t seqs, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t longest,
                                       int64_t keys)
{
    if (check_prefill_sizes(TF_TYPE_BF16, seqs, T, Hq, Hkv, D, longest, keys) != TF_OK || seqs == 0 || T == 0 || longest == 0)
        return 0;
    const int splits = tf::plan_prefill_splits(seqs, T, Hkv, Hq / Hkv, longest, keys, tf::device_cus());
    return (size_t)prefill_part_floats(T, Hq, D, splits) * sizeof(float);
}

int tf_attn_prefill(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k, int64_t k_token,
                    int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head, const int32_t *cu_q,
                    const int32_t *cu_k, uint16_t *out, int64_t seqs, int64_t T, int64_t keys, int64_t Hq, int64_t Hkv,
                    int64_t D, int64_t longest, float scale, void *workspace, size_t ws_bytes, void *stream)
{
    if (int st = check_prefill_sizes(type, seqs, T, Hq, Hkv, D, longest, keys))
        return st;
    if (!scale_ok(scale))
        return TF_ERR_UNSUPPORTED;
    if (seqs == 0 || T == 0 || longest == 0)
        return TF_OK;
    if (int st = check_queries(q, q_token, q_head, cu_q, out, Hq, D))
        return st;
    if (!cu_k)
        return TF_ERR_NULL;
    if (!aligned(cu_k, 4))
        return TF_ERR_ALIGN;
    if (keys) { // without keys nothing of k and v is read
        if (int st = check_strided(k, k_token, k_head, Hkv, D))
            return st;
        if (int st = check_strided(v, v_token, v_head, Hkv, D))
            return st;
    }
    tf::PrefillArgs a = {};
    a.q = q;
    a.q_token = q_token;
    a.q_head = q_head;
    a.k = k;
    a.v = v;
    a.k_token = k_token;
    a.k_head = k_head;
    a.v_token = v_token;
    a.v_head = v_head;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.out = out;
    a.tokens = (int)T;
    a.keys = (int)keys;
    a.hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.longest = (int)longest;
    a.scale_log2 = scale * kLog2E;
    return prefill(type, a, Hq, D, false, seqs, keys, workspace, ws_bytes, stream);
}

int tf_attn_prefill_paged(int type, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k_pages,
                          const uint16_t *v_pages, int64_t pages, int64_t page, const int32_t *tables, int64_t width,
                          const int32_t *cu_q, const int32_t *lens, uint16_t *out, int64_t seqs, int64_t T, int64_t Hq,
                          int64_t Hkv, int64_t D, int64_t longest, float scale, void *workspace, size_t ws_bytes,
                          void *stream)
{
    if (int st = check_prefill_sizes(type, seqs, T, Hq, Hkv, D, longest, 0))
        return st;
    if (!scale_ok(scale))
        return TF_ERR_UNSUPPORTED;
    if (seqs == 0 || T == 0 || longest == 0)
        return TF_OK;
    if (int st = check_queries(q, q_token, q_head, cu_q, out, Hq, D))
        return st;
    if (!lens)
        return TF_ERR_NULL;
    if (!aligned(lens, 4))
        return TF_ERR_ALIGN;
    if (int st = check_paged(k_pages, v_pages, pages, page, tables, width))
        return st;
    tf::PrefillArgs a = {};
    a.q = q;
    a.q_token = q_token;
    a.q_head = q_head;
    a.cache = {k_pages, v_pages, tables, (int)pages, (int)Hkv, page_shift(page), (int)width};
    a.cu_q = cu_q;
    a.lens = lens;
    a.out = out;
    a.tokens = (int)T;
    a.hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.longest = (int)longest;
    a.scale_log2 = scale * kLog2E;
    return prefill(type, a, Hq, D, true, seqs, width * page, workspace, ws_bytes, stream);
}

size_t tf_kv_fork_workspace_bytes(int64_t forks) { return count_ok(forks, 0) ? fork_ws(forks) : 0; }
size_t tf_kv_compact_workspace_bytes(int64_t pages) { return count_ok(pages, 1) ? compact_ws(pages) : 0; }

int tf_kv_fork(uint16_t *cache, int64_t planes, int64_t pages, int64_t Hkv, int64_t page, int64_t D,
               const int32_t *refs, const int32_t *tables, const int32_t *lens, int64_t seqs, int64_t width,
               const int32_t *parents, const int32_t *children, int64_t forks, int32_t *refs_out, int32_t *tables_out,
               int32_t *lens_out, int32_t *status, void *workspace, size_t ws_bytes, void *stream)
{
    // the second launch's workgroups, counted before the first one writes
    if (!count_ok(forks, 0) || planes < 0 || planes > 65536 || seqs < 0 || seqs > kMaxWorkgroups ||
        (planes + 1) * forks > kMaxWorkgroups - seqs)
        return TF_ERR_SHAPE;
    if (int st = check_pool(cache, planes, pages, Hkv, page, D, refs, tables, seqs, width, refs_out, tables_out, status))
        return st;
    if ((seqs && (!lens || !lens_out)) || (forks && (!parents || !children)))
        return TF_ERR_NULL;
    if (!aligned(lens, 4) || !aligned(lens_out, 4) || !aligned(parents, 4) || !aligned(children, 4))
        return TF_ERR_ALIGN;
    if (int st = check_ws(workspace, ws_bytes, fork_ws(forks)))
        return st;
    tf::PoolArgs a = {cache, refs, tables, lens, parents, children, refs_out, tables_out, lens_out, status,
                      static_cast<int32_t *>(workspace), planes, (int)pages, (int)Hkv, (int)page, (int)D, (int)seqs,
                      (int)width, (int)forks};
    return tf::launch_kv_fork(a, static_cast<hipStream_t>(stream)) == hipSuccess ? TF_OK : TF_ERR_HIP;
}

int tf_kv_compact(uint16_t *cache, int64_t planes, int64_t pages, int64_t Hkv, int64_t page, int64_t D,
                  const int32_t *refs, const int32_t *tables, int64_t seqs, int64_t width, int32_t *refs_out,
                  int32_t *tables_out, int32_t *moved, void *workspace, size_t ws_bytes, void *stream)
{
    if (int st = check_pool(cache, planes, pages, Hkv, page, D, refs, tables, seqs, width, refs_out, tables_out, moved))
        return st;
    if (int st = check_ws(workspace, ws_bytes, compact_ws(pages)))
        return st;
    tf::PoolArgs a = {cache, refs, tables, nullptr, nullptr, nullptr, refs_out, tables_out, nullptr, moved,
                      static_cast<int32_t *>(workspace), planes, (int)pages, (int)Hkv, (int)page, (int)D, (int)seqs,
                      (int)width, 0};
    return tf::launch_kv_compact(a, static_cast<hipStream_t>(stream)) == hipSuccess ? TF_OK : TF_ERR_HIP;
}

} // extern "C"
