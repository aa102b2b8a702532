// Host-side launchers of the attention and cache kernels; called by the C ABI
// after validation.
#pragma once

#include <algorithm>

#include "tf_attn_common.h"

namespace tf {

int device_cus();

// ---- one new token per sequence -------------------------------------------
struct DecodeArgs {
    const uint16_t *q;
    int64_t q_token, q_head; // strides in elements
    PagedCache cache;
    const int32_t *lens;
    uint16_t *out; // [seqs][Hq][D]
    float *part;    // [shares][2][16 nt][D]: partial results of items that a share holds in part
    float *stats;   // [shares][2][16 nt][2]: their maximum and sum
    int32_t *spans; // [shares][3]: shares of the item that begins here and ends later (0: none), its sequence and number
    int seqs, G, groups, longest;
    int unit_shift; // shares are cut at multiples of 2^unit_shift keys
    float scale_log2;
};
struct DecodePlan {
    int64_t nt, groups, shares; // shares == 0: a workgroup per item
    int64_t waves, unit_shift;  // of a workgroup per item; of shares
};
DecodePlan plan_decode(int64_t seqs, int64_t hkv, int64_t G, int64_t longest, int cus);
hipError_t launch_attn_decode(const DecodeArgs &a, int D, bool f16, const DecodePlan &p, hipStream_t st);

// ---- packed prompts ---------------------------------------------------------
struct PrefillArgs {
    const uint16_t *q;
    int64_t q_token, q_head;
    const uint16_t *k, *v; // packed keys and values, or NULL for the paged call
    int64_t k_token, k_head, v_token, v_head;
    PagedCache cache;
    const int32_t *cu_q, *cu_k, *lens; // cu_k: packed; lens: paged
    uint16_t *out;                     // [T][Hq][D]
    int tokens, keys, hkv, G, longest;
    float scale_log2;
    int seqs, splits; // ranges of keys
    float *part;      // [T][Hq][splits][D], when splits > 1
    float *stats;     // [T][Hq][splits][2]: maximum, sum
    // set by the launch: row blocks of the longest (sequence, head), heads next to
    // each other in the grid; or, all sequences side by side, no more blocks of
    // a head than all_blocks, and the first step of the search for one
    int blocks, heads_by, all_blocks, steps;
};
constexpr int kPrefillRows = 128; // rows (token, head of a group) of a workgroup
inline int64_t prefill_blocks(int64_t longest, int64_t G) { return (longest * G + kPrefillRows - 1) / kPrefillRows; }
int plan_prefill_splits(int64_t seqs, int64_t T, int64_t hkv, int64_t G, int64_t longest, int64_t keys, int cus);
hipError_t launch_attn_prefill(PrefillArgs a, int D, bool f16, bool paged, int64_t seqs, hipStream_t st);

// ---- the cache -----------------------------------------------------------------
struct AppendArgs {
    const uint16_t *qkv;
    int64_t qkv_token;
    const float *rope;
    int rope_rows;
    const int32_t *seq, *pos, *tables;
    uint16_t *q, *k, *v;
    int tokens, seqs, width, pages, hq, hkv, D, page_shift;
};
hipError_t launch_kv_append(const AppendArgs &a, bool f16, hipStream_t st);

struct PoolArgs {
    uint16_t *cache; // [planes][pages][Hkv][page][D]
    const int32_t *refs, *tables, *lens, *parents, *children;
    int32_t *refs_out, *tables_out, *lens_out;
    int32_t *told; // fork: status [1]; compact: moved [pages]
    int32_t *plan; // workspace
    int64_t planes;
    int pages, hkv, page, D, seqs, width, forks;
};
hipError_t launch_kv_fork(const PoolArgs &a, hipStream_t st);
hipError_t launch_kv_compact(const PoolArgs &a, hipStream_t st);

} // namespace tf
