// Shared pieces of the attention kernels: the online-softmax state, lane
// exchanges, LDS transpose reads, and the addressing of a paged cache.
//
// Both attention kernels hold scores and outputs transposed, S^T = K Q^T and
// O^T = V^T P^T, with one query row per MFMA column.  A lane then owns one
// query (two or four lanes share it), so the running maximum, the rescaling
// of O and the final division are per-lane scalars, and the accumulator
// layout of S^T is already the operand layout of P^T once the keys inside an
// MFMA step are taken in that order; V follows by reading its rows through
// the LDS transpose read in the same order.  No probability ever moves
// between lanes or through memory.
#pragma once

#include "tf_gemm_common.h"

namespace tf {

// Softmax runs in base 2: p = exp2(s c - m) with c = scale log2(e).  The
// running maximum m starts at kLowest, the lowest finite number, rather than
// at -inf, so that a row with no visible key keeps m finite: every
// exp2(-inf - m) is 0, the sum stays 0 and the row's output is 0; no finite
// score lies below it.
constexpr float kLowest = -3.402823466e38f;
// O and the sum are rescaled only when a row's maximum has grown by more
// than this many powers of two: until then p <= 2^8, which bf16, fp16 and
// the fp32 sums all hold with the same relative precision.
constexpr float kRescaleSlack = 8.0f;
// m is held this many powers of two below the maximum: fp16's smallest
// numbers are 2^-24, and a long row's many small weights must not round to
// zero there.  p reaches 2^15 at most, inside fp16; bf16 has fp32's range.
template <bool F16> constexpr float kHeadroom = F16 ? 7.0f : 0.0f;
// s c - m is one fused operation, m a rounded product: they differ by half a
// step of m, 2^-4 below this size.  Scores past it, whose steps reach whole
// powers of two (2^32: 2^8), are multiplied first, rounded as m was, so that
// the largest one's weight is not 2^(half a step), infinite or zero.  Their m
// is held at the maximum itself, for there steps swallow the headroom.
constexpr float kLargeScore = 1048576.0f;
template <bool F16> __device__ __forceinline__ float held_maximum(float top)
{
    return F16 ? top - (fabsf(top) < kLargeScore ? kHeadroom<F16> : 0.f) : top;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max / sum of a value over the lanes l, l ^ 32
__device__ __forceinline__ float max_swap32(float x)
{
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_swap16(float x)
{
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_swap32(float x)
{
    const uint32_t b = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// LDS transpose read: in each group of 16 lanes, lane i supplies the address
// of 4 consecutive 16-bit values; lanes 4 r .. 4 r + 3 together name row r of
// a 4 x 16 matrix, and lane j receives its column j (rows 0..3).
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 lds_read_tr(const uint8_t *__restrict__ p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4 *)p));
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Rows of a run of 16 that lie before `end`; all arguments uniform.  The empty
// asm keeps the compiler from joining the two bounds to a clamp, which it puts
// on the vector unit even for uniform values: a buffer resource made from it
// is then looped over lane by lane.
__device__ __forceinline__ int rows_before(int end, int first)
{
    int left = max(end - first, 0);
    asm("" : "+s"(left));
    return min(left, 16);
}

// A raw buffer of `bytes` bytes: lanes at or past the end read zeros without
// a memory access.
__device__ __forceinline__ Rsrc make_rsrc_n(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)bytes, 0x00020000);
}

// A cache plane [pages][Hkv][page][D] of 16-bit values and the table row of
// one sequence.
struct PagedCache {
    const uint16_t *k, *v;
    const int32_t *tables; // [seqs][width]
    int pages, hkv, page_shift, width;
};

} // namespace tf
