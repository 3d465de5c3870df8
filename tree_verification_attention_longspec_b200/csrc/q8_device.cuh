// The 8-bit cache: argument blocks and conversions shared by its kernels.
//
// A cached value is code * scale, the code an e4m3 number (4 significant bits, largest
// 448) and the scale an fp32 number shared by `scale_block` consecutive tokens of one page
// and kv head, for keys and values apart.
#pragma once
#include <cuda_fp16.h>

#include "ls_device.cuh"
#include "q8_pages.cuh"

namespace ls {

// Block scales outside this range count as its ends: the attention folds a value's scale
// into its weight's exponent, and the sums take it out again, both in fp32.
constexpr int kMinScaleExp = -60, kMaxScaleExp = 64;

// Query rows of a kv head up to which the 8-bit cache streams through registers (attn_q8_rows.cu).
constexpr int kQ8MaxRows = 32;

#if defined(LS_DEBUG)
// Whether the table names a page of the cache for key `key` of sequence b.
__device__ __forceinline__ bool q8_page_exists(const KvQ8& kv, int32_t b, int32_t key) {
  const int32_t lp = key / kv.page_size;
  return lp < kv.max_pages && (uint32_t)kv.page_table[(size_t)b * kv.max_pages + lp] < (uint32_t)kv.num_pages;
}
#endif

// Two e4m3 codes (low 16 bits of w) as packed f16: exact, NaN codes stay NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// (lo, hi) as e4m3 codes in 16 bits, round to nearest even, saturated at +-448.
__device__ __forceinline__ uint16_t f32x2_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// floor(log2 x) of a finite x > 0, with subnormals (which bf16 inputs can hold) as -127.
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

// The f16 forms of bf16 rows are their values times 2^shift with the row's largest
// magnitude in [2^14, 2^15): bf16's 8 significant bits fit f16's 11, and what falls below
// f16's subnormals is 2^-38 of the largest. shift is at most 126 and at least -113 (-114 where
// the largest is infinite).
__device__ __forceinline__ int f16_shift(float amax) { return min(126, 14 - exponent_of(amax)); }

// Attention over the 8-bit cache.
struct Q8Args {
  const uint16_t* q;  // bf16 [N][Hq][d]
  const uint16_t* k_tree;
  const uint16_t* v_tree;
  const int32_t* parent;
  const int32_t* cu;
  const int32_t* cu_tree;
  KvQ8 kv;
  float* o_part;
  float* lse_part;
  uint32_t* chunk_status;
  int32_t after_prep;  // q and k_tree are written by the tree kernel launched just before
  Plan p;
};

// Rows appended to the cache and quantised.
struct AppendArgs {
  const uint16_t* k_new;  // bf16 [rows][Hkv][d]
  const uint16_t* v_new;
  const int32_t* cu;       // [B+1] tokens in the cache before
  const int32_t* cu_new;   // [B+1] rows of each sequence, or (nullptr) the accepted paths:
  const int32_t* accept_len;
  const int32_t* accept_path;
  const int32_t* cu_tree;
  int32_t* cu_out;  // [B+1] tokens in the cache after, or nullptr
  KvQ8 kv;
  int32_t B, Hkv, d, T;
  int32_t rows;     // rows of k_new / v_new
  int32_t max_new;  // rows a sequence may append
  int32_t team_shift;  // log2 of the warps of a block (the kernel's own)
  int64_t blocks;   // scale blocks that the sequences may touch in all
};

cudaError_t launch_q8_rows(const Q8Args& a, cudaStream_t stream);
cudaError_t launch_q8_tc(const Q8Args& a, cudaStream_t stream);
cudaError_t launch_q8_append(const AppendArgs& a, cudaStream_t stream);

}  // namespace ls
