// matrix.h -- matrix-core and softmax helpers shared by the attention kernels
// (gfx950 only): the two MFMA shapes they use with the lane layout each
// assumes, the transposing LDS read, base-2 exp and log, and the exchange of
// a value between the two halves of a wave.
//
// Lane layouts (lane l of 64, operand elements j = 0..7, result elements r):
//   mma32 (32x32x16): A row = l % 32, B column = l % 32, both k = 8 (l / 32) + j;
//     C column = l % 32, row = r % 4 + 8 (r / 4) + 4 (l / 32), r = 0..15.
//   mma16 (16x16x32): A row = l % 16, B column = l % 16, both k = 8 (l / 16) + j;
//     C column = l % 16, row = 4 (l / 16) + r, r = 0..3.
// Products of 16-bit operands are exact in fp32 and the sums are fp32.
#pragma once

#include "coll_internal.h"

namespace coll {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#ifndef COLL_HAVE_MATRIX
template <int DT>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == COLL_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == COLL_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Transposing LDS read: in each group of 16 lanes, lanes 4 j .. 4 j + 3 name
// the 16 columns (4 apiece, 8 bytes) of row j, and lane i gets column i of
// rows 0..3.
__device__ __forceinline__ u32x2 lds_tr16(const void *p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
}

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_f(float x) { return __builtin_amdgcn_logf(x); }

// Between LDS writes of a wave and its reads of what other lanes of the same
// wave wrote (or the other way round): the hardware keeps a wave's LDS
// accesses in order, so only the compiler has to.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// max over lanes l and l ^ 32
__device__ __forceinline__ float max_halves(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
#endif

// Kernel arguments taken to be needed here, all at once: a struct of tables
// spans many cache lines, and lines first touched where their values are used
// cost a trip to memory each, one after the other.  Emits no instruction.
#ifndef COLL_FETCH
#define COLL_FETCH(a, b, c, d, e, f, g, h) \
  asm volatile("" ::"s"(a), "s"(b), "s"(c), "s"(d), "s"(e), "s"(f), "s"(g), "s"(h))
#endif

// x as if computed anew here: what is rarely needed is then not computed ahead
// of a loop and kept (or spilled) through it.  Emits no instruction.
#ifndef COLL_FRESH
#define COLL_FRESH(x) asm volatile("" : "+v"(x))
#endif

// Two fp32 -> a pair of the 16-bit type, round to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == COLL_BF16) return pack_bf16(lo, hi);
  else return pack_f16(lo, hi);
}

// x of lane l ^ m
__device__ __forceinline__ float lane_xor(float x, int m) {
  return __shfl(x, (int)(threadIdx.x & 63) ^ m, 64);
}

// 16-bit element pair -> its bits with the sign cleared are at or above the
// infinity pattern in either half (an infinity or a NaN)
template <int DT>
__device__ __forceinline__ bool pair_not_finite(uint32_t w) {
  constexpr uint32_t inf = DT == COLL_BF16 ? 0x7F80u : 0x7C00u;
  return (w & 0x7FFFu) >= inf || ((w >> 16) & 0x7FFFu) >= inf;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace coll
