// CPU emulation of the HIP device subset the library's kernels use -- TEST
// INFRASTRUCTURE ONLY.  The library's .hip sources compile unchanged against
// this header as plain C++ for the host; kernels then run on the CPU, each
// workgroup's lanes as cooperative fibers grouped in wave64s, so barriers,
// ballots, shuffles and readfirstlane behave as they do on the GPU and every
// memory access goes to host memory, where guard pages catch any access past
// a buffer.  Nothing here is part of the product.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

// ---------------------------------------------------------------- qualifiers
#define __global__
#define __device__
#define __host__
#define __forceinline__ inline __attribute__((always_inline))
#define __launch_bounds__(...)
#define __align__(n) __attribute__((aligned(n)))
// LDS: every __shared__ variable goes to the section emu_lds, which the
// emulator fills with a poison pattern before each workgroup starts, so a
// kernel that reads LDS it did not write first computes garbage.
#define __shared__ __attribute__((section("emu_lds"))) static

// the library's scheduling fences emit nothing on the CPU; COLL_UNIFORM, which
// on the GPU moves its value into a scalar register (lane 0's copy wins if the
// lanes disagree), is checked instead: every active lane must hold the same
// bits, or the run aborts naming the site (see the wave ops below)
#define COLL_OPAQUE(x) ((void)0)
#define COLL_KEEP(x) ((void)0)
#define COLL_SCALAR(x) ((void)0)
#define COLL_FETCH(...) ((void)0)
#define COLL_FRESH(x) ((void)0)
// ld_scalar: the GPU reads through the scalar cache, which needs the address
// to be the same in every lane; here it is a plain load, after checking that
// every active lane asks for the same address (defined below emu_uniform_at)
#define COLL_HAVE_LD_SCALAR 1
#define ld_scalar(p, i) emu_ld_scalar((p), (size_t)(i), __FILE__, __LINE__)
#define COLL_UNIFORM(x) emu_uniform_at(emu_bits(x), __FILE__, __LINE__)

// ------------------------------------------------------------- runtime types
typedef int hipError_t;
enum { hipSuccess = 0, hipErrorInvalidConfiguration = 9, hipErrorInvalidValue = 1 };
typedef struct emu_stream *hipStream_t;
typedef int hipDeviceAttribute_t;
enum { hipDeviceAttributeMultiprocessorCount = 1 };

struct dim3 {
  unsigned x, y, z;
  constexpr dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};
struct emu_uint3 {
  unsigned x, y, z;
};

extern "C" {
hipError_t hipGetLastError(void);
hipError_t hipGetDevice(int *dev);
hipError_t hipDeviceGetAttribute(int *value, hipDeviceAttribute_t attr, int dev);
// scheduler entry points (emu.cpp)
const emu_uint3 *emu_thread_idx(void);
extern emu_uint3 emu_block_idx, emu_block_dim, emu_grid_dim;
void emu_syncthreads(void);
uint64_t emu_wave_op(int op, uint64_t value, int arg, const char *file, int line);
void emu_run_grid(dim3 grid, dim3 block, void (*body)(void *), void *ctx);
}

#define threadIdx (*emu_thread_idx())
#define blockIdx emu_block_idx
#define blockDim emu_block_dim
#define gridDim emu_grid_dim
#define __syncthreads() emu_syncthreads()

static inline hipError_t hipGetSymbolAddress(void **p, const void *sym) {
  *p = const_cast<void *>(sym);
  return hipSuccess;
}
#define HIP_SYMBOL(x) (&(x))

// --------------------------------------------------------------- wave ops
// Each op is a rendezvous of the wave's active lanes at one source position
// (file, line): the same position however the compiler duplicates its code.
// readfirstlane and COLL_UNIFORM also check that every active lane holds the
// same value: the library uses both only on values it takes to be uniform
// (slots, ranks and descriptors loaded from one address), and a lane that
// disagreed would go on with lane 0's address on the GPU.
enum { EMU_BALLOT = 1, EMU_SHFL = 2, EMU_SHFL_UP = 3, EMU_FIRSTLANE = 4, EMU_READLANE = 5,
       EMU_UNIFORM = 6, EMU_MATRIX = 7, EMU_LDS_TR16 = 8 };

// Operands of one lane of a matrix instruction (EMU_MATRIX), passed by the
// address of this record: the whole wave must take part.
struct emu_matrix {
  int dt;               // 0 = bf16, 1 = fp16
  int wide;             // 1: 32x32x16, 0: 16x16x32
  uint16_t a[8], b[8];
  float c[16];
};

template <class T>
static inline uint64_t emu_bits(T v) {
  static_assert(sizeof(T) <= 8, "wave op payload");
  uint64_t b = 0;
  memcpy(&b, &v, sizeof(T));
  return b;
}
template <class T>
static inline T emu_from(uint64_t b) {
  T v;
  memcpy(&v, &b, sizeof(T));
  return v;
}

static inline uint64_t emu_ballot_at(int pred, const char *f, int l) {
  return emu_wave_op(EMU_BALLOT, pred ? 1 : 0, 0, f, l);
}
template <class T>
static inline T emu_shfl_at(T v, int src, int width, const char *f, int l) {
  (void)width;
  return emu_from<T>(emu_wave_op(EMU_SHFL, emu_bits(v), src, f, l));
}
template <class T>
static inline T emu_shfl_up_at(T v, unsigned delta, int width, const char *f, int l) {
  (void)width;
  return emu_from<T>(emu_wave_op(EMU_SHFL_UP, emu_bits(v), (int)delta, f, l));
}
static inline int emu_readfirstlane_at(int v, const char *f, int l) {
  return (int)emu_wave_op(EMU_FIRSTLANE, (uint32_t)v, 0, f, l);
}
static inline void emu_uniform_at(uint64_t bits, const char *f, int l) {
  (void)emu_wave_op(EMU_UNIFORM, bits, 0, f, l);
}

template <class T>
static inline T emu_ld_scalar(const T *p, size_t i, const char *f, int l) {
  emu_uniform_at((uint64_t)(uintptr_t)(p + i), f, l);
  return p[i];
}
static inline int emu_readlane_at(int v, int lane, const char *f, int l) {
  return (int)emu_wave_op(EMU_READLANE, (uint32_t)v, lane, f, l);
}

#define __ballot(p) emu_ballot_at((int)(p), __FILE__, __LINE__)
#define __shfl(v, s, w) emu_shfl_at((v), (s), (w), __FILE__, __LINE__)
#define __shfl_up(v, d, w) emu_shfl_up_at((v), (unsigned)(d), (w), __FILE__, __LINE__)
#define __builtin_amdgcn_readfirstlane(v) emu_readfirstlane_at((int)(v), __FILE__, __LINE__)
#define __builtin_amdgcn_readlane(v, l) emu_readlane_at((int)(v), (int)(l), __FILE__, __LINE__)

// --------------------------------------------------- matrix.h's helpers
// The library's matrix.h leaves these to the including environment when
// COLL_HAVE_MATRIX is defined; layouts as documented there.
#define COLL_HAVE_MATRIX 1
#define __builtin_amdgcn_s_setprio(x) ((void)0)
typedef uint32_t emu_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t emu_u32x2 __attribute__((ext_vector_type(2)));
typedef float emu_f32x4 __attribute__((ext_vector_type(4)));
typedef float emu_f32x16 __attribute__((ext_vector_type(16)));

template <int DT, int WIDE, int NR, class C>
static inline C emu_mma(emu_u32x4 a, emu_u32x4 b, C c, const char *f, int l) {
  emu_matrix m;
  m.dt = DT;
  m.wide = WIDE;
  for (int i = 0; i < 4; i++) {
    m.a[2 * i] = (uint16_t)a[i];
    m.a[2 * i + 1] = (uint16_t)(a[i] >> 16);
    m.b[2 * i] = (uint16_t)b[i];
    m.b[2 * i + 1] = (uint16_t)(b[i] >> 16);
  }
  for (int i = 0; i < NR; i++) m.c[i] = c[i];
  emu_wave_op(EMU_MATRIX, (uint64_t)(uintptr_t)&m, 0, f, l);
  for (int i = 0; i < NR; i++) c[i] = m.c[i];
  return c;
}
template <int DT>
static inline emu_f32x16 emu_mma32(emu_u32x4 a, emu_u32x4 b, emu_f32x16 c, const char *f, int l) {
  return emu_mma<DT, 1, 16>(a, b, c, f, l);
}
template <int DT>
static inline emu_f32x4 emu_mma16(emu_u32x4 a, emu_u32x4 b, emu_f32x4 c, const char *f, int l) {
  return emu_mma<DT, 0, 4>(a, b, c, f, l);
}
template <int DT>
static inline emu_f32x16 mma32(emu_u32x4 a, emu_u32x4 b, emu_f32x16 c,
                               const char *f = __builtin_FILE(), int l = __builtin_LINE()) {
  return emu_mma32<DT>(a, b, c, f, l);
}
template <int DT>
static inline emu_f32x4 mma16(emu_u32x4 a, emu_u32x4 b, emu_f32x4 c,
                              const char *f = __builtin_FILE(), int l = __builtin_LINE()) {
  return emu_mma16<DT>(a, b, c, f, l);
}
static inline emu_u32x2 lds_tr16(const void *p, const char *f = __builtin_FILE(),
                                 int l = __builtin_LINE()) {
  uint64_t v;
  memcpy(&v, p, 8);
  const uint64_t r = emu_wave_op(EMU_LDS_TR16, v, 0, f, l);
  emu_u32x2 x = {(uint32_t)r, (uint32_t)(r >> 32)};
  return x;
}
static inline float exp2_f(float x) { return exp2f(x); }
static inline float log2_f(float x) { return log2f(x); }
static inline float max_halves(float x, const char *f = __builtin_FILE(), int l = __builtin_LINE()) {
  const int other = (int)(emu_thread_idx()->x & 63) ^ 32;
  return fmaxf(x, emu_shfl_at(x, other, 64, f, l));
}
// every lane of the wave gets here before any goes on
static inline void wave_lds_sync(const char *f = __builtin_FILE(), int l = __builtin_LINE()) {
  (void)emu_wave_op(EMU_BALLOT, 1, 0, f, l);
}
struct int4 {
  int x, y, z, w;
};

// ------------------------------------------------------------ integer helpers
static inline int __popcll(unsigned long long x) { return __builtin_popcountll(x); }
static inline int __popc(unsigned x) { return __builtin_popcount(x); }
static inline unsigned __umulhi(unsigned a, unsigned b) {
  return (unsigned)(((unsigned long long)a * b) >> 32);
}
static inline unsigned long long __umul64hi(unsigned long long a, unsigned long long b) {
  return (unsigned long long)(((unsigned __int128)a * b) >> 64);
}
// lanes run one at a time, so a plain read-modify-write is atomic
template <class T>
static inline T atomicAdd(T *p, T v) {
  T old = *p;
  *p = old + v;
  return old;
}
template <class T>
static inline T atomicMax(T *p, T v) {
  T old = *p;
  if (v > old) *p = v;
  return old;
}
template <class T>
static inline T atomicMin(T *p, T v) {
  T old = *p;
  if (v < old) *p = v;
  return old;
}
template <class T>
static inline T atomicCAS(T *p, T expected, T v) {
  T old = *p;
  if (old == expected) *p = v;
  return old;
}

// ------------------------------------------------------------------ launch
template <class Body>
static void emu_trampoline(void *ctx) {
  (*static_cast<Body *>(ctx))();
}

template <class F, class... A>
static void emu_launch(F kernel, dim3 grid, dim3 block, size_t shmem, hipStream_t stream,
                       A... args) {
  (void)shmem;
  (void)stream;
  auto body = [&]() { kernel(args...); };
  emu_run_grid(grid, block, &emu_trampoline<decltype(body)>, &body);
}

#define hipLaunchKernelGGL(K, G, B, S, ST, ...) emu_launch(K, dim3(G), dim3(B), (S), (ST), __VA_ARGS__)
