// attn_decode.hip -- attention of one new token over a paged cache.
//
// Rank r, batch entry b (row seqs[b] of the page table, or row b), head h of
// kv head h / G: with the cache's first len tokens as keys and values,
//   s_t = scale * q . k_t,  m = max s_t,  p_t = exp(s_t - m),  l = sum p_t,
//   o = sum p_t v_t / l,    lse = m + log l.
// Token t lies in page table[row][t / P] at slot t % P.
//
// The keys and values are read once, and that is what bounds it.  The work
// is one list of units of 128 tokens of one (rank, entry, kv head), and
// every workgroup takes an equal, contiguous share of it, whatever the
// lengths: long caches are split among many workgroups, short ones share
// one.  A workgroup that holds all units of a head writes its output;
// otherwise it leaves its partial (m, l, unnormalised o) in the workspace
// and a second kernel joins the partials.
//
// A wave takes 32 tokens at a time, straight from memory to the registers
// the matrix instructions read.  S = K Q^T has a token per row and a head
// per column; the rows are dealt so that a lane ends with 8 consecutive
// tokens of one head, which is how the B operand of O^T = V^T P^T wants
// them.  V's operand holds 8 tokens of one column per lane: a lane loads
// the same few columns of 8 tokens and transposes the block in registers.
#include "matrix.h"

#pragma clang fp contract(off)

namespace coll {
namespace {

constexpr int kUnit = 128;            // tokens of one unit: 32 for each of 4 waves
constexpr int kHeadTile = 16;         // query heads of one kv head that share a pass
constexpr int kJoinLanes = 512;

struct DecodeArgs {
  PtrTable q, k, v, table, lens, seqs;
  MutPtrTable o, lse;
  int64_t q_stride, o_stride;                       // elements between entries
  int64_t page_stride, tok_stride, head_stride;     // elements, both pools
  int64_t num_pages;
  int batch, rows, max_pages, page_size;
  int heads, kv_heads, group, head_tiles;           // head_tiles per kv head
  int entries;                                      // ranks * batch
  FastDiv by_batch, by_page, by_head_tiles;
  float c;                                          // |scale| * log2 e
  int negate;
  float *part;                                      // partial slots, two per workgroup
  int4 *joins;                                      // per workgroup: {partials, first slot, entry, head tile}
};

// Floats of one partial slot: the outputs, then m and l per head.
template <int D>
constexpr int slot_floats() {
  return kHeadTile * D + 2 * kHeadTile;
}

// Length of entry e's cache, clipped to what its table row can hold.
__device__ __forceinline__ int entry_len(const DecodeArgs &A, int e, int *row) {
  const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;
  const int32_t *sq = reinterpret_cast<const int32_t *>(A.seqs.p[r]);
  const int x = sq ? sq[b] : b;
  *row = x;
  if (x < 0 || x >= A.rows) return 0;
  const int64_t n = reinterpret_cast<const int32_t *>(A.lens.p[r])[x];
  const int64_t most = (int64_t)A.max_pages * A.page_size;
  return n < 0 ? 0 : (int)(n < most ? n : most);
}
__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + kUnit - 1) / kUnit : 1; }

// First unit of workgroup w's share of n units among `of` workgroups.
__device__ __forceinline__ int share(int64_t n, int w, int of) { return (int)(n * w / of); }

template <int ND>
struct Chunk {                 // 32 tokens of one wave, as loaded
  u32x4 k[2][ND];
  uint32_t v[8][ND];
  uint32_t ok;                 // bit j: token 8 g + j of the chunk exists
};

template <int DT, int ND, bool P8>
__global__ __launch_bounds__(256, 2) void decode_split(DecodeArgs A) {
  constexpr int D = 32 * ND, NV = P8 ? 1 : 8, NK = P8 ? 1 : 2;
  constexpr int kOutRow = D + 4;
  constexpr bool kAhead = ND <= 4;      // two chunks in registers: 64 of them each at D = 128
  __shared__ int s_pre[257], s_wave[4];
  __shared__ float s_m[4][kHeadTile], s_l[4][kHeadTile];
  __shared__ __align__(16) float s_o[4][kHeadTile][kOutRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int per_entry = A.kv_heads * A.head_tiles;

  // prefix sums of the entries' units, 256 entries at a time: s_pre[i] = units
  // before entry base + i (all head tiles together)
  int base = 0;
  auto scan = [&](int carry) {
    const int e = base + tid;
    int row;
    const int mine = e < A.entries ? units_of(entry_len(A, e, &row)) * per_entry : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int x = __shfl_up(upto, d, 64);
      if (lane >= d) upto += x;
    }
    __syncthreads();
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < 3; w++) before += w < wave ? s_wave[w] : 0;
    s_pre[tid + 1] = before + upto;
    if (tid == 0) s_pre[0] = carry;
    __syncthreads();
  };
  scan(0);
  int total = s_pre[256];
  if (A.entries > 256) {
    for (base = 256; base < A.entries; base += 256) {
      const int carry = s_pre[256];
      scan(carry);
    }
    total = s_pre[256];
    base = 0;
    scan(0);
  }
  // as many workgroups share the units as there are units, so that each of
  // them has one and the joined partials are those of consecutive workgroups
  const int W = (int)gridDim.x < total ? (int)gridDim.x : total, w0 = (int)blockIdx.x;
  int u = w0 < W ? share(total, w0, W) : 0;
  const int u1 = w0 < W ? share(total, w0 + 1, W) : 0, begin = u;
  int4 join = {0, 0, 0, 0};

  while (u < u1) {
    while (u >= s_pre[256]) {
      const int carry = s_pre[256];
      base += 256;
      scan(carry);
    }
    // the entry that holds unit u: the last i with s_pre[i] <= u
    int lo = 0, hi = 256;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= u) lo = mid;
      else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(base + lo);
    int row_v;
    const int len = __builtin_amdgcn_readfirstlane(entry_len(A, e, &row_v));
    const int trow = __builtin_amdgcn_readfirstlane(row_v);
    const int nu = units_of(len);
    const int local = u - s_pre[lo], ht = local / nu, t0 = local - ht * nu;
    const int t1 = nu < t0 + (u1 - u) ? nu : t0 + (u1 - u);
    const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;
    const int kvh = (int)fdiv((uint32_t)ht, A.by_head_tiles), part = ht - kvh * A.head_tiles;
    const int h0 = kvh * A.group + part * kHeadTile;
    const int nh = A.group - part * kHeadTile < kHeadTile ? A.group - part * kHeadTile : kHeadTile;

    // Q as the B operand: column = head, 8 consecutive elements per lane
    u32x4 q[ND];
#pragma unroll
    for (int s = 0; s < ND; s++) {
      u32x4 x = {0, 0, 0, 0};
      if (i16 < nh)
        x = ld<u32x4>(reinterpret_cast<const char *>(A.q.p[r]) +
                          (b * A.q_stride + (int64_t)(h0 + i16) * D) * 2, 4 * s + g);
      if (A.negate) x = x ^ 0x80008000u;
      q[s] = x;
    }
    const char *kp = reinterpret_cast<const char *>(A.k.p[r]) + (int64_t)kvh * A.head_stride * 2;
    const char *vp = reinterpret_cast<const char *>(A.v.p[r]) + (int64_t)kvh * A.head_stride * 2;
    const int32_t *pages = reinterpret_cast<const int32_t *>(A.table.p[r]) +
                           (len > 0 ? (int64_t)trow * A.max_pages : 0);

    // Tokens of a chunk that starts at token `at`: operand row i of K's tile
    // m is token 8 (i / 4) + 4 m + i % 4; V's elements are tokens 8 g + j.
    // With pages of a multiple of 8 tokens, 8 of them share one look-up.
    struct Look {
      int32_t v[NV], k[NK];
    };
    auto look = [&](int at) -> Look {
      Look x;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const int t = at + 8 * g + j;
        x.v[j] = t < len ? pages[fdiv((uint32_t)t, A.by_page)] : -1;
      }
#pragma unroll
      for (int m = 0; m < NK; m++) {
        const int t = at + 8 * (i16 >> 2) + (P8 ? 0 : 4 * m + (i16 & 3));
        x.k[m] = t < len ? pages[fdiv((uint32_t)t, A.by_page)] : -1;
      }
      return x;
    };
    auto slot_of = [&](int t) -> int { return t - (int)fdiv((uint32_t)t, A.by_page) * A.page_size; };
    // an absent token reads the pool's first row instead (its score is
    // masked and its value replaced by 0 before use)
    auto load = [&](int at, const Look &x) -> Chunk<ND> {
      Chunk<ND> ch;
      ch.ok = 0;
#pragma unroll
      for (int m = 0; m < 2; m++) {
        const int t = at + 8 * (i16 >> 2) + 4 * m + (i16 & 3);
        const int32_t pg = x.k[P8 ? 0 : m];
        const bool ok = t < len && pg >= 0 && pg < A.num_pages;
        const int64_t off = ok ? pg * A.page_stride + slot_of(t) * A.tok_stride : 0;
#pragma unroll
        for (int s = 0; s < ND; s++) ch.k[m][s] = ld<u32x4>(kp + off * 2, 4 * s + g);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int t = at + 8 * g + j;
        const int32_t pg = x.v[P8 ? 0 : j];
        const bool ok = t < len && pg >= 0 && pg < A.num_pages;
        const int64_t off = ok ? pg * A.page_stride + slot_of(t) * A.tok_stride : 0;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(vp + off * 2) + i16 * ND;
#pragma unroll
        for (int x2 = 0; x2 < ND; x2++) ch.v[j][x2] = src[x2];
        ch.ok |= ok ? 1u << j : 0u;
      }
      return ch;
    };

    f32x4 acc[2 * ND];
#pragma unroll
    for (int x = 0; x < 2 * ND; x++) acc[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -__builtin_inff(), l = 0.0f;

    auto compute = [&](Chunk<ND> &ch) {
      f32x4 s[2];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        s[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < ND; d++) s[x] = mma16<DT>(ch.k[x][d], q[d], s[x]);
      }
      if (__ballot(ch.ok != 0xFFu)) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const bool ok = (ch.ok >> j) & 1;
          s[j >> 2][j & 3] = ok ? s[j >> 2][j & 3] : -__builtin_inff();
#pragma unroll
          for (int x = 0; x < ND; x++) ch.v[j][x] = ok ? ch.v[j][x] : 0u;
        }
      }
      float mt = s[0][0];
#pragma unroll
      for (int j = 1; j < 8; j++) mt = fmaxf(mt, s[j >> 2][j & 3]);
      mt = fmaxf(mt, lane_xor(mt, 16));
      mt = fmaxf(mt, lane_xor(mt, 32));
      if (__ballot((mt - m) * A.c > 8.0f)) {
        const float mn = fmaxf(m, mt);
        const float f = mn == -__builtin_inff() ? 1.0f : exp2_f((m - mn) * A.c);
        m = mn;
        l *= f;
#pragma unroll
        for (int x = 0; x < 2 * ND; x++)
#pragma unroll
          for (int e2 = 0; e2 < 4; e2++) acc[x][e2] *= f;
      }
      const float mc = m == -__builtin_inff() ? 0.0f : m * A.c;
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        p[j] = exp2_f(__builtin_fmaf(s[j >> 2][j & 3], A.c, -mc));
        l += p[j];
      }
      u32x4 pf;
#pragma unroll
      for (int j = 0; j < 4; j++) pf[j] = pack2<DT>(p[2 * j], p[2 * j + 1]);
#pragma unroll
      for (int x = 0; x < ND; x++) {
        u32x4 even, odd;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          even[j] = (ch.v[2 * j][x] & 0xFFFFu) | (ch.v[2 * j + 1][x] << 16);
          odd[j] = (ch.v[2 * j][x] >> 16) | (ch.v[2 * j + 1][x] & 0xFFFF0000u);
        }
        acc[2 * x] = mma16<DT>(even, pf, acc[2 * x]);
        acc[2 * x + 1] = mma16<DT>(odd, pf, acc[2 * x + 1]);
      }
    };

    // the wave's chunks: tokens 128 t + 32 wave .., loads one chunk ahead of
    // the arithmetic and page look-ups one further
    const int stop = len < t1 * kUnit ? len : t1 * kUnit;
    int at = t0 * kUnit + wave * 32;
    if (at < stop) {
      Look nxt = look(at);
      if constexpr (kAhead) {
        Chunk<ND> cur = load(at, nxt);
        nxt = look(at + kUnit);
        for (;;) {
          const bool more = at + kUnit < stop;
          Chunk<ND> ahead;
          if (more) {
            ahead = load(at + kUnit, nxt);
            nxt = look(at + 2 * kUnit);
          }
          compute(cur);
          if (!more) break;
          cur = ahead;
          at += kUnit;
        }
      } else {
        for (; at < stop; at += kUnit) {
          Chunk<ND> cur = load(at, nxt);
          nxt = look(at + kUnit);
          compute(cur);
        }
      }
    }

    // join the four waves: weights exp2((m_w - m) c), then one sum per output
    l += lane_xor(l, 16);
    l += lane_xor(l, 32);
    if (g == 0) {
      s_m[wave][i16] = m;
      s_l[wave][i16] = l;
    }
    __syncthreads();
    float mm = s_m[0][i16];
#pragma unroll
    for (int w = 1; w < 4; w++) mm = fmaxf(mm, s_m[w][i16]);
    {
      const float f = m == -__builtin_inff() ? (l != l ? l : 0.0f) : exp2_f((m - mm) * A.c);
#pragma unroll
      for (int rr = 0; rr < 4; rr++)
#pragma unroll
        for (int x = 0; x < 2 * ND; x++) s_o[wave][i16][2 * ND * (4 * g + rr) + x] = acc[x][rr] * f;
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nu;
    const int slot = 2 * w0 + (u == begin ? 0 : 1);
    float *ps = A.part + (int64_t)slot * slot_floats<D>();
    for (int x = tid; x < nh * (D / 2); x += 256) {
      const int hh = x / (D / 2), d = 2 * (x - hh * (D / 2));
      float M = s_m[0][hh];
#pragma unroll
      for (int w = 1; w < 4; w++) M = fmaxf(M, s_m[w][hh]);
      float y0 = 0.0f, y1 = 0.0f, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const float mw = s_m[w][hh], lw = s_l[w][hh];
        ll += mw == -__builtin_inff() ? (lw != lw ? lw : 0.0f) : lw * exp2_f((mw - M) * A.c);
        y0 += s_o[w][hh][d];
        y1 += s_o[w][hh][d + 1];
      }
      if (whole) {
        const bool none = ll == 0.0f;
        const float inv = none ? 0.0f : 1.0f / ll;
        char *op = reinterpret_cast<char *>(A.o.p[r]) + (b * A.o_stride + (int64_t)(h0 + hh) * D + d) * 2;
        *reinterpret_cast<uint32_t *>(op) = none ? 0u : pack2<DT>(y0 * inv, y1 * inv);
        if (d == 0 && A.lse.p[r])
          reinterpret_cast<float *>(A.lse.p[r])[(int64_t)b * A.heads + h0 + hh] =
              none ? -__builtin_inff() : (M * A.c + log2_f(ll)) * kLn2;
      } else {
        ps[hh * D + d] = y0;
        ps[hh * D + d + 1] = y1;
        if (d == 0) {
          ps[kHeadTile * D + hh] = M;
          ps[kHeadTile * D + kHeadTile + hh] = ll;
        }
      }
    }
    if (t0 == 0 && !whole) {
      // the head's units end in another workgroup: that many partials follow
      int64_t last = (int64_t)u + nu - 1;
      int w = (int)(last * W / total);
      while (share(total, w + 1, W) <= last) w++;
      join = int4{w - w0 + 1, slot, e, ht};
    }
    __syncthreads();
    u += t1 - t0;
  }
  if (tid == 0) A.joins[w0] = join;
}

// One workgroup per (workgroup of the split, head of the tile): if that
// workgroup began a head that others went on with, join the partials.  Its
// own slot comes first, then slot 0 of each workgroup after it.
template <int DT, int ND>
__global__ __launch_bounds__(kJoinLanes) void decode_join(DecodeArgs A) {
  constexpr int D = 32 * ND, NW = kJoinLanes / 64, PL = (D + 63) / 64;
  __shared__ float s_l[NW], s_o[NW][D];
  const int w0 = (int)blockIdx.x, hh = (int)blockIdx.y;
  const int4 join = A.joins[w0];
  const int n = __builtin_amdgcn_readfirstlane(join.x);
  if (n == 0) return;
  const int e = join.z, ht = join.w;
  const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;
  const int kvh = (int)fdiv((uint32_t)ht, A.by_head_tiles), part = ht - kvh * A.head_tiles;
  const int nh = A.group - part * kHeadTile < kHeadTile ? A.group - part * kHeadTile : kHeadTile;
  if (hh >= nh) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto slot_at = [&](int i) -> const float * {
    return A.part + (int64_t)(i == 0 ? join.y : 2 * (w0 + i)) * slot_floats<D>();
  };
  // every wave finds the maximum of all partials, then sums its share
  float M = -__builtin_inff();
  for (int i = lane; i < n; i += 64) M = fmaxf(M, slot_at(i)[kHeadTile * D + hh]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, lane_xor(M, d));
  float y[PL], ll = 0.0f;
#pragma unroll
  for (int x = 0; x < PL; x++) y[x] = 0.0f;
#pragma unroll 4
  for (int i = wave; i < n; i += NW) {
    const float *s = slot_at(i);
    const float mi = s[kHeadTile * D + hh], li = s[kHeadTile * D + kHeadTile + hh];
    const float f = mi == -__builtin_inff() ? (li != li ? li : 0.0f) : exp2_f((mi - M) * A.c);
    ll += li * f;
#pragma unroll
    for (int x = 0; x < PL; x++) {
      const int d = x * 64 + lane;
      if (D % 64 == 0 || d < D) y[x] += s[hh * D + d] * f;
    }
  }
#pragma unroll
  for (int x = 0; x < PL; x++) {
    const int d = x * 64 + lane;
    if (D % 64 == 0 || d < D) s_o[wave][d] = y[x];
  }
  if (lane == 0) s_l[wave] = ll;
  __syncthreads();
  const int h = kvh * A.group + part * kHeadTile + hh;
  float L = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; w++) L += s_l[w];
  const bool none = L == 0.0f;
  const float inv = none ? 0.0f : 1.0f / L;
  for (int d = 2 * threadIdx.x; d < D; d += 2 * kJoinLanes) {
    float a = 0.0f, c = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      a += s_o[w][d];
      c += s_o[w][d + 1];
    }
    char *op = reinterpret_cast<char *>(A.o.p[r]) + (b * A.o_stride + (int64_t)h * D + d) * 2;
    *reinterpret_cast<uint32_t *>(op) = none ? 0u : pack2<DT>(a * inv, c * inv);
  }
  if (threadIdx.x == 0 && A.lse.p[r])
    reinterpret_cast<float *>(A.lse.p[r])[(int64_t)b * A.heads + h] =
        none ? -__builtin_inff() : (M * A.c + log2_f(L)) * kLn2;
}

// Workgroups of the split: one per unit that may exist, 512 at most (two of
// 4 waves on each of 256 compute units).
constexpr int kMaxSplit = 512;

int64_t unit_bound(int R, int batch, int64_t max_len, int heads, int kv_heads) {
  const int64_t tiles = (heads / kv_heads + kHeadTile - 1) / kHeadTile;
  const int64_t per = max_len > 0 ? (max_len + kUnit - 1) / kUnit : 1;
  return (int64_t)R * batch * kv_heads * tiles * per;
}
int split_of(int64_t units) { return (int)(units < kMaxSplit ? units : kMaxSplit); }

template <int DT, int ND>
int go(const Launch &L, const DecodeArgs &A, int64_t units, bool splits) {
  const int W = split_of(units);
  if (A.page_size % 8 == 0)
    hipLaunchKernelGGL((decode_split<DT, ND, true>), dim3(W), dim3(256), 0, L.stream, A);
  else
    hipLaunchKernelGGL((decode_split<DT, ND, false>), dim3(W), dim3(256), 0, L.stream, A);
  if (splits)
    hipLaunchKernelGGL((decode_join<DT, ND>), dim3(W, A.group < kHeadTile ? A.group : kHeadTile),
                       dim3(kJoinLanes), 0, L.stream, A);
  return hip_status();
}

}  // namespace

size_t attn_decode_workspace_bytes(int R, int batch, int64_t max_len, int heads, int kv_heads, int D) {
  const int64_t units = unit_bound(R, batch, max_len, heads, kv_heads);
  const size_t W = (size_t)split_of(units);
  const size_t slot = (size_t)(kHeadTile * D + 2 * kHeadTile) * sizeof(float);
  return (W * sizeof(int4) + 255) / 256 * 256 + (2 * W * slot + 255) / 256 * 256;
}

int launch_attn_decode(const Launch &L, int R, const PtrTable &q, const PtrTable &k,
                       const PtrTable &v, const PtrTable &table, const PtrTable &lens,
                       const PtrTable &seqs, const MutPtrTable &o, const MutPtrTable &lse, int batch,
                       int rows, int max_pages, int64_t num_pages, int page_size, int heads,
                       int kv_heads, int D, int64_t q_stride, int64_t o_stride, int64_t page_stride,
                       int64_t tok_stride, int64_t head_stride, float scale, int dt, void *ws) {
  const int64_t max_len = (int64_t)max_pages * page_size;
  const int64_t units = unit_bound(R, batch, max_len, heads, kv_heads);
  if (units >= (1ll << 31) || max_len > (1ll << 31) - 8 * kUnit) return COLL_ERR_UNSUPPORTED;
  DecodeArgs A{};
  A.q = q, A.k = k, A.v = v, A.table = table, A.lens = lens, A.seqs = seqs, A.o = o, A.lse = lse;
  A.q_stride = q_stride, A.o_stride = o_stride;
  A.page_stride = page_stride, A.tok_stride = tok_stride, A.head_stride = head_stride;
  A.num_pages = num_pages;
  A.batch = batch, A.rows = num_pages > 0 && max_pages > 0 ? rows : 0, A.max_pages = max_pages, A.page_size = page_size;
  A.heads = heads, A.kv_heads = kv_heads, A.group = heads / kv_heads;
  A.head_tiles = (A.group + kHeadTile - 1) / kHeadTile;
  A.entries = R * batch;
  A.by_batch = make_fastdiv((uint32_t)batch);
  A.by_page = make_fastdiv((uint32_t)page_size);
  A.by_head_tiles = make_fastdiv((uint32_t)A.head_tiles);
  A.negate = scale < 0.0f;
  A.c = __builtin_fabsf(scale) * kLog2e;
  const size_t W = (size_t)split_of(units);
  A.joins = reinterpret_cast<int4 *>(ws);
  A.part = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + (W * sizeof(int4) + 255) / 256 * 256);
  const bool splits = max_len > kUnit;
#define COLL_DECODE(DTV)                                   \
  switch (D) {                                             \
    case 64: return go<DTV, 2>(L, A, units, splits);       \
    case 96: return go<DTV, 3>(L, A, units, splits);       \
    case 128: return go<DTV, 4>(L, A, units, splits);      \
    case 192: return go<DTV, 6>(L, A, units, splits);      \
    case 256: return go<DTV, 8>(L, A, units, splits);      \
    default: return COLL_ERR_UNSUPPORTED;                  \
  }
  if (dt == COLL_BF16) { COLL_DECODE(COLL_BF16) }
  COLL_DECODE(COLL_FP16)
#undef COLL_DECODE
}

}  // namespace coll
