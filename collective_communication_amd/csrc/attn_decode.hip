// attn_decode.hip -- attention of one new token over a paged cache.
//
// Rank r, batch entry b (row seqs[b] of the page table, or row b), head h of
// kv head h / G: with the cache's first len tokens as keys and values,
//   s_t = scale * q . k_t,  m = max s_t,  p_t = exp(s_t - m),  l = sum p_t,
//   o = sum p_t v_t / l,    lse = m + log l.
// Token t lies in page table[row][t / P] at slot t % P.
//
// The keys and values are read once, and that is what bounds it.  The caches
// of all (rank, entry) pairs are one list of units of 128 tokens, cut into
// equal contiguous shares whatever the lengths: long caches are split among
// many workgroups, short ones share one.  A share is taken by one workgroup
// per head (16 query heads of one kv head), next to each other, so that
// those that run together read the neighbouring heads of the same tokens.
// A workgroup that holds all units of an entry writes its output; otherwise it
// leaves its partial (m, l, unnormalised o) in the workspace and a second
// kernel joins the partials.
//
// A wave takes 32 tokens at a time; every load covers whole rows (16 lanes a
// row), since halves of a cache line asked for one after the other cost a
// tenth of the bandwidth.  S = K Q^T has a token per row and a head per
// column; the rows are dealt so that a lane ends with 8 consecutive tokens of
// one head, which is how the B operand of O^T = V^T P^T wants them.  K gets
// into its operand's layout through a piece of LDS of the wave's own; V's
// operand holds 8 tokens of one column per lane, and a lane that has loaded
// the same few columns of 8 tokens transposes the block in registers.
#include "matrix.h"

#pragma clang fp contract(off)

namespace coll {
namespace {

constexpr int kUnit = 128;            // tokens of one unit: 32 for each of 4 waves
constexpr int kHeadTile = 16;         // query heads of one kv head that share a pass
constexpr int kMaxSplit = 512;        // workgroups of the split (more only if there are more heads)
constexpr int kJoinLanes = 512;
constexpr int kFewPartials = 8;       // joined by one wave

struct DecodeArgs {
  PtrTable q, k, v, table, lens, seqs;
  MutPtrTable o, lse;
  int64_t q_stride, o_stride;                       // elements between entries
  int64_t page_stride, tok_stride, head_stride;     // elements, both pools
  int64_t num_pages;
  int batch, rows, max_pages, page_size;
  int heads, kv_heads, group, head_tiles;           // head_tiles per kv head
  int ranks, entries;                               // entries: ranks * batch
  FastDiv by_batch, by_page, by_head_tiles, by_wide;
  float c;                                          // |scale| * log2 e
  int negate;
  float *part;                                      // partial slots, two per workgroup
  int4 *joins;                                      // per workgroup: {partials, first slot, entry, -}
  int heads_wide;                                   // kv_heads * head_tiles: workgroups per share
};

// Floats of one partial slot: the outputs, then m and l per head.
template <int D>
constexpr int slot_floats() {
  return kHeadTile * D + 2 * kHeadTile;
}

// p[r] for a lane-dependent r: a select chain over the table in scalar
// registers.  Indexed, the by-value table becomes a vector load from the
// argument segment, a round trip to memory before the loads that need it.
__device__ __forceinline__ const int32_t *pick(const PtrTable &t, int r, int ranks) {
  uint64_t v = (uint64_t)t.p[0];
  if (ranks > 1) {
#pragma unroll
    for (int q = 1; q < COLL_MAX_RANKS; q++) {
      uint64_t x = (uint64_t)t.p[q];
      COLL_SCALAR(x);
      v = r == q ? x : v;
    }
  }
  return reinterpret_cast<const int32_t *>(v);
}

// Length of entry e's cache, clipped to what its table row can hold.
__device__ __forceinline__ int entry_len(const DecodeArgs &A, int e, int *row) {
  const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;
  const int32_t *sq = pick(A.seqs, r, A.ranks);
  const int x = sq ? sq[b] : b;
  *row = x;
  if (x < 0 || x >= A.rows) return 0;
  const int64_t n = pick(A.lens, r, A.ranks)[x];
  const int64_t most = (int64_t)A.max_pages * A.page_size;
  return n < 0 ? 0 : (int)(n < most ? n : most);
}
__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + kUnit - 1) / kUnit : 1; }

// n units in `of` shares: the first `odd` of them have each + 1, the others each.
struct Shares {
  int each, odd;
  __device__ Shares(int n, int of) : each((int)((uint32_t)n / (uint32_t)of)), odd(n - each * of) {}
  __device__ int first(int w) const { return w * each + (w < odd ? w : odd); }
  __device__ int of(int u) const {                    // the share that holds unit u
    const uint32_t longer = (uint32_t)odd * (uint32_t)(each + 1);
    return (uint32_t)u < longer ? (int)((uint32_t)u / (uint32_t)(each + 1))
                                : odd + (int)(((uint32_t)u - longer) / (uint32_t)each);
  }
};

// ND consecutive dwords, non-temporal: the cache is read once (64 ragged caches
// of 583 MB: 106 us against 120 with plain loads; 128 MB: 34 against 38).
template <int ND>
__device__ __forceinline__ void ld_row(const char *p, uint32_t (&x)[ND]) {
  constexpr int N = ND % 4 == 0 ? 4 : (ND % 2 == 0 ? 2 : 1);
  typedef uint32_t piece __attribute__((ext_vector_type(N), aligned(4)));
#pragma unroll
  for (int h = 0; h < ND / N; h++) {
    const piece v = __builtin_nontemporal_load(reinterpret_cast<const piece *>(p) + h);
#pragma unroll
    for (int i = 0; i < N; i++) x[h * N + i] = v[i];
  }
}

template <int ND>
struct Chunk {                 // 32 tokens of one wave, as loaded: lane 16 g + i has
  uint32_t k[8][ND];           // ND dwords from dword i ND on of the rows of tokens
  uint32_t v[8][ND];           // 8 g + j
  uint32_t ok;                 // bit j: token 8 g + j of the chunk exists
};

template <int DT, int ND, bool P8>
__global__ __launch_bounds__(256, 2) void decode_split(DecodeArgs A) {
  constexpr int D = 32 * ND, NV = P8 ? 1 : 8;
  constexpr int kOutRow = D + 4;
  __shared__ int s_pre[257], s_len[256], s_row[256], s_wave[4];
  __shared__ float s_m[4][kHeadTile], s_l[4][kHeadTile];
  // per wave: K of a chunk, rows in operand order and padded (a stride of 4 mod
  // 32 banks), and after the last chunk the wave's outputs
  constexpr int kKeyRow = 16 * ND + 4;                // dwords
  union Own {
    uint32_t k[32 * kKeyRow];
    float o[kHeadTile][kOutRow];
  };
  __shared__ __align__(16) Own s_own[4];
  constexpr bool kQueryLds = ND > 6;
  __shared__ __align__(16) u32x4 s_q[kQueryLds ? ND : 1][64];
  // (one short cache: 8.3 -> 7.2 us)
  COLL_FETCH(A.q.p[0], A.k.p[0], A.v.p[0], A.table.p[0], A.lens.p[0], A.seqs.p[0], A.o.p[0],
             A.lse.p[0]);
  COLL_FETCH(A.q_stride, A.page_stride, A.num_pages, A.batch, A.heads, A.by_page.m, A.c, A.joins);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int w0 = (int)fdiv(blockIdx.x, A.by_wide), ht = (int)blockIdx.x - w0 * A.heads_wide;
  const int shares = (int)fdiv(gridDim.x, A.by_wide);
  const int kvh = (int)fdiv((uint32_t)ht, A.by_head_tiles), part = ht - kvh * A.head_tiles;
  const int h0 = kvh * A.group + part * kHeadTile;
  const int nh = A.group - part * kHeadTile < kHeadTile ? A.group - part * kHeadTile : kHeadTile;

  // prefix sums of the entries' units, 256 entries at a time: s_pre[i] = units
  // before entry base + i
  int base = 0;
  auto scan = [&](int carry) {
    const int e = base + tid;
    int row = 0, len = 0, mine = 0;
    if (e < A.entries) {
      len = entry_len(A, e, &row);
      mine = units_of(len);
    }
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
    s_len[tid] = len;
    s_row[tid] = row;
    if (tid == 0) s_pre[0] = carry;
    __syncthreads();
  };
  // The first round over the entries finds the total, and with it this
  // workgroup's share: at most as many shares as there are units, so that each
  // has one and the joined partials are those of consecutive shares.
  bool counting = true;
  int carry = 0, u = 0, u1 = 0, begin = 0;
  Shares S(0, 1);
  int4 join = {0, 0, 0, 0};
  for (;;) {
    scan(carry);
    const int end = __builtin_amdgcn_readfirstlane(s_pre[256]);
    if (counting) {
      if (base + 256 < A.entries) {
        carry = end;
        base += 256;
        continue;
      }
      const int W = shares < end ? shares : end;
      S = Shares(end, W);
      if (w0 < W) {
        begin = u = S.first(w0);
        u1 = S.first(w0 + 1);
      }
      counting = false;
      if (A.entries > 256) {
        carry = base = 0;
        continue;
      }
    }
    while (u < u1 && u < end) {
      // the entry that holds unit u: as many end at or before it
      int lo = 0;
#pragma unroll
      for (int x = 0; x < 4; x++) lo += __popcll(__ballot(s_pre[64 * x + lane + 1] <= u));
      lo = __builtin_amdgcn_readfirstlane(lo);
      const int e = base + lo;
      const int len = __builtin_amdgcn_readfirstlane(s_len[lo]);
      const int trow = __builtin_amdgcn_readfirstlane(s_row[lo]);
      const int nu = units_of(len);
      const int t0 = u - __builtin_amdgcn_readfirstlane(s_pre[lo]);
      const int t1 = nu < t0 + (u1 - u) ? nu : t0 + (u1 - u);
      const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;

      // Q as the B operand: column = head, 8 consecutive elements per lane; kept
      // in LDS where the registers would not hold it too
      u32x4 q[kQueryLds ? 1 : ND];
#pragma unroll
      for (int s = 0; s < ND; s++) {
        u32x4 x = {0, 0, 0, 0};
        if (i16 < nh)
          x = ld<u32x4>(reinterpret_cast<const char *>(A.q.p[r]) +
                            (b * A.q_stride + (int64_t)(h0 + i16) * D) * 2, 4 * s + g);
        if (A.negate) x = x ^ 0x80008000u;
        if constexpr (!kQueryLds) q[s] = x;
        else if (wave == 0) s_q[s][lane] = x;
      }
      if constexpr (kQueryLds) __syncthreads();
      const char *kp = reinterpret_cast<const char *>(A.k.p[r]) + (int64_t)kvh * A.head_stride * 2;
      const char *vp = reinterpret_cast<const char *>(A.v.p[r]) + (int64_t)kvh * A.head_stride * 2;
      const int32_t *pages = reinterpret_cast<const int32_t *>(A.table.p[r]) +
                             (len > 0 ? (int64_t)trow * A.max_pages : 0);

      // Pages of the lane's tokens 8 g + j of the chunk at `at`: one look-up where
      // pages are a multiple of 8 tokens.
      struct Look {
        int32_t page[NV];
      };
      auto look = [&](int at) -> Look {
        Look x;
#pragma unroll
        for (int j = 0; j < NV; j++) {
          const int t = at + 8 * g + j;
          x.page[j] = t < len ? pages[fdiv((uint32_t)t, A.by_page)] : -1;
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
        for (int j = 0; j < 8; j++) {
          const int t = at + 8 * g + j;
          const int32_t pg = x.page[P8 ? 0 : j];
          const bool ok = t < len && pg >= 0 && pg < A.num_pages;
          const int64_t row = ok ? pg * A.page_stride + slot_of(t) * A.tok_stride : 0;
          const int64_t off = row * 2 + i16 * (4 * ND);
          ch.ok |= ok ? 1u << j : 0u;
          ld_row<ND>(kp + off, ch.k[j]);
          ld_row<ND>(vp + off, ch.v[j]);
        }
        return ch;
      };

      f32x4 acc[2 * ND];
#pragma unroll
      for (int x = 0; x < 2 * ND; x++) acc[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      float m = -__builtin_inff(), l = 0.0f;

      auto compute = [&](Chunk<ND> &ch) {
        // row i of K's operand x is token 8 (i / 4) + 4 x + i % 4; a wave's LDS
        // accesses are in order, so its own piece needs no barrier
#pragma unroll
        for (int j = 0; j < 8; j++) {
          uint32_t *row = s_own[wave].k + (16 * (j >> 2) + 4 * g + (j & 3)) * kKeyRow + i16 * ND;
#pragma unroll
          for (int x = 0; x < ND; x++) row[x] = ch.k[j][x];
        }
        wave_lds_sync();
        f32x4 s[2];
#pragma unroll
        for (int x = 0; x < 2; x++) {
          s[x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int d = 0; d < ND; d++)
            s[x] = mma16<DT>(*reinterpret_cast<const u32x4 *>(s_own[wave].k + (16 * x + i16) * kKeyRow +
                                                              16 * d + 4 * g),
                           kQueryLds ? s_q[d][lane] : q[kQueryLds ? 0 : d], s[x]);
        }
        wave_lds_sync();
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

      // the wave's chunks, 128 tokens apart.  Page look-ups run one ahead; the
      // loads do not (with two workgroups on a compute unit there are enough in
      // flight: a second chunk in registers measured 1% slower).
      const int stop = len < t1 * kUnit ? len : t1 * kUnit;
      int at = t0 * kUnit + wave * 32;
      if (at < stop) {
        Look nxt = look(at);
        for (; at < stop; at += kUnit) {
          Chunk<ND> cur = load(at, nxt);
          nxt = look(at + kUnit);
          compute(cur);
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
          for (int x = 0; x < 2 * ND; x++)
            s_own[wave].o[i16][2 * ND * (4 * g + rr) + x] = acc[x][rr] * f;
      }
      __syncthreads();
      const bool whole = t0 == 0 && t1 == nu;
      const int slot = 2 * (int)blockIdx.x + (u == begin ? 0 : 1);
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
          y0 += s_own[w].o[hh][d];
          y1 += s_own[w].o[hh][d + 1];
        }
        if (whole) {
          const bool none = ll == 0.0f;
          const float inv = none ? 0.0f : 1.0f / ll;
          char *op = reinterpret_cast<char *>(A.o.p[r]) +
                     (b * A.o_stride + (int64_t)(h0 + hh) * D + d) * 2;
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
        // the entry's units end in another share: that many partials
        const int w = S.of(u + nu - 1);
        join = int4{w - w0 + 1, slot, e, 0};
      }
      __syncthreads();
      u += t1 - t0;
    }
    if (u >= u1) break;
    carry = end;
    base += 256;
  }
  if (tid == 0) A.joins[blockIdx.x] = join;
}

// One workgroup per (workgroup of the split, head of its 16): if that workgroup
// began an entry that later shares went on with, join the partials.  Its own
// slot comes first, then slot 0 of the same heads' workgroup of each share
// after it.
template <int DT, int ND>
__global__ __launch_bounds__(kJoinLanes) void decode_join(DecodeArgs A) {
  constexpr int D = 32 * ND, NW = kJoinLanes / 64;
  constexpr int LR = D / 4, RW = kJoinLanes / LR;     // lanes of a row (4 floats each), rows at a time
  __shared__ float s_f[kMaxSplit], s_m[NW], s_l[NW];
  __shared__ __align__(16) f32x4 s_o[RW][LR];
  COLL_FETCH(A.joins, A.part, A.o.p[0], A.lse.p[0], A.o_stride, A.heads, A.by_wide.m, A.c);
  const int hh = (int)blockIdx.y;
  const int4 join = A.joins[blockIdx.x];
  const int n = __builtin_amdgcn_readfirstlane(join.x);
  if (n == 0) return;
  const int e = join.z, ht = (int)(blockIdx.x - fdiv(blockIdx.x, A.by_wide) * A.heads_wide);
  const int r = (int)fdiv((uint32_t)e, A.by_batch), b = e - r * A.batch;
  const int kvh = (int)fdiv((uint32_t)ht, A.by_head_tiles), part = ht - kvh * A.head_tiles;
  const int nh = A.group - part * kHeadTile < kHeadTile ? A.group - part * kHeadTile : kHeadTile;
  if (hh >= nh) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto slot_at = [&](int i) -> const float * {
    const int slot = i == 0 ? join.y : 2 * ((int)blockIdx.x + i * A.heads_wide);
    return A.part + (int64_t)slot * slot_floats<D>();
  };
  const int h = kvh * A.group + part * kHeadTile + hh;
  char *op = reinterpret_cast<char *>(A.o.p[r]) + (b * A.o_stride + (int64_t)h * D) * 2;
  float *lp = reinterpret_cast<float *>(A.lse.p[r]);
  if (n <= kFewPartials) {
    // the common case in a batch: one wave, no barrier, all rows in flight
    if (wave > 0) return;
    float m1 = -__builtin_inff(), l1 = 0.0f;
    if (lane < n) {
      m1 = slot_at(lane)[kHeadTile * D + hh];
      l1 = slot_at(lane)[kHeadTile * D + kHeadTile + hh];
    }
    constexpr int PL = (D / 2 + 63) / 64;             // pairs of a lane
    f32x2 v[kFewPartials][PL];
#pragma unroll
    for (int i = 0; i < kFewPartials; i++)
#pragma unroll
      for (int x = 0; x < PL; x++) {
        v[i][x] = f32x2{0.0f, 0.0f};
        const int d = 2 * (x * 64 + lane);
        if (i < n && d < D) v[i][x] = *reinterpret_cast<const f32x2 *>(slot_at(i) + hh * D + d);
      }
    float M1 = m1;
#pragma unroll
    for (int d = 1; d < kFewPartials; d <<= 1) M1 = fmaxf(M1, lane_xor(M1, d));
    M1 = __shfl(M1, 0, 64);
    const float f1 = m1 == -__builtin_inff() ? (l1 != l1 ? l1 : 0.0f) : exp2_f((m1 - M1) * A.c);
    float L1 = l1 * f1;
#pragma unroll
    for (int d = 1; d < kFewPartials; d <<= 1) L1 += lane_xor(L1, d);
    L1 = __shfl(L1, 0, 64);
    const bool none = L1 == 0.0f;
    const float inv = none ? 0.0f : 1.0f / L1;
    float y[PL][2] = {};
#pragma unroll
    for (int i = 0; i < kFewPartials; i++) {
      const float w = __shfl(f1, i, 64);
      if (i < n)
#pragma unroll
        for (int x = 0; x < PL; x++) {
          y[x][0] += v[i][x][0] * w;
          y[x][1] += v[i][x][1] * w;
        }
    }
#pragma unroll
    for (int x = 0; x < PL; x++) {
      const int d = 2 * (x * 64 + lane);
      if (d < D)
        *reinterpret_cast<uint32_t *>(op + 2 * d) = none ? 0u : pack2<DT>(y[x][0] * inv, y[x][1] * inv);
    }
    if (lane == 0 && lp)
      lp[(int64_t)b * A.heads + h] = none ? -__builtin_inff() : (M1 * A.c + log2_f(L1)) * kLn2;
    return;
  }
  // a lane per partial (n <= kMaxSplit): its weight exp2((m_i - m) c)
  static_assert(kMaxSplit <= kJoinLanes, "a lane per partial");
  float mi = -__builtin_inff(), li = 0.0f;
  if (tid < n) {
    mi = slot_at(tid)[kHeadTile * D + hh];
    li = slot_at(tid)[kHeadTile * D + kHeadTile + hh];
  }
  float M = mi;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, lane_xor(M, d));
  if (lane == 0) s_m[wave] = M;
  __syncthreads();
  M = s_m[0];
#pragma unroll
  for (int w = 1; w < NW; w++) M = fmaxf(M, s_m[w]);
  const float f = mi == -__builtin_inff() ? (li != li ? li : 0.0f) : exp2_f((mi - M) * A.c);
  if (tid < n) s_f[tid] = f;
  float L = li * f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) L += lane_xor(L, d);
  if (lane == 0) s_l[wave] = L;
  __syncthreads();
  L = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; w++) L += s_l[w];
  // the rows, RW at a time and 8 of each lane's in flight
  const int rw = tid / LR, c = tid - rw * LR;
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
  if (rw < RW) {
    for (int i0 = rw; i0 < n; i0 += 8 * RW) {
      f32x4 v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int i = i0 + j * RW < n ? i0 + j * RW : i0;
        v[j] = *reinterpret_cast<const f32x4 *>(slot_at(i) + hh * D + 4 * c);
        w[j] = i0 + j * RW < n ? s_f[i] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (i0 + j * RW < n)
#pragma unroll
          for (int x = 0; x < 4; x++) y[x] += v[j][x] * w[j];
    }
    s_o[rw][c] = y;
  }
  __syncthreads();
  if (tid >= LR) return;
  y = s_o[0][tid];
#pragma unroll
  for (int i = 1; i < RW; i++)
#pragma unroll
    for (int x = 0; x < 4; x++) y[x] += s_o[i][tid][x];
  const bool none = L == 0.0f;
  const float inv = none ? 0.0f : 1.0f / L;
  u32x2 w2 = {pack2<DT>(y[0] * inv, y[1] * inv), pack2<DT>(y[2] * inv, y[3] * inv)};
  if (none) w2 = u32x2{0u, 0u};
  st<u32x2>(op, tid, w2);
  if (tid == 0 && lp)
    lp[(int64_t)b * A.heads + h] = none ? -__builtin_inff() : (M * A.c + log2_f(L)) * kLn2;
}

// Workgroups of the split: 512 (two of 4 waves on each of 256 compute units),
// in whole shares of one per 16 heads, and no more shares than there may be
// units.

int64_t unit_bound(int R, int batch, int64_t max_len) {
  const int64_t per = max_len > 0 ? (max_len + kUnit - 1) / kUnit : 1;
  return (int64_t)R * batch * per;
}
int64_t wide_of(int heads, int kv_heads) {
  return (int64_t)kv_heads * ((heads / kv_heads + kHeadTile - 1) / kHeadTile);
}
int64_t split_of(int64_t units, int64_t wide) {
  const int64_t most = wide < kMaxSplit ? kMaxSplit / wide : 1;
  return wide * (units < most ? units : most);
}

template <int DT, int ND>
int go(const Launch &L, const DecodeArgs &A, int W, bool splits) {
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
  const size_t W = (size_t)split_of(unit_bound(R, batch, max_len), wide_of(heads, kv_heads));
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
  const int64_t units = unit_bound(R, batch, max_len), wide = wide_of(heads, kv_heads);
  if (units >= (1ll << 31) || max_len > (1ll << 31) - 8 * kUnit) return COLL_ERR_UNSUPPORTED;
  DecodeArgs A{};
  A.q = q, A.k = k, A.v = v, A.table = table, A.lens = lens, A.seqs = seqs, A.o = o, A.lse = lse;
  A.q_stride = q_stride, A.o_stride = o_stride;
  A.page_stride = page_stride, A.tok_stride = tok_stride, A.head_stride = head_stride;
  A.num_pages = num_pages;
  A.batch = batch, A.rows = num_pages > 0 && max_pages > 0 ? rows : 0;
  A.max_pages = max_pages, A.page_size = page_size;
  A.heads = heads, A.kv_heads = kv_heads, A.group = heads / kv_heads;
  A.head_tiles = (A.group + kHeadTile - 1) / kHeadTile;
  A.ranks = R, A.entries = R * batch;
  A.by_batch = make_fastdiv((uint32_t)batch);
  A.by_page = make_fastdiv((uint32_t)page_size);
  A.by_head_tiles = make_fastdiv((uint32_t)A.head_tiles);
  A.negate = scale < 0.0f;
  A.c = __builtin_fabsf(scale) * kLog2e;
  A.heads_wide = (int)wide;
  A.by_wide = make_fastdiv((uint32_t)wide);
  const size_t W = (size_t)split_of(units, wide);
  A.joins = reinterpret_cast<int4 *>(ws);
  A.part = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) +
                                     (W * sizeof(int4) + 255) / 256 * 256);
  const bool splits = max_len > kUnit;
#define COLL_DECODE(DTV)                                   \
  switch (D) {                                             \
    case 64: return go<DTV, 2>(L, A, (int)W, splits);       \
    case 96: return go<DTV, 3>(L, A, (int)W, splits);       \
    case 128: return go<DTV, 4>(L, A, (int)W, splits);      \
    case 192: return go<DTV, 6>(L, A, (int)W, splits);      \
    case 256: return go<DTV, 8>(L, A, (int)W, splits);      \
    default: return COLL_ERR_UNSUPPORTED;                  \
  }
  if (dt == COLL_BF16) { COLL_DECODE(COLL_BF16) }
  COLL_DECODE(COLL_FP16)
#undef COLL_DECODE
}

}  // namespace coll
