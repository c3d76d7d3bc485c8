// attn_prompt.hip -- attention over packed prompts.
//
// Rank r, sequence b with nq query rows and nk key rows, head h of kv head
// h / (H / KV); key j is visible to query i when j <= i + diag (causal) or
// always:
//   s_ij = scale * q_i . k_j,   m_i = max_j s_ij,   p_ij = exp(s_ij - m_i),
//   l_i = sum_j p_ij,   o_i = sum_j p_ij v_j / l_i,   lse_i = m_i + log l_i,
// over the visible j.  One pass over the keys in tiles keeps the running m_i
// and l_i and the unnormalised o_i, which is multiplied by
// exp(m_old - m_new) when the maximum grows.
//
// A workgroup owns NW * 32 query rows of one head, each wave 32 of them.  The
// wave computes S^T = K Q^T (rows = keys, columns = queries), so a lane holds
// keys of one query: the row statistics are in-lane reductions plus one
// exchange between the two halves of the wave, and p, rounded to the input
// type, is already laid out as the B operand of O^T = V^T P^T.  The fixed
// permutation of the keys inside 16 that this implies is undone by where V
// is read: the transposing LDS read takes 4 consecutive keys at a time.
// K and V tiles are staged through registers into two LDS buffers (one
// barrier per tile).
//
// At 128 elements a head it runs at 1000 to 1060 TFLOP/s (8192 tokens x 32 heads:
// 545 us causal, 1035 us with all keys), four fifths of what a large library
// product reaches: matrix pipe 50%, vector pipe 41% and LDS 31% of the cycles.
#include "matrix.h"

#pragma clang fp contract(off)

namespace coll {
namespace {

// One call's arguments, by value (1.2 KiB).
struct PromptArgs {
  PtrTable q, k, v, q_starts, k_starts, diag;
  MutPtrTable o, lse;
  int64_t q_stride, k_stride, v_stride, o_stride;   // elements between tokens
  int64_t q_rows, k_rows;                           // rows the buffers hold
  int nseq, heads, kv_heads, causal;
  uint32_t tiles;                                   // tile slots per (rank, head)
  FastDiv by_group, by_heads, by_tiles;
  float c;                                          // |scale| * log2 e
  int negate;                                       // scale < 0
};

// Where a workgroup's tile lies.
struct TileAt {
  int64_t q0, k0;        // first rows of the sequence
  int32_t nq, nk, diag;  // its lengths; key j visible to query i when j <= i + diag
  int32_t first;         // first query row of the tile in the sequence
  bool any;
};

// Length of rows [a, b) of a buffer of n rows (0 when they do not all exist).
__device__ __forceinline__ int32_t span(int64_t a, int64_t b, int64_t n) {
  return (a < 0 || b <= a || b > n) ? 0 : (int32_t)(b - a);
}

// The sequence that holds tile slot `slot` of rank r, scanned by every wave, 64
// sequences at a time.  Causal tiles get longer towards a sequence's end, and
// the last workgroups to start should be short: 2 to 16 sequences of up to 64
// tiles are taken level by level, every sequence's 64th tile first (8 packed
// prompts of 1 to 2048 tokens: 136 -> 125 us, 4 of 512: 28 -> 24); others from
// the last tile down (a look-up for each sequence, it costs more than it gives
// for 32 sequences of 512 or 256 tokens: 173 and 75 us against 160 and 65).
// Sums over the lanes go by lane reads and ballots: a shuffle is a trip to LDS,
// and this is before a workgroup's first load.
template <int BQ>
__device__ __forceinline__ TileAt find_tile(const PromptArgs &A, int r, uint32_t slot) {
  const int32_t *qs = reinterpret_cast<const int32_t *>(A.q_starts.p[r]);
  const int32_t *ks = reinterpret_cast<const int32_t *>(A.k_starts.p[r]);
  const int32_t *dg = reinterpret_cast<const int32_t *>(A.diag.p[r]);
  const int lane = threadIdx.x & 63;
  const uint32_t tile = A.tiles - 1 - slot;
  const uint64_t to_me = (2ull << lane) - 1;          // the lanes up to this one
  TileAt t{};
  uint32_t before = 0;
  for (int base = 0; base < A.nseq; base += 64) {
    const int b = base + lane;
    int32_t a0 = 0, a1 = 0, c0 = 0, c1 = 0, d = 0;
    if (b < A.nseq) {
      a0 = qs[b];
      a1 = qs[b + 1];
      c0 = ks[b];
      c1 = ks[b + 1];
      if (dg) d = dg[b];
    }
    const int32_t nq = span(a0, a1, A.q_rows);
    const uint32_t mine = ((uint32_t)nq + BQ - 1) / BQ;
    int l = -1;
    uint32_t index = 0;
    if (A.nseq > 1 && A.nseq <= 16 && !__ballot(mine > 64)) {
      uint32_t high = 0;                              // tiles of level `lane` and above
      for (int x = 0; x < A.nseq; x++) {
        const int m = __builtin_amdgcn_readlane((int)mine, x);
        high += m > lane ? m - lane : 0;
      }
      const uint64_t above = __ballot(high > slot);   // the levels up to the slot's
      if (above) {
        const int level = 63 - __builtin_clzll(above);
        const uint32_t rest = slot - (level < 63 ? (uint32_t)__builtin_amdgcn_readlane((int)high, level + 1) : 0);
        const uint64_t in = __ballot(mine > (uint32_t)level);
        l = __builtin_ctzll(__ballot(mine > (uint32_t)level && (uint32_t)__popcll(in & (to_me >> 1)) == rest));
        index = (uint32_t)level;
      }
    } else {
      uint32_t upto = 0;
      for (int x = 0; __ballot(mine >> x != 0); x++)
        upto += (uint32_t)__popcll(__ballot((mine >> x) & 1) & to_me) << x;
      const uint64_t hit = __ballot(before + upto > tile);
      if (hit) {
        l = __builtin_ctzll(hit);
        index = tile - before - (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), l);
      }
      before += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    if (l >= 0) {
      t.any = true;
      t.first = (int32_t)(index * BQ);
      t.nq = __builtin_amdgcn_readlane(nq, l);
      t.q0 = __builtin_amdgcn_readlane(a0, l);
      t.k0 = __builtin_amdgcn_readlane(c0, l);
      t.nk = span(t.k0, __builtin_amdgcn_readlane(c1, l), A.k_rows);
      t.diag = dg ? __builtin_amdgcn_readlane(d, l) : t.nk - t.nq;
      return t;
    }
  }
  return t;
}

// Waves that share 32 query rows.  Beyond 128 elements the registers of a wave
// that holds whole rows would leave a SIMD one wave; two waves then compute the
// same scores and weights, and each half of the output's columns (4096 causal
// tokens x 16 heads x 256: 251 us against 390, x 192: 189 against 220; by now
// 212 and 162).
template <int D>
constexpr int kSplit = D > 128 ? 2 : 1;

constexpr int BN = 64;                 // keys of a tile

// A tile's keys in LDS, two tiles of K and two of V.  The rows are padded so that
// neither the row reads of K (8 lanes, 16 bytes of 8 consecutive rows: a
// stride of 4 mod 32 banks) nor the column reads of V (32 lanes, 64 bytes of
// 4 consecutive rows: 16 or 48 mod 64 banks) meet bank conflicts; a lane's
// address is then one base and a constant.
template <int D>
struct Tiles {
  static constexpr int kRowK = D + 8, kRowV = D % 64 == 0 ? D + 32 : D;   // elements
  uint16_t k[2][BN * kRowK];
  uint16_t v[2][BN * kRowV];
};

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64, D == 64 ? 3 : 2) void prompt_tiles(PromptArgs A) {
  constexpr int SP = kSplit<D>, BQ = NW / SP * 32, CH = D / 8, NT = NW * 64;
  constexpr int NCH = (BN * CH + NT - 1) / NT;        // chunks a thread stages of K and of V
  constexpr bool kWhole = BN * CH % NT == 0;
  constexpr int DK = D / 16, DV = D / 32 / SP, KT = BN / 32;
  using TL = Tiles<D>;
  __shared__ __align__(16) TL s_t;
  __shared__ int s_bad[2];                            // 1 + index of a tile whose V is not finite
  // heads vary fastest, and in steps that keep the heads of one kv head on
  // one XCD (workgroups go round the 8 XCDs); tiles from the last one down,
  // since causal tiles get longer
  const uint32_t H = (uint32_t)A.heads;
  const uint32_t th = fdiv(blockIdx.x, A.by_heads);
  uint32_t h = blockIdx.x - th * H;
  if (H % 8 == 0) h = (h & 7) * (H / 8) + (h >> 3);
  const int r = (int)fdiv(th, A.by_tiles);
  const uint32_t tile = A.tiles - 1 - (th - (uint32_t)r * A.tiles);
  // (8192 x 32 heads x 128: 553 -> 545 us)
  COLL_FETCH(A.q_starts.p[r], A.k_starts.p[r], A.diag.p[r], A.q.p[r], A.k.p[r], A.v.p[r], A.nseq, A.q_rows);
  COLL_FETCH(A.k_rows, A.q_stride, A.k_stride, A.v_stride, A.by_group.m, A.c, A.negate, A.causal);
  COLL_FETCH(A.o.p[r], A.lse.p[r], A.o_stride, A.heads, A.kv_heads, A.tiles, A.by_heads.m, A.by_tiles.m);
  const TileAt t = find_tile<BQ>(A, r, A.tiles - 1 - tile);
  if (!t.any) return;
  const int kvh = (int)fdiv(h, A.by_group);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, g = lane >> 5;

  // keys visible to query row i of the sequence: the first limit(i)
  auto limit = [&](int i) -> int {
    if (!A.causal) return t.nk;
    const int64_t x = (int64_t)i + t.diag + 1;
    return x < 0 ? 0 : (x > t.nk ? t.nk : (int)x);
  };
  const int last_row = (t.first + BQ < t.nq ? t.first + BQ : t.nq) - 1;
  const int n_block = limit(last_row);                // keys any row of the tile sees
  const int see_all = limit(t.first);                 // keys every row of the tile sees
  const int row0 = t.first + wave / SP * 32;          // the wave's rows
  const int d0 = wave % SP * DV;                      // and its first 32 columns of V
  const int row = row0 + col;
  const int n_wave = row0 <= last_row ? limit(row0 + 31 < last_row ? row0 + 31 : last_row) : 0;
  const int lim = limit(row);

  // Q as the B operand: column = query, 8 consecutive elements per lane
  u32x4 q[DK];
  {
    // (a column past the last row repeats that row and is not stored)
    const char *qp = reinterpret_cast<const char *>(A.q.p[r]) +
                     ((t.q0 + (row < last_row ? row : last_row)) * A.q_stride + (int64_t)h * D) * 2;
    const uint32_t sign = A.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < DK; s++) q[s] = ld<u32x4>(qp, 2 * s + g) ^ sign;
  }

  // a thread's chunks of a tile: 16 bytes at chunk_of of key key_of (whole steps
  // from one to the next where the threads take whole keys: one address)
  constexpr bool kSteps = NT % CH == 0;
  auto key_of = [](int t, int i) -> int { return kSteps ? t / CH + i * (NT / CH) : (t + i * NT) / CH; };
  auto chunk_of = [](int t, int i) -> int { return kSteps ? t % CH : (t + i * NT) % CH; };
  u32x4 held[NCH];
  const char *kp = reinterpret_cast<const char *>(A.k.p[r]) + (t.k0 * A.k_stride + (int64_t)kvh * D) * 2;
  const char *vp = reinterpret_cast<const char *>(A.v.p[r]) + (t.k0 * A.v_stride + (int64_t)kvh * D) * 2;
  // Their places in a tile of `rows` keys.  A key behind the last one stands for
  // the last: its score is masked, and a value that is not finite marks the
  // tile in any case.  So no load needs a branch.
  auto places = [&](uint32_t (&at)[NCH], int64_t stride, int rows) {
    int me = tid;
    COLL_FRESH(me);
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int kr = key_of(me, i), last = (rows < BN ? rows : BN) - 1;
      at[i] = (uint32_t)(kr < last ? kr : last) * (uint32_t)(2 * stride) + 16 * chunk_of(me, i);
    }
  };
  uint32_t k_at[NCH], v_at[NCH];
  auto load = [&](const char *src, int64_t stride, uint32_t (&at)[NCH], int kt) {
    const int rows = t.nk - kt * BN;
    if (rows < BN) places(at, stride, rows);
    const char *tile = src + (int64_t)kt * BN * stride * 2;
#pragma unroll
    for (int i = 0; i < NCH; i++) held[i] = *reinterpret_cast<const u32x4 *>(tile + at[i]);
  };
  auto store = [&](uint16_t *tile, int row) {
#pragma unroll
    for (int i = 0; i < NCH; i++)
      if (kWhole || key_of(tid, i) < BN)
        *reinterpret_cast<u32x4 *>(tile + key_of(tid, i) * row + 8 * chunk_of(tid, i)) = held[i];
  };
  auto store_k = [&](int kt) { store(s_t.k[kt & 1], TL::kRowK); };
  auto store_v = [&](int kt) {
    store(s_t.v[kt & 1], TL::kRowV);
    // a value that is not finite at a key some row must not see would reach
    // that row as 0 * inf: such a tile is marked for the careful product
    if ((kt + 1) * BN > see_all) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < NCH; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) bad = bad || pair_not_finite<DT>(held[i][e]);
      if (bad) s_bad[kt & 1] = kt + 1;
    }
  };

  f32x16 acc[DV];
#pragma unroll
  for (int d = 0; d < DV; d++)
#pragma unroll
    for (int e = 0; e < 16; e++) acc[d][e] = 0.0f;
  // m: running maximum, in the units of the unscaled scores; l: this lane's
  // part of the sum, in two
  float m = -__builtin_inff(), l0 = 0.0f, l1 = 0.0f;

  // S^T of 32 keys of a tile
  const int kat = col * TL::kRowK + 8 * g;
  auto scores = [&](int kt, int half) -> f32x16 {
    const uint16_t *base = s_t.k[kt & 1] + kat + 32 * half * TL::kRowK;
    f32x16 s;
#pragma unroll
    for (int e = 0; e < 16; e++) s[e] = 0.0f;
#pragma unroll
    for (int d = 0; d < DK; d++) s = mma32<DT>(*reinterpret_cast<const u32x4 *>(base + 16 * d), q[d], s);
    return s;
  };
  // V^T as the A operand of rows 32 d.., keys 16 s ..: two transposing reads,
  // keys 16 s + 4 g + 0..3 and those 8 further on
  const int vat = (4 * g + ((lane & 15) >> 2)) * TL::kRowV + (lane & 16) + 4 * (lane & 3) + 32 * d0;
  auto v_frag = [&](int kt, int d, int s) -> u32x4 {
    const uint16_t *p = s_t.v[kt & 1] + vat + 16 * s * TL::kRowV + 32 * d;
    const u32x2 x = lds_tr16(p), y = lds_tr16(p + 8 * TL::kRowV);
    u32x4 w = {x[0], x[1], y[0], y[1]};
    return w;
  };
  // The maximum is raised only when it grows by more than 8 / c (p stays below
  // 2^8), so most tiles rescale nothing.
  auto raise = [&](const f32x16 (&s)[KT]) {
    float a = s[0][0], b = s[0][1];
#pragma unroll
    for (int x = 0; x < KT; x++)
#pragma unroll
      for (int e = x == 0 ? 2 : 0; e < 16; e += 2) {
        a = fmaxf(a, s[x][e]);
        b = fmaxf(b, s[x][e + 1]);
      }
    const float mt = max_halves(fmaxf(a, b));
    if (__ballot((mt - m) * A.c > 8.0f)) {
      const float mn = fmaxf(m, mt);
      const float f = mn == -__builtin_inff() ? 1.0f : exp2_f((m - mn) * A.c);
      m = mn;
      l0 *= f;
      l1 *= f;
#pragma unroll
      for (int d = 0; d < DV; d++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[d][e] *= f;
    }
  };
  // the weights of 32 keys, as the B operands of two products of 16
  auto weights = [&](const f32x16 &s, u32x4 (&p)[2]) {
    const float mc = m == -__builtin_inff() ? 0.0f : m * A.c;
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float y0 = exp2_f(__builtin_fmaf(s[e], A.c, -mc));
      const float y1 = exp2_f(__builtin_fmaf(s[e + 1], A.c, -mc));
      l0 += y0;
      l1 += y1;
      p[e >> 3][(e & 7) >> 1] = pack2<DT>(y0, y1);
    }
  };

  const int ntiles = (n_block + BN - 1) / BN;
  const int nfull = see_all / BN < ntiles ? see_all / BN : ntiles;   // tiles that need no mask
  if (tid < 2) s_bad[tid] = 0;
  if (ntiles > 0) {
    // the first tiles of K and V and the second of K, all in flight together
    places(k_at, A.k_stride, BN);
    places(v_at, A.v_stride, BN);
    u32x4 first[2][NCH];
    load(kp, A.k_stride, k_at, 0);
#pragma unroll
    for (int i = 0; i < NCH; i++) first[0][i] = held[i];
    load(vp, A.v_stride, v_at, 0);
#pragma unroll
    for (int i = 0; i < NCH; i++) first[1][i] = held[i];
    if (ntiles > 1) load(kp, A.k_stride, k_at, 1);
    __syncthreads();
    if (ntiles > 1) store_k(1);
#pragma unroll
    for (int i = 0; i < NCH; i++) held[i] = first[0][i];
    store_k(0);
#pragma unroll
    for (int i = 0; i < NCH; i++) held[i] = first[1][i];
    store_v(0);
  }
  __syncthreads();

  // The scores of the next tile are computed with the weights of this one, so
  // that a wave has matrix work while it computes exponentials: K is staged
  // a tile further ahead than V.  One barrier per tile: what is written was
  // last read before the previous one.
  f32x16 s[KT];
  const bool busy = n_wave > 0;
  if (busy)
#pragma unroll
    for (int x = 0; x < KT; x++) s[x] = scores(0, x);
  __syncthreads();
  // the second four waves go first, so that the two of a SIMD do not compute
  // exponentials at the same time (8192 x 32 heads x 128: 574 -> 567 us)
  if (wave & 4) __builtin_amdgcn_s_setprio(1);
  int kt = 0;
  for (; kt < nfull; kt++) {
    // K's tile passes through the staging registers in the first half, V's in
    // the last
    const bool more_k = kt + 2 < ntiles, more_v = kt + 1 < ntiles;
    if (more_k) load(kp, A.k_stride, k_at, kt + 2);
    if (busy) raise(s);
#pragma unroll
    for (int x = 0; x < KT; x++) {
      // (outside of any branch on busy: a wait for a load that only one side has
      // in flight would be paid on both; 8192 x 32 heads x 128: 560 -> 545 us)
      if (x == KT - 1) {
        if (more_k) store_k(kt + 2);
        if (more_v) load(vp, A.v_stride, v_at, kt + 1);
      }
      if (!busy) continue;
      u32x4 p[2];
      weights(s[x], p);
      s[x] = scores(kt + 1, x);                       // of an old tile after the last one: not used
#pragma unroll
      for (int y = 0; y < 2; y++)
#pragma unroll
        for (int d = 0; d < DV; d++) acc[d] = mma32<DT>(v_frag(kt, d, 2 * x + y), p[y], acc[d]);
    }
    if (more_v) store_v(kt + 1);
    __syncthreads();
  }
  for (; kt < ntiles; kt++) {                         // tiles on the diagonal and the last one
    const bool more_k = kt + 2 < ntiles, more_v = kt + 1 < ntiles, sees = kt * BN < n_wave;
    if (more_k) load(kp, A.k_stride, k_at, kt + 2);
    if (sees) {
      const int left = lim - kt * BN - 4 * g;
#pragma unroll
      for (int x = 0; x < KT; x++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          s[x][e] = 32 * x + (e & 3) + 8 * (e >> 2) < left ? s[x][e] : -__builtin_inff();
      raise(s);
    }
    if (more_k) store_k(kt + 2);
    if (more_v) load(vp, A.v_stride, v_at, kt + 1);
    if (sees) {
      const bool bad = s_bad[kt & 1] == kt + 1;
#pragma unroll
      for (int x = 0; x < KT; x++) {
        const int key0 = kt * BN + 32 * x;
        if (key0 >= n_wave) break;
        u32x4 p[2];
        weights(s[x], p);
        if (!bad) {
#pragma unroll
          for (int y = 0; y < 2; y++)
#pragma unroll
            for (int d = 0; d < DV; d++) acc[d] = mma32<DT>(v_frag(kt, d, 2 * x + y), p[y], acc[d]);
          continue;
        }
        // key by key, each added only where it is visible
        int half = g;
        COLL_FRESH(half);
        for (int j = 0; j < 32; j++) {
          const int jj = j & 15;
          // the key's place in the operands: half of the wave and element
          const int gj = (jj >> 2) & 1, ej = (jj & 3) + 4 * (jj >> 3);
          u32x4 keep;
#pragma unroll
          for (int w = 0; w < 4; w++)
            keep[w] = (half == gj && ej >> 1 == w) ? (ej & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
          const u32x4 pj = (j < 16 ? p[0] : p[1]) & keep;
          const bool vis = key0 + j < lim;
#pragma unroll
          for (int d = 0; d < DV; d++) {
            f32x16 one;
#pragma unroll
            for (int e = 0; e < 16; e++) one[e] = 0.0f;
            one = mma32<DT>(v_frag(kt, d, 2 * x + (j >> 4)) & keep, pj, one);
#pragma unroll
            for (int e = 0; e < 16; e++) acc[d][e] += vis ? one[e] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < KT; x++)
        if ((kt + 1) * BN + 32 * x < n_wave) s[x] = scores(kt + 1, x);
    }
    if (more_v) store_v(kt + 1);
    __syncthreads();
  }
  float l = l0 + l1;

  // o = acc / l, lse = m + log l; a row that saw nothing gets 0 and -inf
  l += lane_xor(l, 32);
  if (row > last_row) return;
  const bool none = l == 0.0f;
  const float inv = none ? 0.0f : 1.0f / l;
  char *op = reinterpret_cast<char *>(A.o.p[r]) + ((t.q0 + row) * A.o_stride + (int64_t)h * D) * 2;
#pragma unroll
  for (int d = 0; d < DV; d++)
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      float y[4];
#pragma unroll
      for (int w = 0; w < 4; w++) y[w] = none ? 0.0f : acc[d][e + w] * inv;
      u32x2 w2 = {pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
      st<u32x2>(op, (32 * (d0 + d) + 2 * e + 4 * g) / 4, w2);
    }
  if (A.lse.p[r] && g == 0 && d0 == 0)
    reinterpret_cast<float *>(A.lse.p[r])[(t.q0 + row) * A.heads + h] =
        none ? -__builtin_inff() : (m * A.c + log2_f(l)) * kLn2;
}

template <int DT, int D>
int go(const Launch &L, int R, PromptArgs &A, int64_t q_rows) {
  // 8 waves share a staged tile among 256 rows when the sequences are long (4096
  // keys and more, on average) and give every compute unit two workgroups' work;
  // otherwise 4 waves and 128 rows, two workgroups at a time on a compute unit,
  // so that one computes while the other begins, ends or waits at the diagonal
  // (32 heads x 128: 8192 tokens 555 against 568 us; 8 x 2048: 375 against 363; 8 x
  // 1024: 132 against 114; 32 x 256: 95 against 71; 4096 x 32 heads x 96: 130
  // against 133).  Heads of 64 leave room for three workgroups of 4 waves (8192 x
  // 32 heads x 64: 337 against 346 us), heads beyond 128 for one.
  const uint64_t tiles8 = (uint64_t)(q_rows + 255) / 256 + A.nseq;
  const bool wide = (D == 96 || D == 128) && A.k_rows / A.nseq >= 4096 &&
                    tiles8 * A.heads * R >= 2ull * L.num_cus;
  const uint64_t tiles = wide ? tiles8 : (uint64_t)(q_rows + 127) / 128 + A.nseq;
  const uint64_t groups = tiles * A.heads * R;
  if (groups * (wide || D > 128 ? 512 : 256) > kMaxThreads) return COLL_ERR_UNSUPPORTED;
  A.tiles = (uint32_t)tiles;
  A.by_tiles = make_fastdiv(A.tiles);
  // D = 96 and 128: both forms; 64: 4 waves; 192 and 256: 8 waves, two to a row
  if constexpr (D > 64) {
    if (wide || D > 128) {
      hipLaunchKernelGGL((prompt_tiles<DT, D, 8>), dim3((unsigned)groups), dim3(512), 0, L.stream, A);
      return hip_status();
    }
  }
  if constexpr (D <= 128)
    hipLaunchKernelGGL((prompt_tiles<DT, D, 4>), dim3((unsigned)groups), dim3(256), 0, L.stream, A);
  return hip_status();
}

}  // namespace

int launch_attn_prompt(const Launch &L, int R, const PtrTable &q, const PtrTable &k,
                       const PtrTable &v, const MutPtrTable &o, const MutPtrTable &lse,
                       const PtrTable &q_starts, const PtrTable &k_starts, const PtrTable &diag,
                       int nseq, int64_t q_rows, int64_t k_rows, int heads, int kv_heads, int D,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t o_stride,
                       int causal, float scale, int dt) {
  PromptArgs A{};
  A.q = q, A.k = k, A.v = v, A.o = o, A.lse = lse;
  A.q_starts = q_starts, A.k_starts = k_starts, A.diag = diag;
  A.q_stride = q_stride, A.k_stride = k_stride, A.v_stride = v_stride, A.o_stride = o_stride;
  A.q_rows = q_rows, A.k_rows = k_rows;
  A.nseq = nseq, A.heads = heads, A.kv_heads = kv_heads, A.causal = causal;
  A.by_group = make_fastdiv((uint32_t)(heads / kv_heads));
  A.by_heads = make_fastdiv((uint32_t)heads);
  A.negate = scale < 0.0f;
  A.c = __builtin_fabsf(scale) * kLog2e;
#define COLL_PROMPT(DTV)                                              \
  switch (D) {                                                        \
    case 64: return go<DTV, 64>(L, R, A, q_rows);                 \
    case 96: return go<DTV, 96>(L, R, A, q_rows);                 \
    case 128: return go<DTV, 128>(L, R, A, q_rows);               \
    case 192: return go<DTV, 192>(L, R, A, q_rows);               \
    case 256: return go<DTV, 256>(L, R, A, q_rows);               \
    default: return COLL_ERR_UNSUPPORTED;                             \
  }
  if (dt == COLL_BF16) { COLL_PROMPT(COLL_BF16) }
  COLL_PROMPT(COLL_FP16)
#undef COLL_PROMPT
}

}  // namespace coll
