// pages.hip -- the pages of a key-value cache: allocation, fork, release and
// compaction on the device, the copies they ask for, and writing new tokens.
//
// State (device int32): table[rows][width], the page of each block of
// page_size tokens of a sequence or -1; lens[rows], tokens a sequence holds;
// ref[num_pages], how many table entries name a page, 0 for a free one.  All
// decisions are made on the device from this state, so no call needs a host
// synchronisation, and all results are determined by it: fresh pages are the
// lowest free ones in the order the entries are listed.
//
// The bookkeeping is latency, not bandwidth: one workgroup of 1024 lanes does
// what needs a view of all entries or of all of ref (scans of 4 KiB at a
// time), and a grid does what is independent per entry or per table row.
#include "coll_internal.h"

namespace coll {
namespace {

constexpr int kOne = kKvMaxEntries;        // lanes of the single-workgroup kernels
constexpr int kOneWaves = kOne / 64;
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct PageState {
  int32_t *table, *lens, *ref;
  int rows, width, num_pages, page_size;
  FastDiv by_page;
};

// a + b of numbers from 0 to INT32_MAX, at most INT32_MAX: 1024 entries may ask
// for more pages together than 32 bits hold.
__device__ __forceinline__ int add_sat(int a, int b) {
  const uint32_t s = (uint32_t)a + (uint32_t)b;
  return (int)(s < 0x7FFFFFFFu ? s : 0x7FFFFFFFu);
}

// Inclusive prefix sum over the workgroup's lanes, of numbers from 0 on; *total:
// the whole sum.  Sums stay at INT32_MAX (more than there can be pages).
__device__ __forceinline__ int scan_block(int x, int *s_wave, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(upto, d, 64);
    if (lane >= d) upto = add_sat(upto, y);
  }
  __syncthreads();
  if (lane == 63) s_wave[wave] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kOneWaves; w++) {
    const int y = s_wave[w];
    before = add_sat(before, w < wave ? y : 0);
    all = add_sat(all, y);
  }
  *total = all;
  return add_sat(before, upto);
}

__device__ __forceinline__ int pages_of(const PageState &S, int tokens) {
  return (int)fdiv((uint32_t)(tokens + S.page_size - 1), S.by_page);
}

// Four consecutive refs of the scan, 1 (in use) past the end.
__device__ __forceinline__ i32x4 refs4(const PageState &S, int i) {
  i32x4 x;
#pragma unroll
  for (int j = 0; j < 4; j++) x[j] = i + j < S.num_pages ? S.ref[i + j] : 1;
  return x;
}

// Allocation for extend and fork.  Entry i (lane i) wants need pages; served
// are the entries whose running total, in list order, fits the free pages.
// The first 4096 refs are read once, by the caller, before anything depends
// on them.
struct Demand {
  int upto;       // running total up to and including the entry
  int free;       // free pages
};
__device__ __forceinline__ int zeros(i32x4 x) {
  return (x[0] == 0) + (x[1] == 0) + (x[2] == 0) + (x[3] == 0);
}
__device__ __forceinline__ Demand demand(const PageState &S, i32x4 refs0, int need, int *s_wave) {
  Demand d;
  int total;
  d.upto = scan_block(need, s_wave, &total);
  int n = zeros(refs0);
  for (int i = 4 * (kOne + (int)threadIdx.x); i < S.num_pages; i += 4 * kOne) n += zeros(refs4(S, i));
  scan_block(n, s_wave, &d.free);
  return d;
}
// give(k, page) for the k-th free page, k < want
template <class Give>
__device__ __forceinline__ void take_free(const PageState &S, i32x4 refs0, int want, int *s_wave,
                                          Give give) {
  int done = 0;
  for (int base = 0; base < S.num_pages && done < want; base += 4 * kOne) {
    const int i = base + 4 * (int)threadIdx.x;
    const i32x4 x = base == 0 ? refs0 : refs4(S, i);
    const int mine = zeros(x);
    int total;
    int k = done + scan_block(mine, s_wave, &total) - mine;
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (x[j] == 0) {
        if (k < want) give(k, i + j);
        k++;
      }
    done += total;
  }
}

// First entry whose running total exceeds k.
__device__ __forceinline__ int owner_of(const int *upto, int n, int k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] > k) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The first entry that names each row, in an LDS hash of twice the entries'
// number (open addressing; an entry's probe ends at its row or a free place,
// and there always is one).
constexpr int kHash = 2 * kOne;
struct RowHash {
  int row[kHash], first[kHash];
};
__device__ __forceinline__ void hash_clear(RowHash &T) {
  for (int x = threadIdx.x; x < kHash; x += kOne) {
    T.row[x] = -1;
    T.first[x] = kOne;
  }
}
__device__ __forceinline__ int hash_add(RowHash &T, int row, int i) {     // row >= 0
  int x = (int)(((uint32_t)row * 2654435761u) >> 21);
  for (;;) {
    const int had = atomicCAS(&T.row[x], -1, row);
    if (had == -1 || had == row) break;
    x = (x + 1) & (kHash - 1);
  }
  atomicMin(&T.first[x], i);
  return x;
}
static_assert(kHash == 1 << (32 - 21), "the hash takes the top bits");

__global__ __launch_bounds__(kOne) void extend_rows(PageState S, const int32_t *seqs,
                                                    const int32_t *add, int n, int32_t *status) {
  __shared__ int s_wave[kOneWaves], s_row[kOne], s_upto[kOne], s_have[kOne];
  __shared__ RowHash s_hash;
  __shared__ int s_want;
  const int i = threadIdx.x;
  const int row = i < n ? seqs[i] : -1, more = i < n ? add[i] : 0;
  const i32x4 refs0 = refs4(S, 4 * i);
  s_row[i] = row;
  hash_clear(s_hash);
  if (i == 0) s_want = 0;
  __syncthreads();
  bool ok = i < n && row >= 0 && row < S.rows;
  int len = 0, have = 0, need = 0;
  if (ok) len = S.lens[row];
  const int place = ok ? hash_add(s_hash, row, i) : 0;
  __syncthreads();
  if (ok) {
    ok = s_hash.first[place] == i && len >= 0 && more >= 0 && (int64_t)len + more <= (int64_t)S.width * S.page_size;
  }
  if (ok) {
    have = pages_of(S, len);
    need = pages_of(S, len + more) - have;
  }
  const Demand d = demand(S, refs0, need, s_wave);
  const bool served = ok && d.upto <= d.free;
  s_upto[i] = d.upto;
  s_have[i] = have;
  // the pages of the last served entry end the list
  if (served && need > 0) atomicMax(&s_want, d.upto);
  __syncthreads();
  take_free(S, refs0, s_want, s_wave, [&](int k, int page) {
    const int e = owner_of(s_upto, kOne, k);
    const int at = s_have[e] + k - (e ? s_upto[e - 1] : 0);
    S.table[(int64_t)s_row[e] * S.width + at] = page;
    S.ref[page] = 1;
  });
  if (i < n) {
    if (served) S.lens[row] = len + more;
    status[i] = served ? 0 : (ok ? -2 : -1);
  }
}

// Fork, first kernel: which entries are served, a fresh page and a copy for
// each partly filled one, and the destinations' lengths.  Every length is
// read before any is written.  Few rows (kForkInline table entries) are
// shared here too, more of them in fork_rows (free, fork and copy of 4 forks of
// 20 columns: 14.8 us against 18.5 with the second kernel; of 128 forks of 45
// columns: 42.7 against 39).
constexpr int kForkInline = 4 * kOne;
// Column c of a destination's row: the source's page, shared, below `full`, the
// fresh page (written by fork_plan) up to `used`, none behind it.
__device__ __forceinline__ void share_page(const PageState &S, int from, int to, int c, int full,
                                           int used) {
  int32_t *d = S.table + (int64_t)to * S.width + c;
  if (c < full) {
    const int32_t p = S.table[(int64_t)from * S.width + c];
    *d = p;
    if (p >= 0 && p < S.num_pages) atomicAdd(&S.ref[p], 1);
  } else if (c >= used) {
    *d = -1;
  }
}
__global__ __launch_bounds__(kOne) void fork_plan(PageState S, const int32_t *src,
                                                  const int32_t *dst, int n, int32_t *moves,
                                                  int32_t *count, int32_t *status, int inline_rows,
                                                  FastDiv by_width) {
  __shared__ int s_wave[kOneWaves], s_row[kOne], s_upto[kOne], s_src[kOne], s_full[kOne];
  __shared__ int s_used[kOne];
  __shared__ RowHash s_hash;
  __shared__ int s_want;
  const int i = threadIdx.x;
  const int from = i < n ? src[i] : -1, to = i < n ? dst[i] : -1;
  const i32x4 refs0 = refs4(S, 4 * i);
  s_row[i] = to;
  s_src[i] = from;
  hash_clear(s_hash);
  if (i == 0) s_want = 0;
  __syncthreads();
  bool ok = i < n && from >= 0 && from < S.rows && to >= 0 && to < S.rows && from != to;
  const bool named = i < n && to >= 0;
  int len = 0, had = 0, full = 0, need = 0;
  if (ok) {
    len = S.lens[from];
    had = S.lens[to];
  }
  const int place = named ? hash_add(s_hash, to, i) : 0;
  __syncthreads();
  ok = ok && s_hash.first[place] == i && len >= 0 && len <= (int64_t)S.width * S.page_size && had == 0;
  if (ok) {
    full = (int)fdiv((uint32_t)len, S.by_page);
    need = len - full * S.page_size > 0;
  }
  const Demand d = demand(S, refs0, need, s_wave);
  const bool served = ok && d.upto <= d.free;
  s_upto[i] = d.upto;
  s_full[i] = full;
  s_used[i] = served ? full + need : -1;
  if (served && need > 0) atomicMax(&s_want, d.upto);
  __syncthreads();
  const int want = s_want;
  take_free(S, refs0, want, s_wave, [&](int k, int page) {
    const int e = owner_of(s_upto, kOne, k);
    const int old = S.table[(int64_t)s_src[e] * S.width + s_full[e]];
    S.table[(int64_t)s_row[e] * S.width + s_full[e]] = page;
    S.ref[page] = 1;
    moves[2 * k] = old;
    moves[2 * k + 1] = page;
  });
  for (int k = want + i; k < n; k += kOne) {
    moves[2 * k] = -1;
    moves[2 * k + 1] = -1;
  }
  if (i == 0) *count = want;
  if (i < n) {
    if (served) S.lens[to] = len;
    status[i] = served ? 0 : (ok ? -2 : -1);
  }
  if (inline_rows)
    for (int x = i; x < n * S.width; x += kOne) {
      const int e = (int)fdiv((uint32_t)x, by_width);
      if (s_used[e] >= 0) share_page(S, s_src[e], s_row[e], x - e * S.width, s_full[e], s_used[e]);
    }
}

// Fork, second kernel: one workgroup per entry shares the source's whole
// pages (the source's length is the destination's by now; an entry whose
// source is another entry's destination copies nothing, as that row was
// empty when the call began).
__global__ __launch_bounds__(kBlock) void fork_rows(PageState S, const int32_t *src,
                                                    const int32_t *dst, const int32_t *status) {
  const int i = blockIdx.x;
  if (status[i] != 0) return;
  const int from = src[i], to = dst[i];
  const int len = S.lens[to], full = (int)fdiv((uint32_t)len, S.by_page);
  const int used = full + (len > full * S.page_size);
  for (int c = threadIdx.x; c < S.width; c += kBlock) share_page(S, from, to, c, full, used);
}

__global__ __launch_bounds__(kBlock) void free_rows(PageState S, const int32_t *seqs) {
  const int i = blockIdx.x, row = seqs[i];
  if (row < 0 || row >= S.rows) return;
  // only the first entry that names a row releases it
  bool seen = false;
  for (int j = threadIdx.x; j < i; j += kBlock) seen = seen || seqs[j] == row;
  __shared__ int s_seen;
  if (threadIdx.x == 0) s_seen = 0;
  __syncthreads();
  if (seen) s_seen = 1;
  __syncthreads();
  if (s_seen) return;
  int32_t *a = S.table + (int64_t)row * S.width;
  for (int c = threadIdx.x; c < S.width; c += kBlock) {
    const int32_t p = a[c];
    if (p >= 0 && p < S.num_pages) atomicAdd(&S.ref[p], -1);
    a[c] = -1;
  }
  if (threadIdx.x == 0) S.lens[row] = 0;
}

// Compaction: with n pages in use, the k-th used page at or above n moves to
// the k-th free page below n (there are as many of one as of the other, at
// most half of all pages).  map[p]: where page p goes.
__global__ __launch_bounds__(kOne) void compact_plan(PageState S, int32_t *map, int32_t *moves,
                                                     int max_moves, int32_t *count) {
  __shared__ int s_wave[kOneWaves];
  int n = 0, live;
  for (int i = 4 * (int)threadIdx.x; i < S.num_pages; i += 4 * kOne) {
    const i32x4 x = refs4(S, i);
#pragma unroll
    for (int j = 0; j < 4; j++) n += i + j < S.num_pages && x[j] != 0;
  }
  scan_block(n, s_wave, &live);
  // the two lists, each into its column of moves
  int holes = 0, high = 0;
  for (int base = 0; base < S.num_pages; base += 4 * kOne) {
    const int i = base + 4 * (int)threadIdx.x;
    const i32x4 x = refs4(S, i);
    int hole = 0, up = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int p = i + j;
      hole += p < live && x[j] == 0;
      up += p >= live && p < S.num_pages && x[j] != 0;
    }
    // both counts in one scan: at most 4 * 1024 each
    int both;
    const int upto = scan_block(hole | (up << 16), s_wave, &both);
    int kh = holes + (upto & 0xFFFF) - hole, ku = high + (upto >> 16) - up;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int p = i + j;
      if (p < live && x[j] == 0) {
        moves[2 * kh + 1] = p;
        kh++;
      }
      if (p >= live && p < S.num_pages && x[j] != 0) {
        moves[2 * ku] = p;
        ku++;
      }
      if (p < S.num_pages) map[p] = p;
    }
    holes += both & 0xFFFF;
    high += both >> 16;
  }
  for (int k = high + (int)threadIdx.x; k < max_moves; k += kOne) {
    moves[2 * k] = -1;
    moves[2 * k + 1] = -1;
  }
  if (threadIdx.x == 0) *count = high;
  __syncthreads();
  for (int k = threadIdx.x; k < high; k += kOne) {
    const int a = moves[2 * k], b = moves[2 * k + 1];
    map[a] = b;
    S.ref[b] = S.ref[a];
    S.ref[a] = 0;
  }
}
__global__ __launch_bounds__(kBlock) void compact_table(PageState S, const int32_t *map,
                                                        int64_t entries) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= entries) return;
  const int32_t p = S.table[i];
  if (p >= 0 && p < S.num_pages) S.table[i] = map[p];
}

// Copies pages moves[m] = (from, to) of every pool and layer, m < *count.  The
// grid is resident and loops over 16 KiB tiles, since only the device knows
// the count; all moves of one pool and layer come before the next, so that
// what is in flight lies within one region (1 GB of traffic over 2 pools of
// 8 layers: 191-195 us against 206 with the pools and layers of a move first;
// 2, 3, 4 and 8 workgroups a compute unit: 191, 195, 198, 201; plain instead of
// non-temporal accesses: 208).
constexpr int kCopyPer = 4, kCopyTile = kCopyPer * kBlock;     // units of a lane and of a tile
constexpr unsigned kCopyGrid = 3;                              // workgroups a compute unit
template <int B, bool NT>
__global__ __launch_bounds__(kBlock) void copy_pages(MutPtrTable pools, FastDiv by_pools,
                                                     FastDiv by_tiles, uint32_t regions,
                                                     uint64_t num_pages, uint64_t page_units,
                                                     const int32_t *moves, int max_moves,
                                                     const int32_t *count) {
  typedef typename UnitT<B>::T U;
  int c = count ? *count : max_moves;
  const uint32_t n = c < 0 ? 0 : (uint32_t)(c < max_moves ? c : max_moves);
  const uint32_t total = regions * by_tiles.d * n;               // < 2^31 - the grid
  for (uint32_t x = blockIdx.x; x < total; x += gridDim.x) {
    const uint32_t q = fdiv(x, by_tiles), tile = x - q * by_tiles.d;
    const uint32_t z = q / n, m = q - z * n;
    const uint32_t layer = fdiv(z, by_pools), pool = z - layer * by_pools.d;
    const int64_t a = moves[2 * (size_t)m], b = moves[2 * (size_t)m + 1];
    if (a < 0 || b < 0 || (uint64_t)a >= num_pages || (uint64_t)b >= num_pages || a == b) continue;
    char *base = reinterpret_cast<char *>(pools.p[pool]) + layer * num_pages * page_units * B;
    const U *s = reinterpret_cast<const U *>(base) + (uint64_t)a * page_units;
    U *d = reinterpret_cast<U *>(base) + (uint64_t)b * page_units;
    const uint64_t at = (uint64_t)tile * kCopyTile + threadIdx.x;
    U v[kCopyPer];
#pragma unroll
    for (int j = 0; j < kCopyPer; j++)
      if (at + j * kBlock < page_units) v[j] = ld<U, NT>(s, at + j * kBlock);
#pragma unroll
    for (int j = 0; j < kCopyPer; j++)
      if (at + j * kBlock < page_units) st<U, NT>(d, at + j * kBlock, v[j]);
  }
}

struct WriteArgs {
  PtrTable k, v, table, lens, starts, seqs;
  MutPtrTable kp, vp;
  int64_t k_stride, v_stride, page_stride, tok_stride, head_stride;   // elements
  int64_t tokens, num_pages;
  int batch, rows, max_pages, page_size;
  uint32_t head_units;           // 16-byte units of a head
  uint32_t row_units;            // ... of a token: heads * head_units
  FastDiv by_page, by_head, by_tokens;
};

// New tokens' keys and values: a wave per (rank, token) copies both rows.  It
// loads up to 2 KiB of each before it looks up where they go.
constexpr int kWriteAhead = 2;           // units of a lane loaded ahead, of each row
__global__ __launch_bounds__(kBlock) void write_rows(WriteArgs A, uint32_t waves) {
  const uint32_t w = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  if (w >= waves) return;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t r = fdiv(w, A.by_tokens);
  const int64_t t = w - r * (uint32_t)A.tokens;
  const char *ks = reinterpret_cast<const char *>(A.k.p[r]) + t * A.k_stride * 2;
  const char *vs = reinterpret_cast<const char *>(A.v.p[r]) + t * A.v_stride * 2;
  u32x4 kx[kWriteAhead], vx[kWriteAhead];
#pragma unroll
  for (int j = 0; j < kWriteAhead; j++)
    if (lane + 64 * j < A.row_units) {
      kx[j] = ld<u32x4>(ks, lane + 64 * j);
      vx[j] = ld<u32x4>(vs, lane + 64 * j);
    }
  // the last b with starts[b] <= t, 64 ways at a time
  const int32_t *starts = reinterpret_cast<const int32_t *>(A.starts.p[r]);
  int lo = 0, n = A.batch;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = (int)lane * step;
    const uint64_t below = __ballot(i < n && starts[lo + i] <= t);
    const int c = below ? 63 - __builtin_clzll(below) : 0;
    lo += c * step;
    n = n - c * step < step ? n - c * step : step;
  }
  const int64_t a = starts[lo], z = starts[lo + 1];
  if (a < 0 || t < a || t >= z) return;
  const int32_t *sq = reinterpret_cast<const int32_t *>(A.seqs.p[r]);
  const int row = sq ? sq[lo] : lo;
  if (row < 0 || row >= A.rows) return;
  const int64_t pos = reinterpret_cast<const int32_t *>(A.lens.p[r])[row] - (z - t);
  if (pos < 0 || pos >= (int64_t)A.max_pages * A.page_size) return;
  const int pi = (int)fdiv((uint32_t)pos, A.by_page), slot = (int)pos - pi * A.page_size;
  const int64_t page = reinterpret_cast<const int32_t *>(A.table.p[r])[(int64_t)row * A.max_pages + pi];
  if (page < 0 || page >= A.num_pages) return;
  const int64_t to = page * A.page_stride + slot * A.tok_stride;
  char *kd = reinterpret_cast<char *>(A.kp.p[r]), *vd = reinterpret_cast<char *>(A.vp.p[r]);
  auto put = [&](uint32_t u, u32x4 x, u32x4 y) {
    const uint32_t h = fdiv(u, A.by_head);
    const int64_t off = (to + h * A.head_stride) * 2 + (u - h * A.head_units) * 16;
    *reinterpret_cast<u32x4 *>(kd + off) = x;
    *reinterpret_cast<u32x4 *>(vd + off) = y;
  };
#pragma unroll
  for (int j = 0; j < kWriteAhead; j++)
    if (lane + 64 * j < A.row_units) put(lane + 64 * j, kx[j], vx[j]);
  for (uint32_t u = lane + 64 * kWriteAhead; u < A.row_units; u += 64)
    put(u, ld<u32x4>(ks, u), ld<u32x4>(vs, u));
}

PageState state(int32_t *table, int32_t *lens, int32_t *ref, int rows, int width, int num_pages,
                int page_size) {
  PageState S{};
  S.table = table, S.lens = lens, S.ref = ref;
  S.rows = rows, S.width = width, S.num_pages = num_pages, S.page_size = page_size;
  S.by_page = make_fastdiv((uint32_t)page_size);
  return S;
}

}  // namespace

int launch_kv_extend(const Launch &L, int32_t *table, int32_t *lens, int32_t *ref, int rows,
                     int width, int num_pages, int page_size, const int32_t *seqs,
                     const int32_t *add, int n, int32_t *status) {
  const PageState S = state(table, lens, ref, rows, width, num_pages, page_size);
  hipLaunchKernelGGL(extend_rows, dim3(1), dim3(kOne), 0, L.stream, S, seqs, add, n, status);
  return hip_status();
}

int launch_kv_fork(const Launch &L, int32_t *table, int32_t *lens, int32_t *ref, int rows,
                   int width, int num_pages, int page_size, const int32_t *src,
                   const int32_t *dst, int n, int32_t *moves, int32_t *count, int32_t *status) {
  const PageState S = state(table, lens, ref, rows, width, num_pages, page_size);
  const bool few = (int64_t)n * width <= kForkInline;
  hipLaunchKernelGGL(fork_plan, dim3(1), dim3(kOne), 0, L.stream, S, src, dst, n, moves, count,
                     status, (int)few, make_fastdiv((uint32_t)(width > 0 ? width : 1)));
  if (!few)
    hipLaunchKernelGGL(fork_rows, dim3(n), dim3(kBlock), 0, L.stream, S, src, dst,
                       (const int32_t *)status);
  return hip_status();
}

int launch_kv_free(const Launch &L, int32_t *table, int32_t *lens, int32_t *ref, int rows,
                   int width, int num_pages, const int32_t *seqs, int n) {
  const PageState S = state(table, lens, ref, rows, width, num_pages, 1);
  hipLaunchKernelGGL(free_rows, dim3(n), dim3(kBlock), 0, L.stream, S, seqs);
  return hip_status();
}

int launch_kv_compact(const Launch &L, int32_t *table, int32_t *ref, int rows, int width,
                      int num_pages, int32_t *moves, int max_moves, int32_t *count, int32_t *map) {
  const PageState S = state(table, nullptr, ref, rows, width, num_pages, 1);
  if ((uint64_t)rows * (uint64_t)width > kMaxThreads - kBlock) return COLL_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(compact_plan, dim3(1), dim3(kOne), 0, L.stream, S, map, moves, max_moves,
                     count);
  const int64_t entries = (int64_t)rows * width;
  if (entries > 0) {
    const int64_t groups = (entries + kBlock - 1) / kBlock;
    hipLaunchKernelGGL(compact_table, dim3((unsigned)groups), dim3(kBlock), 0, L.stream, S,
                       (const int32_t *)map, entries);
  }
  return hip_status();
}

int launch_kv_copy_pages(const Launch &L, int npools, const MutPtrTable &pools, size_t layers,
                         size_t num_pages, size_t page_bytes, const int32_t *moves, int max_moves,
                         const int32_t *count) {
  uintptr_t bits = page_bytes;
  for (int i = 0; i < npools; i++) bits |= (uintptr_t)pools.p[i];
  const int unit = copy_unit(bits);
  const uint64_t units = page_bytes / unit;
  const uint64_t tiles = (units + kCopyTile - 1) / kCopyTile;
  const uint64_t resident = (uint64_t)L.num_cus * kCopyGrid, lim = (1ull << 31) - resident;
  const uint64_t regions = (uint64_t)npools * layers;
  if (layers >= lim || tiles >= lim || regions >= lim / tiles ||
      (uint64_t)max_moves >= lim / (regions * tiles))
    return COLL_ERR_UNSUPPORTED;
  const uint64_t most = regions * tiles * (uint64_t)max_moves;
  const unsigned grid = (unsigned)(most < resident ? most : resident);
  const bool nt = 2 * regions * page_bytes * (uint64_t)max_moves >= L.nt_bytes;
  COLL_UNIT_SWITCH(copy_pages, unit, nt, dim3(grid), L.stream, pools, make_fastdiv((uint32_t)npools),
                   make_fastdiv((uint32_t)tiles), (uint32_t)regions, (uint64_t)num_pages, units, moves,
                   max_moves, count);
  return hip_status();
}

int launch_kv_write(const Launch &L, int R, const PtrTable &k, const PtrTable &v,
                    const MutPtrTable &kp, const MutPtrTable &vp, const PtrTable &table,
                    const PtrTable &lens, const PtrTable &starts, const PtrTable &seqs,
                    int64_t tokens, int batch, int rows, int max_pages, int64_t num_pages,
                    int page_size, int kv_heads, int D, int64_t k_stride, int64_t v_stride,
                    int64_t page_stride, int64_t tok_stride, int64_t head_stride) {
  WriteArgs A{};
  A.k = k, A.v = v, A.kp = kp, A.vp = vp;
  A.table = table, A.lens = lens, A.starts = starts, A.seqs = seqs;
  A.k_stride = k_stride, A.v_stride = v_stride;
  A.page_stride = page_stride, A.tok_stride = tok_stride, A.head_stride = head_stride;
  A.tokens = tokens, A.num_pages = num_pages;
  A.batch = batch, A.rows = rows, A.max_pages = max_pages, A.page_size = page_size;
  A.head_units = (uint32_t)D / 8;
  A.row_units = A.head_units * (uint32_t)kv_heads;
  A.by_page = make_fastdiv((uint32_t)page_size);
  A.by_head = make_fastdiv(A.head_units);
  if ((uint64_t)tokens * R * 64 > kMaxThreads - kBlock) return COLL_ERR_UNSUPPORTED;
  A.by_tokens = make_fastdiv((uint32_t)tokens);
  const uint32_t waves = (uint32_t)(tokens * R), per = kBlock / 64;
  hipLaunchKernelGGL(write_rows, dim3((waves + per - 1) / per), dim3(kBlock), 0, L.stream, A, waves);
  return hip_status();
}

}  // namespace coll
