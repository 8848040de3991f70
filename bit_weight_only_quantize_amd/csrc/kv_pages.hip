// Pages of the 4-bit key/value cache on gfx950: copied (awq_kv_copy_pages), shared by
// branches of a request (awq_kv_fork), given back (awq_kv_release) and drawn together
// at the front of the pool (awq_kv_compact).
//
// A page is three runs of memory, its codes, steps and zero points, each a multiple
// of 16 bytes, so copies are of 16-byte units with no regard to what they hold.
// `shared` counts, for each page, the block tables' entries that hold it beyond the
// first: awq_kv_assign's fresh pages have none and it need not know of the counts.
// Counts change by atomic additions, whose order does not matter, and lists are
// written by rank, so every result is the same whatever the order of execution.

#include "awq_internal.h"
#include "device_common.h"

namespace awq {

constexpr int kPageThreads = 256;
constexpr int kPieceUnits = 1024;          // 16-byte units that a workgroup copies at a time

// The runs of a page, in 16-byte units.
struct PageRuns {
  int64_t codes, scales, zeros;
};
__host__ __device__ __forceinline__ PageRuns page_runs(const KvCache &c) {
  const int64_t n = (int64_t)c.page_size * c.heads;
  return PageRuns{n * c.head_dim / 16, n / 4, c.zeros ? n / 8 : 0};
}
// Pieces of a page: of its codes, and of its steps and zero points together.
__host__ __device__ __forceinline__ int64_t pieces_of(const PageRuns &r) {
  return (r.codes + kPieceUnits - 1) / kPieceUnits + (r.scales + r.zeros + kPieceUnits - 1) / kPieceUnits;
}

// Piece `piece` of page `from` to page `to`, by a workgroup: four loads in flight per lane.
// (Codes have a path of their own, whose addresses are the same for all lanes but for the
// lane's place: with one path for all three runs, each lane telling which, 2000 pages of 69 KB
// took 63 us.)
__device__ __forceinline__ void copy_piece(const KvCache &c, const PageRuns &r, int64_t from, int64_t to, int64_t piece) {
  constexpr int kPer = kPieceUnits / kPageThreads;
  u32x4 v[kPer];
  const int64_t code_pieces = (r.codes + kPieceUnits - 1) / kPieceUnits;
  if (piece < code_pieces) {
    const u32x4 *src = reinterpret_cast<const u32x4 *>(c.codes) + from * r.codes + piece * kPieceUnits;
    u32x4 *dst = reinterpret_cast<u32x4 *>(c.codes) + to * r.codes + piece * kPieceUnits;
    const int64_t left = r.codes - piece * kPieceUnits;
    const int n = (int)(left < kPieceUnits ? left : kPieceUnits);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kPageThreads + (int)threadIdx.x < n) v[i] = src[i * kPageThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kPageThreads + (int)threadIdx.x < n) dst[i * kPageThreads + threadIdx.x] = v[i];
    return;
  }
  const u32x4 *scales = reinterpret_cast<const u32x4 *>(c.scales) + from * r.scales;
  const u32x4 *zeros = reinterpret_cast<const u32x4 *>(c.zeros) + from * r.zeros;
  u32x4 *scales_to = reinterpret_cast<u32x4 *>(c.scales) + to * r.scales;
  u32x4 *zeros_to = reinterpret_cast<u32x4 *>(c.zeros) + to * r.zeros;
  const int64_t first = (piece - code_pieces) * kPieceUnits + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t u = first + i * kPageThreads;
    if (u < r.scales) v[i] = scales[u];
    else if (u < r.scales + r.zeros) v[i] = zeros[u - r.scales];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t u = first + i * kPageThreads;
    if (u < r.scales) scales_to[u] = v[i];
    else if (u < r.scales + r.zeros) zeros_to[u - r.scales] = v[i];
  }
}

__device__ __forceinline__ bool is_page(int64_t id, int64_t pages) { return id >= 0 && id < pages; }

// Blocks that `len` tokens take of a row of max_blocks.
__device__ __forceinline__ int64_t blocks_of(int64_t len, int pshift, int max_blocks) {
  const int64_t n = len > 0 ? (len + ((int64_t)1 << pshift) - 1) >> pshift : 0;
  return n < max_blocks ? n : max_blocks;
}

// ---- copy ---------------------------------------------------------------------------
// Bound by memory: a read and a write of every byte.  2000 pages of 69 KB: 57 us, 4.8 TB/s (4096
// workgroups in a loop: 65).
__global__ __launch_bounds__(kPageThreads) void kv_copy_pages_kernel(KvCache c, const int32_t *__restrict__ src,
                                                                     const int32_t *__restrict__ dst, int64_t units,
                                                                     int64_t pieces) {
  const PageRuns r = page_runs(c);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t i = u / pieces;
    const int32_t from = src[i], to = dst[i];
    if (is_page(from, c.pages) && is_page(to, c.pages) && from != to) copy_piece(c, r, from, to, u - i * pieces);
  }
}

// ---- fork ---------------------------------------------------------------------------
// Workgroup (i, part): fork i's share of the table entries, and of the page that is copied.
// The free page that it takes is numbered by the forks before it that take one, which every
// workgroup counts itself: a few hundred pairs of loads, where an exchange between
// workgroups would cost another launch.  Bound by latency: lists, lengths, the parent's
// entries, the page (8 forks of up to 1500 tokens 5.4 us; 200 of up to 20000 in small pages, 120000
// counts, 9.8).  That is quadratic in the forks: 700 of 20 tokens take 17 us, 5000 79, 20000 395 and
// 65535, the most, 3.2 ms.
struct ForkPage {
  int64_t last;            // the parent's page that is copied, or -1
  bool takes;
};
__device__ __forceinline__ ForkPage fork_page(const ForkArgs &a, int i) {
  const int parent = a.parents[i], child = a.children[i];
  ForkPage f = {-1, false};
  if (!is_page(parent, a.num_seqs) || !is_page(child, a.num_seqs) || parent == child) return f;
  const int64_t cap = (int64_t)a.max_blocks << a.pshift;
  int64_t len = a.lens[i];
  len = len < cap ? len : cap;
  if (len <= 0 || (len & (((int64_t)1 << a.pshift) - 1)) == 0) return f;
  f.last = a.table[(int64_t)parent * a.max_blocks + (len >> a.pshift)];
  f.takes = is_page(f.last, a.pages);
  return f;
}

__global__ __launch_bounds__(kPageThreads) void kv_fork_kernel(ForkArgs a, KvCache c) {
  __shared__ int64_t s_count[kPageThreads / 64];
  const int i = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
  const int parent = a.parents[i], child = a.children[i];
  const bool valid = is_page(parent, a.num_seqs) && is_page(child, a.num_seqs) && parent != child;
  const int64_t cap = (int64_t)a.max_blocks << a.pshift;
  int64_t len = a.lens[i];
  len = !valid || len < 0 ? 0 : len < cap ? len : cap;
  const int64_t full = len >> a.pshift;
  const bool partial = (len & (((int64_t)1 << a.pshift) - 1)) != 0;
  const int32_t *from = a.table + (int64_t)parent * a.max_blocks;
  int32_t *to = a.table + (int64_t)child * a.max_blocks;
  for (int64_t j = (int64_t)part * kPageThreads + threadIdx.x; j < full; j += (int64_t)parts * kPageThreads) {
    const int32_t id = from[j];
    to[j] = id;
    if (is_page(id, a.pages)) atomicAdd(a.shared + id, 1);
  }
  const bool reports = i == a.n - 1 && part == 0;
  if (!partial && !reports) return;
  // forks before this one that take a page
  const int64_t taken = a.taken && *a.taken > 0 ? *a.taken : 0;
  int64_t before = 0;
  for (int64_t j = threadIdx.x; j < i; j += kPageThreads) before += fork_page(a, (int)j).takes;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d, 64);
  if ((threadIdx.x & 63) == 0) s_count[threadIdx.x >> 6] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kPageThreads / 64; ++w) before += s_count[w];
  const ForkPage mine = fork_page(a, i);
  if (reports && threadIdx.x == 0) {
    const int64_t all = taken + before + mine.takes;
    *a.pages_used = all > 0x7FFFFFFF ? 0x7FFFFFFF : (int32_t)all;
  }
  if (!partial) return;
  int64_t fresh = -1;
  if (mine.takes && taken + before < a.num_free) fresh = a.free_pages[taken + before];
  if (!is_page(fresh, a.pages)) fresh = -1;
  if (part == 0 && threadIdx.x == 0) to[full] = (int32_t)fresh;
  if (fresh < 0 || fresh == mine.last) return;
  const PageRuns r = page_runs(c);
  const int64_t pieces = pieces_of(r);
  for (int64_t p = part; p < pieces; p += parts) copy_piece(c, r, mine.last, fresh, p);
}

__global__ void kv_fork_none_kernel(const int32_t *taken, int32_t *pages_used) {
  *pages_used = taken && *taken > 0 ? *taken : 0;
}

// ---- ranks ---------------------------------------------------------------------------
// A workgroup ranks the flagged ones of its items, item r * THREADS + thread in round r so that
// loads are coalesced: each wave's ballots are counted in LDS, and one scan of the counts
// gives every ballot's first rank.
constexpr int kChunkRounds = 4;
constexpr int kChunk = kChunkRounds * kPageThreads;    // items of a workgroup of many
constexpr int kAlone = 1024;                           // threads of a single workgroup
constexpr int kAloneRounds = 32;
constexpr int64_t kAloneItems = (int64_t)kAloneRounds * kAlone;
constexpr int64_t kAloneEntries = 65536;               // table entries that one workgroup looks through,
constexpr int64_t kAloneReleases = 2048;               // ... and releases

template <int THREADS>
struct Ranks {
  static constexpr int kWaves = THREADS / 64, kRounds = THREADS == kAlone ? kAloneRounds : kChunkRounds;
  static constexpr int kCounts = kRounds * kWaves;
  struct Shared {
    int32_t first[kCounts];
    int32_t total;
  };
  Shared &s;
  int rounds;                                          // that hold items
  uint32_t mask = 0;                                   // bit r: the thread's item of round r
  __device__ __forceinline__ Ranks(Shared &sh, int64_t items)
      : s(sh), rounds(items >= (int64_t)kRounds * THREADS ? kRounds : items > 0 ? (int)((items + THREADS - 1) / THREADS) : 0) {}
  // All threads call it; returns the number of flagged items.
  template <class F>
  __device__ __forceinline__ int32_t count(F flag) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // (rolled up: code that one workgroup runs once costs its fetching)
#pragma unroll 1
    for (int r = 0; r < kRounds; r += 4) {
      bool f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = r < rounds && flag((r + i) * THREADS + (int)threadIdx.x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mask |= (uint32_t)f[i] << (r + i);
        const uint64_t b = __ballot(f[i]);
        if (lane == 0) s.first[(r + i) * kWaves + wave] = __popcll(b);
      }
    }
    __syncthreads();
    if (wave == 0) {                                   // exclusive scan, kPer per lane
      constexpr int kPer = kCounts < 64 ? 1 : kCounts / 64;
      int32_t v[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = sum;
        if (lane * kPer + i < kCounts) sum += s.first[lane * kPer + i];
      }
      int32_t up = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t x = __shfl_up(up, d, 64);
        if (lane >= d) up += x;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane * kPer + i < kCounts) s.first[lane * kPer + i] = up - sum + v[i];
      if (lane == 63) s.total = up;
    }
    __syncthreads();
    return s.total;
  }
  // Flagged items before the thread's item of round r, and whether it is flagged itself.
  __device__ __forceinline__ int32_t rank(int r, bool &f) const {
    f = (mask >> r) & 1u;
    const uint64_t below = __ballot(f) & (((uint64_t)1 << (threadIdx.x & 63)) - 1);
    return s.first[r * kWaves + (threadIdx.x >> 6)] + __popcll(below);
  }
};

// Sum of n counts and of the first `mine` of them, by a workgroup of kPageThreads.
struct Sums {
  int64_t before, all;
};
__device__ __forceinline__ Sums sum_counts(const int32_t *counts, int64_t n, int64_t mine) {
  __shared__ int64_t s_sum[2][kPageThreads / 64];
  Sums t = {0, 0};
  for (int64_t i = threadIdx.x; i < n; i += kPageThreads) {
    const int64_t x = counts[i];
    t.all += x;
    t.before += i < mine ? x : 0;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    t.all += __shfl_xor(t.all, d, 64);
    t.before += __shfl_xor(t.before, d, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    s_sum[0][threadIdx.x >> 6] = t.before;
    s_sum[1][threadIdx.x >> 6] = t.all;
  }
  __syncthreads();
  t = Sums{0, 0};
#pragma unroll
  for (int w = 0; w < kPageThreads / 64; ++w) {
    t.before += s_sum[0][w];
    t.all += s_sum[1][w];
  }
  return t;
}

// ---- release ---------------------------------------------------------------------------
// Released entries become -1 and their pages' counts fall by one, below zero for a page without
// another holder.  Then the free list: what is left of the old one, and the pages below zero by
// number.  A workgroup per 256 entries of a row, and a second launch whose one workgroup
// ranks the list, or for long ones two, in chunks: counts, then places.  A small table and a short
// list take one launch of one workgroup: whoever brings a count below zero marks the page in
// LDS, so counts are not read again.  One launch against two, in a graph: 256 entries of 1024 pages, all
// released, 5.9 us and 6.9; 1024 entries 6.5 and 6.8; 1536 entries 7.8 and 7.4; 4096 entries 13.8 and 9.2.  With
// two rows of many released, as a step has it: 2048 entries 6.9 and 7.4, 4096 entries 9.3 and 9.1.  So up to 2048.
// Blocks of row b that are released: those whose tokens below its length all lie in [lo, hi).
struct Blocks {
  int64_t first, stop;
};
__device__ __forceinline__ Blocks released(const ReleaseArgs &a, int64_t b) {
  const int64_t cap = (int64_t)a.max_blocks << a.pshift;
  int64_t len = a.seq_lens[b];
  len = len < 0 ? 0 : len < cap ? len : cap;
  int64_t lo = a.start ? a.start[b] : 0, hi = a.end ? a.end[b] : len;
  lo = lo < 0 ? 0 : lo;
  return Blocks{(lo + ((int64_t)1 << a.pshift) - 1) >> a.pshift,
                hi >= len ? blocks_of(len, a.pshift, a.max_blocks) : hi > 0 ? hi >> a.pshift : 0};
}

__global__ __launch_bounds__(kPageThreads) void kv_release_rows_kernel(ReleaseArgs a) {
  const int64_t b = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
  const Blocks blocks = released(a, b);
  const int64_t first = blocks.first, stop = blocks.stop;
  int32_t *row = a.table + b * a.max_blocks;
  for (int64_t j = first + part * kPageThreads + threadIdx.x; j < stop; j += parts * kPageThreads) {
    const int32_t id = row[j];
    row[j] = -1;
    if (is_page(id, a.pages)) atomicSub(a.shared + id, 1);
  }
}

// Item i of the list: an entry of the old free list, then the pages.  `marks`: of the pages
// to free, a bit each (one launch), or null where their counts say so.
struct ReleaseItems {
  const ReleaseArgs &a;
  int64_t taken;
  const uint32_t *marks;
  __device__ __forceinline__ bool flag(int64_t i) const {
    if (i < a.num_free) return i >= taken && is_page(a.free_pages[i], a.pages);
    const int64_t id = i - a.num_free;
    if (id >= a.pages) return false;
    return marks ? (marks[id >> 5] >> (id & 31)) & 1u : a.shared[id] < 0;
  }
  __device__ __forceinline__ void place(int64_t i, int64_t at) const {
    const int64_t id = i < a.num_free ? (int64_t)a.free_pages[i] : i - a.num_free;
    if (at < a.num_out) a.free_out[at] = (int32_t)id;
    if (i >= a.num_free) a.shared[id] = 0;
  }
};
__device__ __forceinline__ int64_t taken_of(const ReleaseArgs &a) { return a.taken && *a.taken > 0 ? *a.taken : 0; }

__global__ __launch_bounds__(kPageThreads) void kv_release_count_kernel(ReleaseArgs a, int32_t *counts) {
  __shared__ Ranks<kPageThreads>::Shared s;
  const ReleaseItems items{a, taken_of(a), nullptr};
  const int64_t base = (int64_t)blockIdx.x * kChunk;
  Ranks<kPageThreads> ranks(s, a.num_free + a.pages - base);
  const int32_t n = ranks.count([&](int i) { return items.flag(base + i); });
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// THREADS = kAlone: one workgroup has all items; ROWS: the table's entries too.
template <int THREADS, bool ROWS>
__global__ __launch_bounds__(THREADS) void kv_release_list_kernel(ReleaseArgs a, const int32_t *counts) {
  __shared__ typename Ranks<THREADS>::Shared s;
  __shared__ uint32_t marks[ROWS ? kAloneItems / 32 : 1];
  const ReleaseItems items{a, taken_of(a), ROWS ? marks : nullptr};
  const int64_t base = (int64_t)blockIdx.x * (Ranks<THREADS>::kRounds * THREADS);
  Ranks<THREADS> ranks(s, a.num_free + a.pages - base);
  if constexpr (ROWS) {
    marks[threadIdx.x] = 0;
    __syncthreads();
    const int entries = a.num_seqs * a.max_blocks;
#pragma unroll 1
    for (int e = threadIdx.x; e < entries; e += THREADS) {
      const int b = e / a.max_blocks, j = e - b * a.max_blocks;
      const int32_t id = a.table[e];
      const Blocks blocks = released(a, b);
      if (j < blocks.first || j >= blocks.stop) continue;
      a.table[e] = -1;
      // (the one that finds no further holder; a page given back too often was marked then)
      if (is_page(id, a.pages) && atomicSub(a.shared + id, 1) == 0) atomicOr(&marks[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
  }
  const int32_t n = ranks.count([&](int i) { return items.flag(base + i); });
  Sums sums = {0, n};
  if constexpr (THREADS != kAlone) sums = sum_counts(counts, gridDim.x, blockIdx.x);
#pragma unroll 1
  for (int r = 0; r < ranks.rounds; ++r) {
    bool f;
    const int64_t at = sums.before + ranks.rank(r, f);
    if (f) items.place(base + r * THREADS + threadIdx.x, at);
  }
  for (int64_t i = sums.all + (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.num_out; i += (int64_t)gridDim.x * THREADS)
    a.free_out[i] = -1;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = (int32_t)(sums.all > 0x7FFFFFFF ? 0x7FFFFFFF : sums.all);
}

// ---- compact ---------------------------------------------------------------------------
// Of n pages in use, those numbered n or more move into the holes below n, the last into
// the first: the k-th hole from the front, number p, has p - (used ones before it) = k, and
// the k-th page from the back has n - 1 - (used ones before it) = k, so both lists are
// written from one ranking of the used pages.  One workgroup marks and ranks a pool of up
// to 32768 pages and a table of up to 65536 entries in LDS (one launch); larger ones take
// four: clear, mark, count, list.
// The last launch copies the pages, moves their counts and renumbers the tables.  (7300 pages of 68
// KB, 96 rows, 1700 pages moved: 11 us for the lists and 53, 4.4 TB/s, for the pages.)
__global__ __launch_bounds__(kPageThreads) void kv_compact_clear_kernel(uint8_t *used, int64_t pages) {
  for (int64_t i = (int64_t)blockIdx.x * kPageThreads + threadIdx.x; i < pages; i += (int64_t)gridDim.x * kPageThreads)
    used[i] = 0;
}

__global__ __launch_bounds__(kPageThreads) void kv_compact_mark_kernel(CompactArgs a, int64_t pages, uint8_t *used) {
  const int64_t b = blockIdx.x, n = blocks_of(a.seq_lens[b], a.pshift, a.max_blocks);
  const int32_t *row = a.table + b * a.max_blocks;
  for (int64_t j = threadIdx.x; j < n; j += kPageThreads) {
    const int32_t id = row[j];
    if (is_page(id, pages)) used[id] = 1;
  }
}

__global__ __launch_bounds__(kPageThreads) void kv_compact_count_kernel(const uint8_t *used, int64_t pages, int32_t *counts) {
  __shared__ Ranks<kPageThreads>::Shared s;
  const int64_t base = (int64_t)blockIdx.x * kChunk;
  Ranks<kPageThreads> ranks(s, pages - base);
  const int32_t n = ranks.count([&](int i) { return base + i < pages && used[base + i] != 0; });
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_compact_list_kernel(CompactArgs a, int64_t pages, const uint8_t *used,
                                                                  const int32_t *counts) {
  __shared__ typename Ranks<THREADS>::Shared s;
  __shared__ uint32_t marks[THREADS == kAlone ? kAloneItems / 32 : 1];
  const int64_t base = (int64_t)blockIdx.x * (Ranks<THREADS>::kRounds * THREADS);
  Ranks<THREADS> ranks(s, pages - base);
  int32_t in_chunk;
  if constexpr (THREADS == kAlone) {
    marks[threadIdx.x] = 0;
    __syncthreads();
    // all entries, four to a thread in flight, and the lengths beside them
    constexpr int kPer = 4;
    // (One workgroup's instructions count here: row numbers by one multiplication, exact
    // because entries times the divisor's error stay below 2^32, and 32 bits throughout.)
    const int entries = a.num_seqs * a.max_blocks;      // (at most kAloneEntries)
    const uint32_t inverse = a.max_blocks > 1 ? 0xFFFFFFFFu / (uint32_t)a.max_blocks + 1 : 0;
#pragma unroll 1
    for (int e0 = threadIdx.x; e0 < entries; e0 += kPer * kAlone) {
      int32_t id[kPer];
      bool live[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = e0 + i * kAlone < entries ? e0 + i * kAlone : e0;
        const int b = a.max_blocks > 1 ? (int)__umulhi((uint32_t)e, inverse) : e;
        const int len = a.seq_lens[b];
        id[i] = a.table[e];
        live[i] = len > 0 && e - b * a.max_blocks <= (len - 1) >> a.pshift;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (live[i] && (uint32_t)id[i] < (uint32_t)pages) atomicOr(&marks[id[i] >> 5], 1u << (id[i] & 31));
    }
    __syncthreads();
    in_chunk = ranks.count([&](int i) { return i < (int)pages && ((marks[i >> 5] >> (i & 31)) & 1u); });
  } else {
    in_chunk = ranks.count([&](int i) { return base + i < pages && used[base + i] != 0; });
  }
  Sums sums = {0, in_chunk};
  if constexpr (THREADS != kAlone) sums = sum_counts(counts, gridDim.x, blockIdx.x);
  // (numbers of pages fit 31 bits)
  const int32_t n = (int32_t)sums.all, total = (int32_t)pages;
#pragma unroll 1
  for (int r = 0; r < ranks.rounds; ++r) {
    bool f;
    const int32_t p = (int32_t)base + r * THREADS + threadIdx.x, before = (int32_t)sums.before + ranks.rank(r, f);
    if (p >= total) continue;
    if (p < n && !f) a.holes[p - before] = p;
    if (p >= n && f) {
      a.movers[n - 1 - before] = p;
      a.place[p] = n - 1 - before;
    }
    if (p >= n && !f) a.shared[p] = 0;
    if (p == n) *a.moves = n - before;
    a.free_out[p] = p < total - n ? p + n : -1;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.num_used = n;
    if (n == total) *a.moves = 0;
  }
}

// The first num_seqs workgroups renumber a row each, the others copy.
__global__ __launch_bounds__(kPageThreads) void kv_compact_move_kernel(CompactArgs a, KvCache c) {
  const int64_t b = blockIdx.x, n = *a.num_used, moves = *a.moves;
  if (b < a.num_seqs) {
    const int64_t blocks = blocks_of(a.seq_lens[b], a.pshift, a.max_blocks);
    int32_t *row = a.table + b * a.max_blocks;
    for (int64_t j = threadIdx.x; j < blocks; j += kPageThreads) {
      const int32_t id = row[j];
      if (id >= n && id < c.pages) row[j] = a.holes[a.place[id]];
    }
    return;
  }
  const PageRuns r = page_runs(c);
  const int64_t pieces = pieces_of(r), units = moves * pieces;
  for (int64_t u = b - a.num_seqs; u < units; u += gridDim.x - a.num_seqs) {
    const int64_t k = u / pieces, piece = u - k * pieces;
    const int32_t from = a.movers[k], to = a.holes[k];
    if (piece == 0 && threadIdx.x == 0) {
      a.shared[to] = a.shared[from];
      a.shared[from] = 0;
    }
    copy_piece(c, r, from, to, piece);
  }
}

// ---- launch -----------------------------------------------------------------------------
namespace {
constexpr int64_t kCopyWgs = 1 << 20;      // of a copy: a workgroup for each piece, but for the largest
constexpr int64_t kFillWgs = 4096;         // 16 workgroups per CU
int64_t chunks_of(int64_t items) { return (items + kChunk - 1) / kChunk; }
// Workgroups along a row of the table: one for 256 entries, while that fills the card.
unsigned row_parts(int64_t rows, int64_t blocks) {
  const int64_t parts = (blocks + kPageThreads - 1) / kPageThreads, most = (kFillWgs + rows - 1) / rows;
  return (unsigned)(parts < most ? parts : most);
}
size_t region(int64_t bytes) { return ((size_t)bytes + 255) & ~(size_t)255; }
}  // namespace

hipError_t launch_kv_copy_pages(const KvCache &c, const int32_t *src, const int32_t *dst, int64_t n, hipStream_t st) {
  const int64_t pieces = pieces_of(page_runs(c)), units = n * pieces;
  kv_copy_pages_kernel<<<(unsigned)(units < kCopyWgs ? units : kCopyWgs), kPageThreads, 0, st>>>(c, src, dst, units, pieces);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const ForkArgs &a, const KvCache &c, hipStream_t st) {
  if (a.n == 0) {
    kv_fork_none_kernel<<<1, 1, 0, st>>>(a.taken, a.pages_used);
    return hipGetLastError();
  }
  // a part for each piece of the page and 256 entries of the row, while that fills the card
  int64_t parts = pieces_of(page_runs(c)), rows = row_parts(a.n, a.max_blocks);
  parts = parts > rows ? parts : rows;
  const int64_t most = (kFillWgs + a.n - 1) / a.n;
  parts = parts < most ? parts : most;
  kv_fork_kernel<<<dim3((unsigned)a.n, (unsigned)parts), kPageThreads, 0, st>>>(a, c);
  return hipGetLastError();
}

size_t kv_release_workspace(int64_t pages, int64_t num_free) {
  const int64_t items = pages + num_free;
  return items <= kAloneItems ? 0 : region(chunks_of(items) * 4);
}

hipError_t launch_kv_release(const ReleaseArgs &a, void *workspace, hipStream_t st) {
  const int64_t items = a.pages + a.num_free, entries = (int64_t)a.num_seqs * a.max_blocks;
  if (items <= kAloneItems && entries <= kAloneReleases) {
    kv_release_list_kernel<kAlone, true><<<1, kAlone, 0, st>>>(a, nullptr);
    return hipGetLastError();
  }
  if (entries > 0) {
    kv_release_rows_kernel<<<dim3((unsigned)a.num_seqs, row_parts(a.num_seqs, a.max_blocks)), kPageThreads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (items <= kAloneItems) {
    kv_release_list_kernel<kAlone, false><<<1, kAlone, 0, st>>>(a, nullptr);
    return hipGetLastError();
  }
  int32_t *counts = reinterpret_cast<int32_t *>(workspace);
  kv_release_count_kernel<<<(unsigned)chunks_of(items), kPageThreads, 0, st>>>(a, counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  kv_release_list_kernel<kPageThreads, false><<<(unsigned)chunks_of(items), kPageThreads, 0, st>>>(a, counts);
  return hipGetLastError();
}

// Workspace: moves, holes, movers, places, marks, the chunks' counts.
size_t kv_compact_workspace(int64_t pages) {
  return 256 + 3 * region(pages * 4) + region(pages) + region(chunks_of(pages) * 4);
}

hipError_t launch_kv_compact(CompactArgs a, const KvCache &c, void *workspace, hipStream_t st) {
  char *w = reinterpret_cast<char *>(workspace);
  const size_t list = region(c.pages * 4);
  a.moves = reinterpret_cast<int32_t *>(w);
  a.holes = reinterpret_cast<int32_t *>(w + 256);
  a.movers = reinterpret_cast<int32_t *>(w + 256 + list);
  a.place = reinterpret_cast<int32_t *>(w + 256 + 2 * list);
  hipError_t e;
  if (c.pages <= kAloneItems && (int64_t)a.num_seqs * a.max_blocks <= kAloneEntries) {
    kv_compact_list_kernel<kAlone><<<1, kAlone, 0, st>>>(a, c.pages, nullptr, nullptr);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    uint8_t *used = reinterpret_cast<uint8_t *>(w + 256 + 3 * list);
    int32_t *counts = reinterpret_cast<int32_t *>(w + 256 + 3 * list + region(c.pages));
    const unsigned chunks = (unsigned)chunks_of(c.pages);
    kv_compact_clear_kernel<<<chunks, kPageThreads, 0, st>>>(used, c.pages);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.num_seqs > 0) {
      kv_compact_mark_kernel<<<(unsigned)a.num_seqs, kPageThreads, 0, st>>>(a, c.pages, used);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    kv_compact_count_kernel<<<chunks, kPageThreads, 0, st>>>(used, c.pages, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    kv_compact_list_kernel<kPageThreads><<<chunks, kPageThreads, 0, st>>>(a, c.pages, used, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const int64_t units = c.pages / 2 * pieces_of(page_runs(c));       // (at most that many move)
  const int64_t copies = units < 1 ? 1 : units < kCopyWgs ? units : kCopyWgs;
  kv_compact_move_kernel<<<(unsigned)(a.num_seqs + copies), kPageThreads, 0, st>>>(a, c);
  return hipGetLastError();
}

}  // namespace awq
