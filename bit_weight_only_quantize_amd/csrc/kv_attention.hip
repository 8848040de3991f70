// Attention over the 4-bit paged key/value cache on gfx950: the plan of a call, and the
// kernels (kv_attention.h) for all the keys that a row sees.

#include "kv_attention.h"

namespace awq {

KvAttnPlan kv_attention_plan(int64_t T, int B, int heads, int group, int D, int max_q, int64_t max_kv,
                             int window, int sinks) {
  KvAttnPlan pl{};
  const int64_t rows = (int64_t)max_q * group;
  // keys that a tile of rows can see at most
  int64_t span = max_kv;
  if (window > 0 && (int64_t)window + max_q + sinks < span) span = (int64_t)window + max_q + sinks;
  span = span < 1 ? 1 : span > 0x7FFFFF00 ? 0x7FFFFF00 : span;
  pl.prompt = rows > 32;
  pl.tile_rows = pl.prompt ? kPtRows : 16;
  const int64_t wgs = (int64_t)B * heads * ((rows + pl.tile_rows - 1) / pl.tile_rows);
  pl.waves = 4;
  int64_t splits;
  if (pl.prompt) {
    // Fewer workgroups than two per CU: eight waves each, two groups over
    // alternate tiles, which halves the time of the longest request (six ragged
    // requests, 408 workgroups of D = 64: 25.8 us against 39.8; seven, 476 of D =
    // 128: 67 against 107; three of one length, 384, are slower, 87 against 78).
    // From 512 on four waves serve better (2048 tokens, 32 heads over 8: 84 us
    // against 93).  Every request is counted with max_q tokens, so these are more
    // than the workgroups that have rows where lengths differ; counted by the tokens
    // in all, some batches gain and some lose (a chunk of 200 among 11 single tokens
    // after 20000: 361 -> 105 us; one of 512 among 15 after 4000: 422 -> 600).  Keys are split while there is less than a workgroup per CU, into
    // parts of 512 keys, or 256 for few rows: the parts' fp32 results are written
    // and read again (512 tokens of 32 heads: 19.9 us in one part, 29.3 in two; 64
    // tokens after 936: 19.8 us in four parts, 23.9 in two).
    pl.chunk = wgs < 64 ? 256 : 512;
    if (wgs < 512) pl.waves = 8;
    splits = wgs > 0 && wgs < 256 ? 256 / wgs : 1;
  } else if (span <= 1536 && wgs < 512) {
    // Short contexts of few requests: eight waves and no join, which costs a launch
    // (1500 tokens, 32 heads over 8: one request 16.2 -> 13.0 us a call, in a graph
    // 11.6 -> 12.5; sixteen 16.8 -> 13.7 and 14.8 -> 13.3).  Later the waves' own
    // steps cost more (2048 tokens, one request: 11.4 us in a graph, 15.0 with eight).
    pl.waves = 8;
    pl.chunk = 1536;
    splits = 1;
  } else {
    // four workgroups to a CU; with as many rows as that anyway, two parts for
    // the long requests of a batch, which would otherwise finish last
    pl.chunk = wgs < 1024 ? 512 : 1024;
    splits = wgs > 0 && wgs < 1024 ? 1024 / wgs : 2;
  }
  const int64_t most = (span + pl.chunk - 1) / pl.chunk;
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  pl.splits = splits < 1 ? 1 : (int)splits;
  if (pl.splits > 1) {
    const int64_t n = T * heads * group;
    pl.sum_offset = (size_t)pl.splits * n * D * 4;
    pl.lo_offset = pl.sum_offset + (size_t)pl.splits * n * 8;
    pl.workspace_bytes = pl.lo_offset + (size_t)pl.splits * n * 4;
  }
  return pl;
}

// The prefix' keys for the T * group rows of all requests, and the requests' own.
KvPrefixPlan kv_prefix_plan(int64_t T, int B, int heads, int group, int D, int max_q, int64_t max_kv, int prefix_len) {
  KvPrefixPlan pl{};
  pl.rest = kv_attention_plan(T, B, heads, group, D, max_q, max_kv > prefix_len ? max_kv - prefix_len : 1, 0, 0);
  if (pl.rest.splits > kMaxSplits / 2) pl.rest.splits = kMaxSplits / 2;
  const int64_t rows = T * group, n = prefix_len;
  KvAttnPlan &sh = pl.shared;
  // Up to 32 rows take the decode kernel (32768 tokens, 32 rows of 8 heads: 31.9 us a call, 39.2 as a
  // prompt's), up to 64 the prompt kernel's tiles of 64 (64 rows of 32 heads: 109 us, 116 in a tile of
  // 128; of 8 heads 42.6, 47.7).
  sh.prompt = rows > 32;
  sh.tile_rows = !sh.prompt ? 16 : rows <= kPtRows / 2 ? kPtRows / 2 : kPtRows;
  sh.waves = 4;
  const int64_t wgs = heads * ((rows + sh.tile_rows - 1) / sh.tile_rows);
  // Two workgroups to a CU: with one, or four, 384 rows of 8 heads over 32768 tokens took 117 and 116 us a
  // call for 102 (32 rows, by the decode kernel: four to a CU 34.3 us, two 31.9).  Parts of 256 keys, since every part's results are
  // written and read again (4096 tokens, 256 rows of 8 heads of 64: 28.1 us, 31.7 with parts of 128), and
  // of 128 where that leaves half the CUs without one (2000 tokens, 128 rows of 8 heads: 24.8 us, 26.7).
  sh.chunk = wgs * ((n + 255) / 256) < 128 ? 128 : 256;
  int64_t splits = 512 / wgs;
  const int64_t most = (n + sh.chunk - 1) / sh.chunk;
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits - pl.rest.splits ? splits : kMaxSplits - pl.rest.splits;
  sh.splits = splits < 1 ? 1 : (int)splits;
  pl.parts = 1;                                       // (as keys_of counts them)
  if (sh.splits > 1) {
    const int64_t want = most < sh.splits ? most : sh.splits;
    const int64_t each = ((n - 1) / want + 64) & -64;
    pl.parts = (int)((n - 1) / each + 1);
  }
  const int64_t results = (pl.parts + pl.rest.splits) * T * heads * group;
  pl.sum_offset = (size_t)results * D * 4;
  pl.lo_offset = pl.sum_offset + (size_t)results * 8;
  pl.workspace_bytes = pl.lo_offset + (size_t)results * 4;
  return pl;
}

// Reading a prefix once saves passes over its keys, in which the kernels' tiles of rows differ: of 16
// (decode) cost 1 a key and head, of a prompt's 64 rows 2, of its 128 rows 3, about 1/35000 us each where the
// card is full (48 requests of up to 4096 tokens, 32 heads of 128: 90 us; half for heads of 64).  It costs two
// launches, 6 us, and that the parts' results are written and read, 4 TB/s.  Calls of 8 requests of 4 tokens
// behind 2000 (32 heads over 8) take 15 us in one pass and 25 in two; 32 single tokens behind 200: 9.5 and 21; 64
// behind 8192 of 32 heads: 275 and 68.  Of 46 calls of all sizes two took the way that was slower by more than 15% (15 requests of 4 tokens behind
// 3630, 64 heads over 8: 42 us for 33).
bool kv_prefix_pays(const KvPrefixPlan &pl, int64_t T, int B, int heads, int group, int D, int max_q, int prefix_len) {
  const int64_t each = (int64_t)max_q * group, all = T * group;
  const int64_t apart = B * (each <= 32 ? (each + 15) / 16 : 3 * ((each + kPtRows - 1) / kPtRows));
  const int64_t once = all <= 32 ? (all + 15) / 16 : all <= kPtRows / 2 ? 2 : 3 * ((all + kPtRows - 1) / kPtRows);
  const double saved = (double)(apart - once) * heads * prefix_len * D / 128 / 35e3;
  return saved > 6.0 + 2.0 * (double)pl.workspace_bytes / 4e6;
}

hipError_t launch_kv_attention(KvAttn p, int B, int D, XType xt, const KvAttnPlan &pl,
                               void *workspace, hipStream_t st) {
  if (pl.splits > 1) {
    p.part_o = reinterpret_cast<float *>(workspace);
    p.part_sum = reinterpret_cast<float2 *>(reinterpret_cast<char *>(workspace) + pl.sum_offset);
    p.part_lo = reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + pl.lo_offset);
  }
  if (p.sinks > 0) return attn_launch_some(p, B, D, xt, pl, st);
  return attn_launch<kAll>(p, B, D, xt, pl, st);
}

hipError_t launch_kv_attention_prefix(KvAttn p, int B, int D, XType xt, const KvPrefixPlan &pl, void *workspace,
                                      hipStream_t st) {
  p.part_o = reinterpret_cast<float *>(workspace);
  p.part_sum = reinterpret_cast<float2 *>(reinterpret_cast<char *>(workspace) + pl.sum_offset);
  p.part_lo = reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + pl.lo_offset);
  p.prefix_parts = pl.parts;
  const hipError_t e = attn_launch_shared(p, D, xt, pl.shared, st);
  return e != hipSuccess ? e : attn_launch_some(p, B, D, xt, pl.rest, st);
}

}  // namespace awq
