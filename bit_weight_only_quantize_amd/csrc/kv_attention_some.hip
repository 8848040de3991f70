// Attention over the 4-bit cache for some of the keys that rows see: with a window, its
// keys and the first few (sinks); behind a prefix that other launches take, the rest.

#include "kv_attention.h"

namespace awq {

hipError_t attn_launch_some(const KvAttn &p, int B, int D, XType xt, const KvAttnPlan &pl, hipStream_t st) {
  return attn_launch<kSome>(p, B, D, xt, pl, st);
}

}  // namespace awq
