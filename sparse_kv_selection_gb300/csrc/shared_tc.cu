// Attention with shared keys on bf16 caches: one launch, whose first CTAs run the
// tcgen05 part (tree_tc.cuh) and whose others the few rows' part (few.cuh), and the join
// of its states (shared.cu). From a graph: 16 samples of 4096 keys, 32 heads, 36.5 us (bytes 14);
// 128 tokens in 8 groups of 3.7 to 5K keys with up to 3K own ones, 32 / 8 heads, 16-key pages,
// 80 (48); 32 drafts on 2K shared keys 118 (89); 32 questions on one prefix of 131072 keys, 115
// (85); 913 prompt tokens of 24 sequences on 8192 keys 128 (65, the flops).
// Each list's CTAs are as many as its work takes, a unit's beginning and end counted (REST,
// FEW_REST). Bound by those ends: 3 to 4 us a tile unit, which one CTA does not overlap, 2 to 3 us
// of dependent reads before a warp's first keys, and the join.
#include "tree_tc.cuh"

namespace prhs {

void few_shape(TreeLaunch* a, int sms) {
  if (a->kv.dtype != PRHS_BF16) return;
  a->few_rows = (long long)a->max_new * (a->kv.Hq / a->kv.Hkv) <= 8 ? 8 : 16;
  a->few_warps = FEW_WARPS * sms;
}
size_t few_state_bytes(const KVView& kv, int sms) {
  if (kv.dtype != PRHS_BF16) return 0;
  return (size_t)2 * FEW_WARPS * sms * 16 * (kv.d * sizeof(float) + sizeof(float2));
}
size_t shared_where_bytes(const KVView& kv, int T) {
  return kv.dtype != PRHS_BF16 ? 0 : (size_t)2 * T * kv.Hq * sizeof(int2);
}

prhs_status launch_shared_tc(const TreeLaunch& a, int sms, void* ws, cudaStream_t st, cudaError_t* err) {
  *err = cudaSuccess;
  TcLaunch p;
  CUtensorMap maps[7];
  const prhs_status s = tc_prepare(a, sms, ws, &p, maps);
  if (s != PRHS_OK) return s;
  cudaError_t e;
  if (a.few_rows == 8) e = a.kv.d == 128 ? tc_go<128, 1>(p, maps, sms, st) : tc_go<64, 1>(p, maps, sms, st);
  else e = a.kv.d == 128 ? tc_go<128, 2>(p, maps, sms, st) : tc_go<64, 2>(p, maps, sms, st);
  *err = e != cudaSuccess ? e : launch_shared_join(a, p.rec, sms, st);
  return PRHS_OK;
}

}  // namespace prhs
