// Attention with shared keys on bf16 caches: one launch, whose first CTAs run the
// tcgen05 part (tree_tc.cuh) and whose others the few rows' part (few.cuh), and the join
// of its states (shared.cu).
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
