// Tree attention on bf16 caches (tree_tc.cuh), and the join of its cut units.
#include "tree_tc.cuh"

namespace prhs {

size_t tree_tc_workspace(const KVView& kv, int max_new, int sms) {
  return tree_record_bytes(kv.d, sms, tc_rows_max(kv, max_new));
}

template <int D>
static cudaError_t tree_go(const TcLaunch& p, const CUtensorMap* maps, int sms, cudaStream_t st) {
  const cudaError_t e = tc_go<D, 0>(p, maps, sms, st);
  return e != cudaSuccess ? e : launch_tree_join<__nv_bfloat16, D, false>(p.a, p.rec, sms, st);
}

prhs_status launch_tree_tc(const TreeLaunch& a, int sms, void* ws, cudaStream_t st, cudaError_t* err) {
  *err = cudaSuccess;
  TcLaunch p;
  CUtensorMap maps[7];
  const prhs_status s = tc_prepare(a, sms, ws, &p, maps);
  if (s == PRHS_OK) *err = a.kv.d == 128 ? tree_go<128>(p, maps, sms, st) : tree_go<64>(p, maps, sms, st);
  return s;
}

}  // namespace prhs
