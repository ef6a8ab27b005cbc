// Joins the two partial states of tokens whose sequences share leading keys: the
// one against the shared keys, which one pass over them gave for all the group's
// tokens, and the one against the sequence's other keys.
//
//   m = max(m1, m2),  o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2)
//
// A thread takes four columns of a row; the CTAs of a sequence share its rows.
// Bound: L2 and latency (the states are 2 (4 d + 8) bytes a row, just written).
#include "tree_join.cuh"

namespace prhs {

constexpr int SJ_THREADS = 256, SJ_PER = 4;

template <typename T, int D>
__global__ void __launch_bounds__(SJ_THREADS) shared_join_kernel(const __grid_constant__ TreeLaunch a) {
  constexpr int C4 = D / 4;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  const TreeItem x = tree_item<true>(a, 2 * b + 1);
  if (x.part != 2 || *a.part_ok == 0) return;
  const long long total = (long long)x.n * a.kv.Hq * C4, row0 = (long long)x.c0 * a.kv.Hq, other = tree_part_row(a, 2, 0);
  for (long long i0 = (long long)blockIdx.y * SJ_THREADS * SJ_PER + threadIdx.x; i0 < total;
       i0 += (long long)gridDim.y * SJ_THREADS * SJ_PER) {
    float2 ml[SJ_PER][2];
    float4 o[SJ_PER][2];
#pragma unroll
    for (int k = 0; k < SJ_PER; k++) {
      const long long i = min(i0 + k * SJ_THREADS, total - 1), row = row0 + i / C4;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        ml[k][h] = __ldcg(a.part_ml + row + h * other);
        o[k][h] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (row + h * other) * C4 + i % C4);
      }
    }
#pragma unroll
    for (int k = 0; k < SJ_PER; k++) {
      const long long i = i0 + k * SJ_THREADS, row = row0 + i / C4;
      if (i >= total) break;
      const float M = fmaxf(ml[k][0].x, ml[k][1].x);
      const float w0 = tree_weight(ml[k][0].x, M), w1 = tree_weight(ml[k][1].x, M);
      // (a state that holds NaN has it in its sum, whatever its maximum)
      const float L = fmaf(w1, ml[k][1].y, w0 * ml[k][0].y), inv = tree_inv(L);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      tree_fma(y, w0, o[k][0]);
      tree_fma(y, w1, o[k][1]);
      tree_put(static_cast<T*>(a.out) + row * D + i % C4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (i % C4 == 0) a.lse[row] = tree_lse(M, L);
    }
  }
}

template <typename T>
static cudaError_t shared_go(const TreeLaunch& a, cudaStream_t st) {
  const long long pass = (long long)SJ_THREADS * SJ_PER, y = ((long long)a.max_new * a.kv.Hq * a.kv.d / 4 + pass - 1) / pass;
  const dim3 grid(a.kv.B, (unsigned)(y < 64 ? y : 64));
  if (a.kv.d == 128) return launch_pdl(shared_join_kernel<T, 128>, grid, dim3(SJ_THREADS), 0, st, true, a);
  return launch_pdl(shared_join_kernel<T, 64>, grid, dim3(SJ_THREADS), 0, st, true, a);
}

cudaError_t launch_shared_join(const TreeLaunch& a, cudaStream_t st) {
  return a.kv.dtype == PRHS_BF16 ? shared_go<__nv_bfloat16>(a, st) : shared_go<float>(a, st);
}

}  // namespace prhs
