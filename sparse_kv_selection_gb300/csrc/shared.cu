// The last launch of the attention that reads shared prefixes once. A token of a
// group has two states, one against the shared keys (one pass over them gave it for
// all the group's tokens) and one against its sequence's other keys:
//
//   m = max(m1, m2),  o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2)
//
// On bf16 each may lie in pieces, one for each CTA or warp of the launch before that had
// a run of its unit's keys (`where`: the first, how many). A thread takes four columns of
// a row; eight consecutive rows are neighbours, as the pieces keep them. Bound: L2
// and latency (where, then the states).
#include "tree_join.cuh"

namespace prhs {

constexpr int SJ_THREADS = 256;

template <typename T, int D>
__global__ void __launch_bounds__(SJ_THREADS) shared_join_kernel(const __grid_constant__ TreeLaunch a,
                                                                 const __grid_constant__ TreeRecords rec, int ctas) {
  constexpr int C4 = D / 4;
  pdl_wait();
  pdl_trigger();
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, gl = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3, b = blockIdx.x;
  const TreeItem x = tree_item<true>(a, 2 * b + 1, true);
  const bool few = few_item(a, x.n, x.t);
  if (x.n == 0 || (sizeof(T) == 4 && x.part != 2) || *a.part_ok == 0) return;
  // the group's first token (its units of the shared keys count rows from there)
  const int group0 = x.part == 2 ? max(0, a.cu_new[a.shared[b].x]) : 0;
  const int rows = x.n << gl, blocks = (rows + 7) / 8;
  const long long total = (long long)kv.Hkv * blocks * 8 * C4;
  for (long long i = (long long)blockIdx.y * SJ_THREADS + threadIdx.x; i < total; i += (long long)gridDim.y * SJ_THREADS) {
    const int in = (int)i & 7, c4 = (int)(i / 8 % C4), hr = (int)(i / (8 * C4)), kvh = hr / blocks, r = (hr - kvh * blocks) * 8 + in;
    if (r >= rows) continue;
    const int tok = x.c0 + (r >> gl), h = r & (G - 1);
    int2 at[2] = {make_int2(0, 1), make_int2(0, 1)};  // of the states against the shared and the other keys
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 2; k++)
        if (k == 1 || x.part == 2) at[k] = __ldcg(a.where + part_row<T>(a, k + 1, tok, kvh, h, gl));
    }
    if (x.part != 2 && at[1].y == 1) continue;  // its result stands
    float M = -INFINITY, L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 o) {  // (a state that holds NaN has it in its sum, whatever its maximum)
      const float m = fmaxf(M, ml.x), w0 = tree_weight(M, m), w1 = tree_weight(ml.x, m);
      L = fmaf(w1, ml.y, w0 * L);
      y = make_float4(y.x * w0, y.y * w0, y.z * w0, y.w * w0);
      tree_fma(y, w1, o);
      M = m;
    };
#pragma unroll
    for (int k = 0; k < 2; k++) {
      if (k == 0 && x.part != 2) continue;
      if (at[k].y == 1) {
        add(__ldcg(a.part_ml + part_row<T>(a, k + 1, tok, kvh, h, gl)), __ldcg(part_at<T, D>(a, k + 1, tok, kvh, h, c4, gl)));
        continue;
      }
      if constexpr (sizeof(T) == 2) {
        // piece w: the first writer's second slot, the others' first ones; rows as their unit counts them
        const bool warps = k == 1 && few;
        const int writers = warps ? a.few_warps : ctas, unit = warps ? a.few_rows : 256;
        const int first = max(0, min(at[k].x, writers - 1)), n = max(1, min(at[k].y, writers - first));
        const int row = (k == 0 ? ((tok - group0) << gl) + h : r) & (unit - 1);
        const float2* ml = warps ? reinterpret_cast<const float2*>(static_cast<const float4*>(a.few_states) +
                                                                   (long long)2 * writers * C4 * unit)
                                 : rec.ml;
        const float4* o = warps ? static_cast<const float4*>(a.few_states) : rec.o;
        const int stride = warps ? unit : rec.rows_max;
#pragma unroll 4
        for (int w = 0; w < n; w++) {
          const long long slot = 2ll * (first + w) + (w == 0);
          add(__ldcg(ml + slot * stride + row), __ldcg(o + (slot * C4 + c4) * stride + row));
        }
      }
    }
    const float inv = tree_inv(L);
    const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
    tree_put(static_cast<T*>(a.out) + orow * D + c4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    if (c4 == 0) a.lse[orow] = tree_lse(M, L);
  }
}

template <typename T, int D>
static cudaError_t join_go(const TreeLaunch& a, const TreeRecords& rec, int sms, cudaStream_t st) {
  const long long rows = ((long long)a.max_new * (a.kv.Hq / a.kv.Hkv) + 7) / 8 * 8;
  const long long y = (rows * a.kv.Hkv * D / 4 + SJ_THREADS - 1) / SJ_THREADS;
  return launch_pdl(shared_join_kernel<T, D>, dim3(a.kv.B, (unsigned)(y < 256 ? y : 256)), dim3(SJ_THREADS), 0, st, true, a, rec, sms);
}
cudaError_t launch_shared_join(const TreeLaunch& a, const TreeRecords& rec, int sms, cudaStream_t st) {
  if (a.kv.dtype == PRHS_BF16)
    return a.kv.d == 128 ? join_go<__nv_bfloat16, 128>(a, rec, sms, st) : join_go<__nv_bfloat16, 64>(a, rec, sms, st);
  return a.kv.d == 128 ? join_go<float, 128>(a, rec, sms, st) : join_go<float, 64>(a, rec, sms, st);
}

}  // namespace prhs
