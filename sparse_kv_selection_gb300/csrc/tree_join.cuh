// Joins the partial states that tree attention leaves of the units cut by a
// run's end (the last unit that a CTA of the main launch begins or carries on and
// does not finish).
#pragma once

#include "tokens.h"

namespace prhs {

// What a CTA's run leaves behind: the unit that does not end in it.
struct __align__(16) TreeSplit {
  int rows, kvh, tok, n_rec;  // rows of the unit (0: none), KV head, first token (packed), records
  int first, part, pad[2];    // the CTA that begins it; where its state goes (TreeItem)
};

// Partial states: the running maximum (base 2), the sum and O against that
// maximum. Record 2 c + 1 is of the unit that CTA c begins, 2 c of one begun before.
struct TreeRecords {
  int group_log2;    // log2 of the query heads of a KV head
  int rows_max;      // rows a record may hold
  int cta0;          // the launch's first CTA
  TreeSplit* split;  // [CTAs]
  float2* ml;        // [2 CTAs][rows_max]
  float4* o;         // [2 CTAs][rows_max][D / 4] (ROW_MAJOR) or [2 CTAs][D / 4][rows_max]
};

// A thread takes four columns of a row (T: the result's type). A unit's records
// are those of its CTAs, which have consecutive numbers; the thread blocks of all of
// them but the last share its elements. Records are read as the main launch finds it
// cheapest to write them, neighbouring threads neighbouring elements either way. Of
// many records, 2, 4 or 16 groups of threads take a share each.
// Bound: L2 and latency.
constexpr int JOIN_THREADS = 256, JOIN_CH = 4;  // (records in flight)

// Results of a row from its maximum M (base 2) and sum L: 0 and -inf where it attends
// nothing (L = 0); NaN in the query or an attended key makes L and O NaN, and M what
// the other keys leave.
__device__ __forceinline__ float tree_inv(float L) { return L == 0.f ? 0.f : 1.f / L; }
__device__ __forceinline__ float tree_lse(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Weight of a state with maximum x against m (0 where it has nothing in it).
__device__ __forceinline__ float tree_weight(float x, float m) { return x == -INFINITY ? 0.f : exp2f(x - m); }
__device__ __forceinline__ void tree_fma(float4& o, float w, float4 x) {
  o = make_float4(fmaf(w, x.x, o.x), fmaf(w, x.y, o.y), fmaf(w, x.z, o.z), fmaf(w, x.w, o.w));
}
__device__ __forceinline__ void tree_put(float* dst, float4 x) { *reinterpret_cast<float4*>(dst) = x; }
__device__ __forceinline__ void tree_put(__nv_bfloat16* dst, float4 x) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Where a row's partial state is kept: its maximum and sum, and its columns 4 c .. 4 c + 3.
template <typename T>
__device__ __forceinline__ long long part_row(const TreeLaunch& a, int part, long long tok, int kvh, int g, int gl) {
  const TreeLaunch& x = a;
  if (sizeof(T) == 4) return ((long long)(part - 1) * x.T + tok) * x.kv.Hq + (kvh << gl) + g;
  return ((long long)(part - 1) * x.kv.Hkv + kvh) * ((long long)x.T << gl) + (tok << gl) + g;
}
template <typename T, int D>
__device__ __forceinline__ float4* part_at(const TreeLaunch& a, int part, long long tok, int kvh, int g, int c, int gl) {
  float4* o = reinterpret_cast<float4*>(a.part_o);
  if (sizeof(T) == 4) return o + part_row<T>(a, part, tok, kvh, g, gl) * (D / 4) + c;
  return o + (((long long)(part - 1) * a.kv.Hkv + kvh) * (D / 4) + c) * ((long long)a.T << gl) + (tok << gl) + g;
}

template <typename T, int D, bool ROW_MAJOR>
__global__ void __launch_bounds__(JOIN_THREADS) tree_join_kernel(const __grid_constant__ TreeLaunch a,
                                                                 const __grid_constant__ TreeRecords p) {
  constexpr int C4 = D / 4, CH = JOIN_CH;
  __shared__ float4 so[JOIN_THREADS];
  __shared__ float2 sml[JOIN_THREADS];
  pdl_wait();
  pdl_trigger();
  const TreeSplit s = p.split[blockIdx.x];
  if (s.rows == 0) return;
  const int ways = s.n_rec <= CH ? 1 : s.n_rec <= 2 * CH ? 2 : s.n_rec <= 8 * CH ? 4 : 16, step = JOIN_THREADS / ways;
  const int way = threadIdx.x / step, in = threadIdx.x % step;
  const int slot = ((int)blockIdx.x - s.first) * gridDim.y + blockIdx.y, slots = (s.n_rec - 1) * gridDim.y;
  const int total = s.rows * C4;
  for (int i0 = slot * step; i0 < total; i0 += slots * step) {
    const int i = min(i0 + in, total - 1);  // (threads behind the last repeat it)
    const int row = ROW_MAJOR ? i / C4 : i % s.rows, c = ROW_MAJOR ? i % C4 : i / s.rows;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r0 = way; r0 < s.n_rec; r0 += CH * ways) {
      float2 ml[CH];
      float4 x[CH];
#pragma unroll
      for (int k = 0; k < CH; k++) {
        const int r = r0 + k * ways;
        const long long rec = r == 0 ? 2ll * s.first + 1 : 2ll * (s.first + r);
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < s.n_rec) {
          ml[k] = __ldcg(p.ml + rec * p.rows_max + row);
          x[k] = __ldcg(p.o + (ROW_MAJOR ? (rec * p.rows_max + row) * C4 + c : (rec * C4 + c) * p.rows_max + row));
        }
      }
      float m = M;
#pragma unroll
      for (int k = 0; k < CH; k++) m = fmaxf(m, ml[k].x);
      const float corr = tree_weight(M, m);
      L *= corr;
      o = make_float4(o.x * corr, o.y * corr, o.z * corr, o.w * corr);
#pragma unroll
      for (int k = 0; k < CH; k++) {
        const float w = tree_weight(ml[k].x, m);
        L = fmaf(w, ml[k].y, L);
        tree_fma(o, w, x[k]);
      }
      M = m;
    }
    if (ways > 1) {
      __syncthreads();  // (the elements before are done with)
      so[threadIdx.x] = o;
      sml[threadIdx.x] = make_float2(M, L);
      __syncthreads();
      if (way != 0) continue;
      for (int w = in; w < JOIN_THREADS; w += step) M = fmaxf(M, sml[w].x);
      L = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = in; w < JOIN_THREADS; w += step) {
        const float2 ml = sml[w];
        const float wt = tree_weight(ml.x, M);
        L = fmaf(wt, ml.y, L);
        tree_fma(o, wt, so[w]);
      }
    }
    if (i0 + in >= total) continue;
    const int gl = p.group_log2;
    const float inv = tree_inv(L);
    const long long orow = (long long)(s.tok + (row >> gl)) * a.kv.Hq + (s.kvh << gl) + (row & ((1 << gl) - 1));
    if (sizeof(T) == 4 && s.part != 0) {
      const int tok = s.tok + (row >> gl), g = row & ((1 << gl) - 1);
      *part_at<T, D>(a, s.part, tok, s.kvh, g, c, gl) = o;
      if (c == 0) a.part_ml[part_row<T>(a, s.part, tok, s.kvh, g, gl)] = make_float2(M, L);
      continue;
    }
    tree_put(static_cast<T*>(a.out) + orow * D + c * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (c == 0) a.lse[orow] = tree_lse(M, L);
  }
}

template <typename T, int D, bool ROW_MAJOR>
cudaError_t launch_tree_join(const TreeLaunch& a, const TreeRecords& p, unsigned ctas, cudaStream_t st) {
  const int y = p.rows_max * (D / 4) / JOIN_THREADS;  // a pass over a record of rows_max rows, eight at most
  return launch_pdl(tree_join_kernel<T, D, ROW_MAJOR>, dim3(ctas, y < 1 ? 1 : y > 8 ? 8 : y), dim3(JOIN_THREADS), 0, st, true, a, p);
}

// Workspace of `ctas` runs, and its parts.
inline size_t tree_up(size_t x) { return (x + 255) / 256 * 256; }
inline size_t tree_record_bytes(int d, size_t ctas, size_t rows_max) {
  return tree_up(ctas * sizeof(TreeSplit)) + tree_up(2 * ctas * rows_max * sizeof(float2)) + 2 * ctas * rows_max * d * sizeof(float);
}
inline TreeRecords tree_records(void* ws, int group_log2, size_t ctas, int rows_max) {
  TreeRecords p;
  char* w = static_cast<char*>(ws);
  p.group_log2 = group_log2;
  p.rows_max = rows_max;
  p.cta0 = 0;
  p.split = reinterpret_cast<TreeSplit*>(w);
  w += tree_up(ctas * sizeof(TreeSplit));
  p.ml = reinterpret_cast<float2*>(w);
  w += tree_up(2 * ctas * rows_max * sizeof(float2));
  p.o = reinterpret_cast<float4*>(w);
  return p;
}

}  // namespace prhs
