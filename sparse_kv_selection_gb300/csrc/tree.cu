// Attention of a batch of new tokens over their sequences' caches and over
// each other (a tree by its masks, or a causal chunk), fp32 on the CUDA cores
// (the tensor cores' fp32 forms drop mantissa bits).
//
// The G query heads of one KV head see the same keys, so a CTA takes TR rows of
// one (sequence, KV head): row r is token r / G, query head r % G of the group.
// Key tiles of TK rows (the cache's, then the new tokens') pass through shared
// memory; each thread computes 2 rows by 4 keys of the logits, the 16 threads
// of a row pair keep its running maximum and sum (base 2) by shuffles, and the
// weights go through shared memory to the product with V, 2 rows by D / 16
// columns a thread, in fp32 throughout. Where the row blocks are fewer than the
// CTAs that fill the SMs, the key tiles of each are split over several CTAs,
// whose partial states a second launch joins.
#include "tokens.h"

namespace prhs {

constexpr int TR = 32;            // query rows of a CTA
constexpr int TK = 64;            // keys of a tile
constexpr int TREE_THREADS = 256;
constexpr float T_LOG2E = 1.4426950408889634f;
constexpr float T_LN2 = 0.6931471805599453f;

// Splits of a row block's key tiles: enough CTAs for two waves of two an SM,
// while each has a tile of the longest cache.
static int tree_splits(const KVView& kv, long long max_new, int sms) {
  const long long G = kv.Hq / kv.Hkv;
  const long long blocks = ((max_new * G + TR - 1) / TR) * kv.Hkv * kv.B;
  const long long tiles = ((long long)kv.t_max + TK - 1) / TK + 1;
  long long s = 4ll * sms / blocks;
  if (s > tiles) s = tiles;
  return s < 1 ? 1 : (int)s;
}

// Rows of partial records: (row block, split, row).
static size_t tree_records(const KVView& kv, long long max_new, int splits) {
  const long long G = kv.Hq / kv.Hkv;
  return splits == 1 ? 0 : (size_t)(((max_new * G + TR - 1) / TR) * kv.Hkv * kv.B) * splits * TR;
}

size_t tree_workspace(const KVView& kv, int max_new, int sms) {
  const size_t r = tree_records(kv, max_new, tree_splits(kv, max_new, sms));
  return 256 + r * (kv.d + 2) * sizeof(float);
}

template <int D>
struct TreeShape {
  static constexpr int LD = D + 4;  // row stride of Q and K: float4 reads of 8 rows hit distinct banks
  static constexpr size_t SMEM = ((size_t)TR * LD + (size_t)TK * LD + (size_t)TK * D + (size_t)TR * (TK + 1)) * 4;
};

template <int D>
__global__ void __launch_bounds__(TREE_THREADS, 2) tree_kernel(const TreeLaunch a, int splits, float2* rec_ml, float* rec_o) {
  using T = float;
  using S = TreeShape<D>;
  constexpr int E = Elem<T>::per16, PPR = D / E;
  constexpr int OC = D / 64;  // float4 column groups a thread holds
  extern __shared__ __align__(16) float tree_smem[];
  float* sq = tree_smem;
  float* sk = sq + TR * S::LD;
  float* sv = sk + TK * S::LD;
  float* sp = sv + TK * D;  // [TR][TK + 1]
  __shared__ int sh_key[TK];  // 1: the tile's key is attended by someone

  pdl_wait();
  pdl_trigger();
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, kvh = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int block = blockIdx.x / splits, split = blockIdx.x - block * splits;
  const int t = seq_len(kv, b);
  int c0 = 0;
  const int n = seq_tokens(a.cu_new, b, a.T, a.max_new, kv.err, &c0);
  const int r0 = block * TR;
  if (r0 >= n * G) return;
  const int last_tok = min(n, (r0 + TR + G - 1) / G);  // one past the CTA's last token
  const int n_keys = a.mask != nullptr ? n : last_tok;  // new tokens that may be attended

  // ---- Q rows ----
  for (int x = tid; x < TR * PPR; x += TREE_THREADS) {
    const int r = x / PPR, p = x - r * PPR;
    const int j = (r0 + r) / G, g = (r0 + r) % G;
    float f[E];
#pragma unroll
    for (int e = 0; e < E; e++) f[e] = 0.f;
    if (j < n) {
      const T* src = static_cast<const T*>(a.q) + ((long long)(c0 + j) * kv.Hq + kvh * G + g) * D;
      Elem<T>::unpack(reinterpret_cast<const uint4*>(src)[p], f);
    }
#pragma unroll
    for (int e = 0; e < E; e++) sq[r * S::LD + p * E + e] = f[e];
  }

  const int ty = tid >> 4, tx = tid & 15;  // rows 2 ty, 2 ty + 1; keys tx + 16 i
  const float qs = a.scale * T_LOG2E;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[2][OC * 4];
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int c = 0; c < OC * 4; c++) o[i][c] = 0.f;

  const int cache_tiles = (t + TK - 1) / TK, new_tiles = (n_keys + TK - 1) / TK;
  const int per = (cache_tiles + new_tiles + splits - 1) / splits;
  const int it_end = min(cache_tiles + new_tiles, (split + 1) * per);
  for (int it = split * per; it < it_end; it++) {
    const bool cached = it < cache_tiles;
    const int key0 = (cached ? it : it - cache_tiles) * TK;
    const int lim = cached ? t : n_keys;
    __syncthreads();
    for (int x = tid; x < TK * PPR; x += TREE_THREADS) {
      const int key = x / PPR, p = x - key * PPR, i = key0 + key;
      float kf[E], vf[E];
#pragma unroll
      for (int e = 0; e < E; e++) kf[e] = vf[e] = 0.f;
      bool have = i < lim;
      if (have) {
        const T *ks, *vs;
        if (cached) {
          const long long row = kv_row(kv, b, kvh, i);
          if (row < 0) {
            raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
            have = false;
          }
          ks = static_cast<const T*>(kv.k) + row * D;
          vs = static_cast<const T*>(kv.v) + row * D;
        } else {
          ks = static_cast<const T*>(a.k_new) + (c0 + i) * a.ks + kvh * D;
          vs = static_cast<const T*>(a.v_new) + (c0 + i) * a.vs + kvh * D;
        }
        if (have) {
          Elem<T>::unpack(reinterpret_cast<const uint4*>(ks)[p], kf);
          Elem<T>::unpack(reinterpret_cast<const uint4*>(vs)[p], vf);
        }
      }
      if (p == 0) sh_key[key] = have;
#pragma unroll
      for (int e = 0; e < E; e++) {
        sk[key * S::LD + p * E + e] = kf[e];
        sv[key * D + p * E + e] = vf[e];
      }
    }
    __syncthreads();
    float acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int k = 0; k < 4; k++) acc[i][k] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      const float4 q0 = *reinterpret_cast<const float4*>(sq + (2 * ty) * S::LD + e);
      const float4 q1 = *reinterpret_cast<const float4*>(sq + (2 * ty + 1) * S::LD + e);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float4 x = *reinterpret_cast<const float4*>(sk + (tx + 16 * k) * S::LD + e);
        acc[0][k] = fmaf(q0.x, x.x, fmaf(q0.y, x.y, fmaf(q0.z, x.z, fmaf(q0.w, x.w, acc[0][k]))));
        acc[1][k] = fmaf(q1.x, x.x, fmaf(q1.y, x.y, fmaf(q1.z, x.z, fmaf(q1.w, x.w, acc[1][k]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int r = 2 * ty + i, j = (r0 + r) / G;
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int key = tx + 16 * k, p = key0 + key;
        bool see = sh_key[key] != 0;
        if (see && !cached)
          see = a.mask == nullptr ? p <= j
                                  : j < n && (a.mask[(long long)(c0 + j) * PRHS_TREE_WORDS + (p >> 5)] >> (p & 31)) & 1u;
        acc[i][k] = see ? acc[i][k] * qs : -INFINITY;
        mx = fmaxf(mx, acc[i][k]);
      }
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, s));
      mx = fmaxf(m[i], mx);
      const float corr = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mx);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float w = mx == -INFINITY ? 0.f : exp2f(acc[i][k] - mx);
        sum += w;
        sp[r * (TK + 1) + tx + 16 * k] = w;
      }
      l[i] = l[i] * corr + sum;
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < OC * 4; c++) o[i][c] *= corr;
    }
    __syncwarp();  // a row pair's weights are written and read by one half warp
#pragma unroll 4
    for (int key = 0; key < TK; key++) {
      const float w0 = sp[(2 * ty) * (TK + 1) + key], w1 = sp[(2 * ty + 1) * (TK + 1) + key];
#pragma unroll
      for (int c = 0; c < OC; c++) {
        const float4 x = *reinterpret_cast<const float4*>(sv + key * D + c * 64 + tx * 4);
        o[0][4 * c] = fmaf(w0, x.x, o[0][4 * c]);
        o[0][4 * c + 1] = fmaf(w0, x.y, o[0][4 * c + 1]);
        o[0][4 * c + 2] = fmaf(w0, x.z, o[0][4 * c + 2]);
        o[0][4 * c + 3] = fmaf(w0, x.w, o[0][4 * c + 3]);
        o[1][4 * c] = fmaf(w1, x.x, o[1][4 * c]);
        o[1][4 * c + 1] = fmaf(w1, x.y, o[1][4 * c + 1]);
        o[1][4 * c + 2] = fmaf(w1, x.z, o[1][4 * c + 2]);
        o[1][4 * c + 3] = fmaf(w1, x.w, o[1][4 * c + 3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int r = r0 + 2 * ty + i, j = r / G, g = r % G;
    float sum = l[i];
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, s);
    if (j >= n) continue;
    if (splits > 1) {  // a partial record (m, l and O against m)
      const long long rec = ((((long long)b * kv.Hkv + kvh) * (gridDim.x / splits) + block) * splits + split) * TR + 2 * ty + i;
#pragma unroll
      for (int c = 0; c < OC; c++)
        *reinterpret_cast<float4*>(rec_o + rec * D + c * 64 + tx * 4) =
            make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
      if (tx == 0) rec_ml[rec] = make_float2(m[i], sum);
      continue;
    }
    const long long orow = (long long)(c0 + j) * kv.Hq + kvh * G + g;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int c = 0; c < OC; c++) {
      *reinterpret_cast<float4*>(static_cast<T*>(a.out) + orow * D + c * 64 + tx * 4) =
          make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv);
    }
    if (tx == 0) a.lse[orow] = sum > 0.f ? (m[i] + log2f(sum)) * T_LN2 : -INFINITY;
  }
}

// One warp per row joins its splits' records.
constexpr int TREE_JOIN_WARPS = 4;
template <int D>
__global__ void __launch_bounds__(TREE_JOIN_WARPS * 32) tree_join_f32_kernel(const TreeLaunch a, int splits, int blocks,
                                                                             const float2* rec_ml, const float* rec_o) {
  pdl_wait();
  pdl_trigger();
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, kvh = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  int c0 = 0;
  const int n = seq_tokens(a.cu_new, b, a.T, a.max_new, kv.err, &c0);
  const int row = blockIdx.x * TREE_JOIN_WARPS + (threadIdx.x >> 5);
  if (row >= n * G) return;
  const long long rec0 = ((((long long)b * kv.Hkv + kvh) * blocks + row / TR) * splits) * TR + row % TR;
  float M = -INFINITY;
  for (int i = lane; i < splits; i += 32) M = fmaxf(M, __ldcg(rec_ml + rec0 + (long long)i * TR).x);
  M = warp_max(M);
  constexpr int F = D / 32;
  float L = 0.f, o[F];
#pragma unroll
  for (int f = 0; f < F; f++) o[f] = 0.f;
  if (M != -INFINITY) {
#pragma unroll 8
    for (int i = 0; i < splits; i++) {
      const long long rec = rec0 + (long long)i * TR;
      const float2 ml = __ldcg(rec_ml + rec);
      const float wt = exp2f(ml.x - M);  // 0 where the split had nothing
      L += wt * ml.y;
#pragma unroll
      for (int f = 0; f < F; f++) o[f] += wt * __ldcg(rec_o + rec * D + f * 32 + lane);
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const long long orow = (long long)(c0 + row / G) * kv.Hq + kvh * G + row % G;
#pragma unroll
  for (int f = 0; f < F; f++) static_cast<float*>(a.out)[orow * D + f * 32 + lane] = o[f] * inv;
  if (lane == 0) a.lse[orow] = L > 0.f ? (M + log2f(L)) * T_LN2 : -INFINITY;
}

template <int D>
static cudaError_t tree_go(const TreeLaunch& a, int splits, float2* rec_ml, float* rec_o, cudaStream_t st) {
  auto k = tree_kernel<D>;
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(k, TreeShape<D>::SMEM, smem_set);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.max_new * (a.kv.Hq / a.kv.Hkv);
  const unsigned blocks = (unsigned)((rows + TR - 1) / TR);
  e = launch_pdl(k, dim3(blocks * splits, a.kv.Hkv, a.kv.B), dim3(TREE_THREADS), TreeShape<D>::SMEM, st, a.kv.pdl, a, splits,
                 rec_ml, rec_o);
  if (e != cudaSuccess || splits == 1) return e;
  abi_count_launch();
  return launch_pdl(tree_join_f32_kernel<D>, dim3((unsigned)((rows + TREE_JOIN_WARPS - 1) / TREE_JOIN_WARPS), a.kv.Hkv, a.kv.B),
                    dim3(TREE_JOIN_WARPS * 32), 0, st, true, a, splits, (int)blocks, (const float2*)rec_ml, (const float*)rec_o);
}

cudaError_t launch_tree(const TreeLaunch& a, int max_new, int sms, void* ws, cudaStream_t st) {
  // (the workspace was sized for max_new, of which a.max_new is what T leaves)
  const int splits = tree_splits(a.kv, max_new, sms);
  float2* ml = static_cast<float2*>(ws);
  float* o = reinterpret_cast<float*>(static_cast<char*>(ws) + (tree_records(a.kv, max_new, splits) * 8 + 255) / 256 * 256);
  return a.kv.d == 128 ? tree_go<128>(a, splits, ml, o, st) : tree_go<64>(a, splits, ml, o, st);
}

}  // namespace prhs
