// Rotary positions on the q and k of a batch of tokens, with the cache append.
//
// A pair (x, y) of a head's rotated elements becomes (x c - y s, x s + y c),
// c and s the cosine and sine of position * theta. The angle is taken in turns
// as a 64-bit binary fraction: position * turns modulo 2^64 wraps exactly where
// the angle does, so it is as exact at position 2^31 as at 1, without float64
// (whose rate is low on this part) and without a range reduction. Its top 32
// bits, read as a signed number, are the angle in [-1/2, 1/2) turns to 2^-33.
//
// Every head of a token takes the same rot_dim / 2 angles, so a CTA computes
// them once into shared memory. The work is cut into tasks of two 16-byte
// pieces of one head row (the two halves of E pairs, E elements a piece, or
// two pieces that are only copied), PER tasks a thread: the loads are issued
// before the angles are computed, which hides one behind the other.
//
// Bound: HBM, each element read once and written once.
#include "tokens.h"

namespace prhs {

constexpr int ROPE_THREADS = 256;

template <typename T>
__device__ __forceinline__ uint4 pack_piece(const float* f);
template <>
__device__ __forceinline__ uint4 pack_piece<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack_piece<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int PER>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeLaunch a, int rows, int tpr) {
  constexpr int E = Elem<T>::per16;
  extern __shared__ __align__(16) float2 rope_cs[];  // [tokens of this CTA][rot_dim / 2]
  pdl_wait();
  pdl_trigger();
  const KVView& kv = a.kv;
  const int half = a.rot_dim / 2, rot_tasks = half / E;
  const long long total = (long long)a.T * rows * tpr;
  const long long x0 = (long long)blockIdx.x * (ROPE_THREADS * PER);
  const int tok0 = (int)(x0 / (rows * tpr));
  const int tok1 = (int)((min(total, x0 + ROPE_THREADS * PER) - 1) / (rows * tpr));

  uint4 lo[PER], hi[PER];
  int tok[PER], row[PER], x[PER], p0[PER], p1[PER];
#pragma unroll
  for (int u = 0; u < PER; u++) {
    const long long g = x0 + u * ROPE_THREADS + threadIdx.x;
    tok[u] = -1;
    if (g < total) {
      const int rem = (int)(g - (long long)tok0 * rows * tpr);  // from the CTA's first token
      const int r = rem / tpr;
      x[u] = rem - r * tpr;
      const int k = r / rows;
      row[u] = r - k * rows;
      tok[u] = tok0 + k;
      const bool rotated = x[u] < rot_tasks;
      p0[u] = rotated && !a.interleaved ? x[u] : 2 * x[u];
      p1[u] = rotated && !a.interleaved ? x[u] + rot_tasks : 2 * x[u] + 1;
      const T* src;
      if (row[u] < kv.Hq) src = static_cast<const T*>(a.q) + tok[u] * a.qs + (long long)row[u] * kv.d;
      else if (row[u] < kv.Hq + kv.Hkv) src = static_cast<const T*>(a.k) + tok[u] * a.ks + (long long)(row[u] - kv.Hq) * kv.d;
      else src = static_cast<const T*>(a.v) + tok[u] * a.vs + (long long)(row[u] - kv.Hq - kv.Hkv) * kv.d;
      lo[u] = reinterpret_cast<const uint4*>(src)[p0[u]];
      hi[u] = reinterpret_cast<const uint4*>(src)[p1[u]];
    }
  }

  for (int i = threadIdx.x; i < (tok1 - tok0 + 1) * half; i += ROPE_THREADS) {
    const int k = i / half, f = i - k * half;
    const uint64_t turn = (uint64_t)(int64_t)a.positions[tok0 + k] * a.turns[f];
    // half turns in [-1, 1)
    const float ht = (float)(int32_t)(turn >> 32) * 0x1p-31f;
    float s, c;
    sincospif(ht, &s, &c);
    rope_cs[i] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < PER; u++) {
    if (tok[u] < 0) continue;
    int slot = 0;
    if (a.slots != nullptr) {
      slot = a.slots[tok[u]];
      const int slots = kv.block_table != nullptr ? kv.num_blocks * kv.block_size : kv.B * kv.t_max;
      if (slot < 0 || slot >= slots) {
        if (slot != -1) raise_error(kv.err, PRHS_DEV_BAD_INDEX);
        continue;
      }
    }
    if (x[u] < rot_tasks && row[u] < kv.Hq + kv.Hkv) {
      float e0[E], e1[E];
      Elem<T>::unpack(lo[u], e0);
      Elem<T>::unpack(hi[u], e1);
      const float2* cs = rope_cs + (tok[u] - tok0) * half + x[u] * E;
      if (!a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; e++) {
          const float2 t = cs[e];
          const float r0 = e0[e] * t.x - e1[e] * t.y;
          e1[e] = e0[e] * t.y + e1[e] * t.x;
          e0[e] = r0;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          const float2 t = cs[e], w = cs[E / 2 + e];
          const float r0 = e0[2 * e] * t.x - e0[2 * e + 1] * t.y;
          e0[2 * e + 1] = e0[2 * e] * t.y + e0[2 * e + 1] * t.x;
          e0[2 * e] = r0;
          const float r1 = e1[2 * e] * w.x - e1[2 * e + 1] * w.y;
          e1[2 * e + 1] = e1[2 * e] * w.y + e1[2 * e + 1] * w.x;
          e1[2 * e] = r1;
        }
      }
      lo[u] = pack_piece<T>(e0);
      hi[u] = pack_piece<T>(e1);
    }
    if (row[u] < kv.Hq) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + ((long long)tok[u] * kv.Hq + row[u]) * kv.d);
      dst[p0[u]] = lo[u];
      dst[p1[u]] = hi[u];
      continue;
    }
    const bool is_k = row[u] < kv.Hq + kv.Hkv;
    const int h = row[u] - kv.Hq - (is_k ? 0 : kv.Hkv);
    if (is_k && a.k_out != nullptr) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + ((long long)tok[u] * kv.Hkv + h) * kv.d);
      dst[p0[u]] = lo[u];
      dst[p1[u]] = hi[u];
    }
    if (a.slots != nullptr) {
      int head_rows;
      const long long r = slot_row(kv, slot, &head_rows) + (long long)h * head_rows;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(const_cast<void*>(is_k ? kv.k : kv.v)) + r * kv.d);
      dst[p0[u]] = lo[u];
      dst[p1[u]] = hi[u];
    }
  }
}

template <typename T, int PER>
static cudaError_t rope_go(const RopeLaunch& a, cudaStream_t st) {
  constexpr int E = Elem<T>::per16;
  const int rows = a.kv.Hq + (a.slots != nullptr ? 2 : 1) * a.kv.Hkv;
  const int tpr = a.kv.d / (2 * E);
  const long long total = (long long)a.T * rows * tpr;
  const int chunk = ROPE_THREADS * PER;
  // tokens a CTA may touch: its whole ones and one cut at each end
  const long long toks = (chunk + rows * tpr - 1) / (rows * tpr) + 1;
  const size_t smem = (size_t)(toks < a.T ? toks : a.T) * (a.rot_dim / 2) * sizeof(float2);
  auto k = rope_kernel<T, PER>;
  static int smem_set[SMEM_DEVICES];
  const cudaError_t e = allow_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)((total + chunk - 1) / chunk)), dim3(ROPE_THREADS), smem, st, a.kv.pdl, a,
                    rows, tpr);
}

cudaError_t launch_rope(const RopeLaunch& a, int sms, cudaStream_t st) {
  const int es = a.kv.dtype == PRHS_BF16 ? 2 : 4;
  const long long tasks = (long long)a.T * (a.kv.Hq + 2 * a.kv.Hkv) * a.kv.d * es / 32;
  // one task a thread while that leaves SMs idle, four (eight loads in flight) above
  const bool small = tasks <= (long long)ROPE_THREADS * 4 * sms;
  if (a.kv.dtype == PRHS_BF16)
    return small ? rope_go<__nv_bfloat16, 1>(a, st) : rope_go<__nv_bfloat16, 4>(a, st);
  return small ? rope_go<float, 1>(a, st) : rope_go<float, 4>(a, st);
}

}  // namespace prhs
