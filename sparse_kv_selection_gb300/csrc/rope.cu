// Rotary positions on the q and k of a batch of tokens, with the cache append.
//
// A pair (x, y) of a head's rotated elements becomes (x c - y s, x s + y c),
// c and s the cosine and sine of position * theta. The angle is taken in turns
// as a 64-bit binary fraction: position * turns modulo 2^64 wraps exactly where
// the angle does, so it is as exact at position 2^31 as at 1, without float64
// (whose rate is low on this part). The nearest quarter turn is taken off in
// integers and the rest, in [-1/8, 1/8) turns to 2^-34, goes to fp32, so that what the
// conversion rounds is relative to the rest: sine and cosine keep their last bits near
// their zeros too. (The whole angle in fp32 is 2^-25 of a half turn off.)
//
// Every head of a token takes the same rot_dim / 2 angles, so a CTA computes
// them once into shared memory, with the tokens' cache rows. The work is cut
// into tasks of two 16-byte pieces of one head row (the two halves of E pairs, E
// elements a piece, or two pieces that are only copied), PER tasks a thread: the
// loads are issued before the angles are computed, which hides one behind the
// other.
//
// Bound: HBM, each element read once and written once. 16601 tokens of 32 / 8
// heads of 128 in bf16 into a paged cache (408 MB): 62.5 us, 0.96 of the measured
// copy bandwidth. Twelve CTAs of 128 threads an SM, two tasks a thread: small
// CTAs, since each waits for its loads once (256 threads with four tasks: 71 us),
// and stores marked streaming (71 -> 66.6 us: a prompt's results exceed L2).
// One token of 96 head rows: 2.6 us.
#include "tokens.h"

namespace prhs {

constexpr int ROPE_THREADS = 128;

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

// `rows` head rows a token (q, k and, with slots, v), 1 << tpr_log2 tasks a row.
template <typename T, int PER>
__global__ void __launch_bounds__(ROPE_THREADS, PER == 1 ? 1 : 12)
    rope_kernel(const RopeLaunch a, int rows, float inv_rows, int tpr_log2, int max_tokens) {
  constexpr int E = Elem<T>::per16;
  extern __shared__ __align__(16) uint8_t rope_smem[];
  const KVView& kv = a.kv;
  const int half = a.rot_dim / 2, rot_tasks = half / E;
  float2* cs = reinterpret_cast<float2*>(rope_smem);                    // [max_tokens][half]
  // the tokens' cache rows (KV head 0; -1: nothing of the token is written)
  long long* token_row = reinterpret_cast<long long*>(cs + max_tokens * half);  // [max_tokens]
  pdl_wait();
  pdl_trigger();

  // Thread t takes piece pair x = t mod tasks of the head rows r0, r0 + step, ...
  const int x = threadIdx.x & ((1 << tpr_log2) - 1), step = ROPE_THREADS >> tpr_log2;
  const long long first = (long long)blockIdx.x * (step * PER), total = (long long)a.T * rows;
  const int tok0 = (int)(first / rows);
  const int base = (int)(first - (long long)tok0 * rows);     // head rows of tok0 before the CTA's
  const int n_rows = (int)min((long long)step * PER, total - first);
  const int tokens = (int)((base + n_rows - 1 + 0.5f) * inv_rows) + 1;
  const bool rotated = x < rot_tasks;
  const int p0 = rotated && !a.interleaved ? x : 2 * x;       // its two 16-byte pieces
  const int p1 = rotated && !a.interleaved ? x + rot_tasks : 2 * x + 1;

  uint4 lo[PER], hi[PER];
#pragma unroll
  for (int u = 0; u < PER; u++) {
    const int r = (threadIdx.x >> tpr_log2) + u * step;
    if (r < n_rows) {
      const int k = (int)((base + r + 0.5f) * inv_rows), row = base + r - k * rows;
      const long long tok = tok0 + k;
      const T* src;
      if (row < kv.Hq) src = static_cast<const T*>(a.q) + tok * a.qs + (long long)row * kv.d;
      else if (row < kv.Hq + kv.Hkv) src = static_cast<const T*>(a.k) + tok * a.ks + (long long)(row - kv.Hq) * kv.d;
      else src = static_cast<const T*>(a.v) + tok * a.vs + (long long)(row - kv.Hq - kv.Hkv) * kv.d;
      lo[u] = __ldcs(reinterpret_cast<const uint4*>(src) + p0);
      hi[u] = __ldcs(reinterpret_cast<const uint4*>(src) + p1);
    }
  }

  for (int i = threadIdx.x; i < tokens * half; i += ROPE_THREADS) {
    const int k = i / half, f = i - k * half;
    const uint64_t turn = (uint64_t)(int64_t)a.positions[tok0 + k] * a.turns[f];
    const unsigned quarter = (unsigned)((turn + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)((int64_t)(turn - ((uint64_t)quarter << 62)) >> 30);  // 2^-34 turns
    float s, c;
    sincospif((float)rest * 0x1p-33f, &s, &c);
    float2 r = quarter & 1 ? make_float2(-s, c) : make_float2(c, s);
    if (quarter & 2) r = make_float2(-r.x, -r.y);
    cs[i] = make_float2(r.x * a.mscale, r.y * a.mscale);
  }
  for (int k = threadIdx.x; k < tokens; k += ROPE_THREADS) {
    long long row = 0;
    if (a.slots != nullptr) {
      const int slot = a.slots[tok0 + k];
      const int slots = kv.block_table != nullptr ? kv.num_blocks * kv.block_size : kv.B * kv.t_max;
      int head_rows;
      row = -1;
      if (slot >= 0 && slot < slots) row = slot_row(kv, slot, &head_rows);
      else if (slot != -1) raise_error(kv.err, PRHS_DEV_BAD_INDEX);
    }
    token_row[k] = row;
  }
  __syncthreads();
  const int head_rows = kv.block_table != nullptr ? kv.block_size : kv.t_max;

#pragma unroll
  for (int u = 0; u < PER; u++) {
    const int r = (threadIdx.x >> tpr_log2) + u * step;
    if (r >= n_rows) break;
    const int k = (int)((base + r + 0.5f) * inv_rows), row = base + r - k * rows;
    const long long tok = tok0 + k, cache_row = token_row[k];
    if (cache_row < 0) continue;
    if (rotated && row < kv.Hq + kv.Hkv) {
      float e0[E], e1[E];
      Elem<T>::unpack(lo[u], e0);
      Elem<T>::unpack(hi[u], e1);
      const float2* t = cs + k * half + x * E;
      if (!a.interleaved) {
#pragma unroll
        for (int e = 0; e < E; e++) {
          const float r0 = e0[e] * t[e].x - e1[e] * t[e].y;
          e1[e] = e0[e] * t[e].y + e1[e] * t[e].x;
          e0[e] = r0;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E / 2; e++) {
          const float2 v = t[e], w = t[E / 2 + e];
          const float r0 = e0[2 * e] * v.x - e0[2 * e + 1] * v.y;
          e0[2 * e + 1] = e0[2 * e] * v.y + e0[2 * e + 1] * v.x;
          e0[2 * e] = r0;
          const float r1 = e1[2 * e] * w.x - e1[2 * e + 1] * w.y;
          e1[2 * e + 1] = e1[2 * e] * w.y + e1[2 * e + 1] * w.x;
          e1[2 * e] = r1;
        }
      }
      lo[u] = pack_piece<T>(e0);
      hi[u] = pack_piece<T>(e1);
    }
    if (row < kv.Hq) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (tok * kv.Hq + row) * kv.d);
      __stcs(dst + p0, lo[u]);
      __stcs(dst + p1, hi[u]);
      continue;
    }
    const bool is_k = row < kv.Hq + kv.Hkv;
    const int h = row - kv.Hq - (is_k ? 0 : kv.Hkv);
    if (is_k && a.k_out != nullptr) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + (tok * kv.Hkv + h) * kv.d);
      __stcs(dst + p0, lo[u]);
      __stcs(dst + p1, hi[u]);
    }
    if (a.slots != nullptr) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(const_cast<void*>(is_k ? kv.k : kv.v)) +
                                            (cache_row + (long long)h * head_rows) * kv.d);
      __stcs(dst + p0, lo[u]);
      __stcs(dst + p1, hi[u]);
    }
  }
}

template <typename T, int PER>
static cudaError_t rope_go(const RopeLaunch& a, cudaStream_t st) {
  constexpr int E = Elem<T>::per16;
  const int rows = a.kv.Hq + (a.slots != nullptr ? 2 : 1) * a.kv.Hkv;
  int tpr_log2 = 0;
  while ((2 * E) << tpr_log2 < a.kv.d) tpr_log2++;  // d / (2 E) tasks a row: 4, 8 or 16
  const int chunk = (ROPE_THREADS >> tpr_log2) * PER;  // head rows of a CTA
  // tokens a CTA may touch: its whole ones and one cut at each end
  const long long most = (chunk + rows - 1) / rows + 1;
  const int max_tokens = (int)(most < a.T ? most : a.T);
  const size_t smem = (size_t)max_tokens * (a.rot_dim / 2 * sizeof(float2) + sizeof(long long));
  auto k = rope_kernel<T, PER>;
  static int smem_set[SMEM_DEVICES];
  const cudaError_t e = allow_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)(((long long)a.T * rows + chunk - 1) / chunk)), dim3(ROPE_THREADS), smem, st,
                    a.kv.pdl, a, rows, 1.0f / rows, tpr_log2, max_tokens);
}

cudaError_t launch_rope(const RopeLaunch& a, int sms, cudaStream_t st) {
  const int es = a.kv.dtype == PRHS_BF16 ? 2 : 4;
  const long long tasks = (long long)a.T * (a.kv.Hq + 2 * a.kv.Hkv) * a.kv.d * es / 32;
  // one task a thread while that leaves SMs idle, two (four loads in flight) above
  const bool small = tasks <= (long long)ROPE_THREADS * 8 * sms;
  if (a.kv.dtype == PRHS_BF16)
    return small ? rope_go<__nv_bfloat16, 1>(a, st) : rope_go<__nv_bfloat16, 2>(a, st);
  return small ? rope_go<float, 1>(a, st) : rope_go<float, 2>(a, st);
}

}  // namespace prhs
