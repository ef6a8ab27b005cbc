// Accepted tokens join the cache: their packed key and value rows are written
// behind each sequence's cached prefix and its length advances.
//
// One cluster of CTAs per sequence. Every CTA checks the sequence's whole
// request (numbers, room, pages, planned slots; also where only the length advances)
// before anything is written, so a refused sequence keeps its rows and its length; then the cluster copies the rows in
// 16-byte pieces, COMMIT_PER loads of a thread in flight, and the length is
// written behind a cluster barrier, since it may be the array that every CTA
// read. Bound: latency (a handful of rows), HBM for long batches.
#include <cooperative_groups.h>

#include "tokens.h"

namespace prhs {

constexpr int COMMIT_THREADS = 512;
constexpr int COMMIT_PER = 4;
constexpr int COMMIT_STAGE = 256;  // accepted rows whose addresses are staged at a time

template <typename T>
__global__ void __launch_bounds__(COMMIT_THREADS) commit_kernel(const CommitLaunch a) {
  __shared__ int sh_src[COMMIT_STAGE];
  __shared__ long long sh_row[COMMIT_STAGE];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  pdl_wait();
  pdl_trigger();
  const KVView& kv = a.kv;
  const int b = blockIdx.x / ranks, tid = threadIdx.x;
  const int t = kv.seq_lens[b];
  int m = a.accept_n[b], c0 = 0;
  const int n = seq_tokens(a.cu_new, b, a.T, a.T, kv.err, &c0);
  const int32_t* idx = a.accept_idx != nullptr ? a.accept_idx + (long long)b * a.accept_cap : nullptr;
  unsigned bits = 0;
  if (t < 0 || t > kv.t_max || m < 0 || m > n || (idx != nullptr && m > a.accept_cap)) bits = PRHS_DEV_BAD_LEN;
  else if ((long long)t + m > kv.t_max) bits = PRHS_DEV_CAPACITY;
  if (bits != 0) m = 0;
  for (int i = tid; i < m; i += COMMIT_THREADS) {
    if (idx != nullptr && (idx[i] < 0 || idx[i] >= n)) bits |= PRHS_DEV_BAD_INDEX;
    const long long row = kv_row(kv, b, 0, t + i);
    const int slot = a.slots != nullptr ? a.slots[c0 + i] : 0;  // what planning gave to position t + i
    int head_rows;
    if (slot < 0) bits |= PRHS_DEV_CAPACITY;
    else if (row < 0) bits |= PRHS_DEV_BAD_BLOCK;
    else if (a.slots != nullptr && slot_row(kv, slot, &head_rows) != row) bits |= PRHS_DEV_BAD_INDEX;
  }
  if (bits != 0 && rank == 0) raise_error(kv.err, bits);
  if (__syncthreads_or((int)bits)) m = 0;

  if (a.k_new != nullptr) {
    const int ppr = kv.d * (int)sizeof(T) / 16;  // 16-byte pieces of a row
    const int per_row = kv.Hkv * ppr;
    const int head_rows = kv.block_table != nullptr ? kv.block_size : kv.t_max;
    for (int s0 = 0; s0 < m; s0 += COMMIT_STAGE) {
      const int ns = min(COMMIT_STAGE, m - s0);
      if (s0 > 0) __syncthreads();
      for (int i = tid; i < ns; i += COMMIT_THREADS) {
        sh_src[i] = c0 + (idx != nullptr ? idx[s0 + i] : s0 + i);
        sh_row[i] = kv_row(kv, b, 0, t + s0 + i);
      }
      __syncthreads();
      const int pieces = ns * per_row * 2;  // K, then V
      for (int x0 = rank * COMMIT_THREADS + tid; x0 < pieces; x0 += ranks * COMMIT_THREADS * COMMIT_PER) {
        uint4 c[COMMIT_PER];
        uint4* dst[COMMIT_PER];
#pragma unroll
        for (int u = 0; u < COMMIT_PER; u++) {
          const int x = x0 + u * ranks * COMMIT_THREADS;
          dst[u] = nullptr;
          if (x < pieces) {
            const bool is_v = x >= ns * per_row;
            const int y = x - (is_v ? ns * per_row : 0);
            const int i = y / per_row, hp = y - i * per_row;  // entry, (head, piece)
            const int h = hp / ppr, p = hp - h * ppr;
            const T* src = is_v ? static_cast<const T*>(a.v_new) + sh_src[i] * a.vs
                                : static_cast<const T*>(a.k_new) + sh_src[i] * a.ks;
            c[u] = reinterpret_cast<const uint4*>(src)[hp];
            dst[u] = static_cast<uint4*>(const_cast<void*>(is_v ? kv.v : kv.k)) +
                     (sh_row[i] + (long long)h * head_rows) * ppr + p;
          }
        }
#pragma unroll
        for (int u = 0; u < COMMIT_PER; u++)
          if (dst[u] != nullptr) *dst[u] = c[u];
      }
    }
  }
  cluster.sync();  // every CTA has read the old length
  if (rank == 0 && tid == 0) a.new_lens[b] = t + m;
}

template <typename T>
static cudaError_t commit_go(const CommitLaunch& a, int cl, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.kv.B * cl);
  cfg.blockDim = dim3(COMMIT_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.kv.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, commit_kernel<T>, a);
}

cudaError_t launch_commit(const CommitLaunch& a, int sms, cudaStream_t st) {
  // as many CTAs a sequence (a power of two up to 8) as fill the SMs, while
  // the sequence has a sweep of pieces for each
  const int es = a.kv.dtype == PRHS_BF16 ? 2 : 4;
  const long long most = a.accept_idx != nullptr ? (a.accept_cap < a.T ? a.accept_cap : a.T) : a.T;
  const long long pieces = a.k_new != nullptr ? most * a.kv.Hkv * a.kv.d * es / 8 : 0;
  int cl = 1;
  while (cl < 8 && (long long)a.kv.B * cl * 2 <= 2 * sms && pieces >= 2ll * cl * COMMIT_THREADS) cl *= 2;
  return a.kv.dtype == PRHS_BF16 ? commit_go<__nv_bfloat16>(a, cl, st) : commit_go<float>(a, cl, st);
}

}  // namespace prhs
