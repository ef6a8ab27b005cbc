// Finds the prefixes that consecutive rows of a batch share, in their page tables.
//
// Two rows share the leading pages that both name, whole ones within both
// lengths. A group is a run of rows with new tokens (rows without are passed over);
// a row joins the group above it while that does not lower what the group saves,
// (rows - 1) * shared pages, and the shared keys stay at least min_keys. Rows whose
// own query rows fill a tile of the attention (GROUP_FULL a KV head) have nothing to
// gain and stay alone.
//
// One cluster of CTAs: a warp compares two rows, 512 entries at a time; then one
// CTA forms the groups, a thread for each run of rows between two that share
// nothing, and writes them. Bound: latency (lengths, tables, the groups' chain; the tables
// are read twice, from L2): 128 rows in 8 groups of up to 5072 keys on 16-key pages 8 to
// 11 us, 8 rows 7.6.
#include <cooperative_groups.h>

#include "pages.h"

namespace prhs {

namespace cg = cooperative_groups;

constexpr int FIND_THREADS = 1024;
constexpr int FIND_WARPS = FIND_THREADS / 32;
constexpr int FIND_CLUSTER = 8;
constexpr int FIND_COLS = 16;
constexpr int GROUP_FULL = 256;

__global__ void __launch_bounds__(FIND_THREADS) find_kernel(const __grid_constant__ FindLaunch a) {
  // of the k-th row with new tokens: the row; the pages it shares with the one before it (-1: it
  // stays alone), later those of its group up to it; its group's first (k's; at that one: ~ the last)
  extern __shared__ int find_smem[];
  __shared__ int wsum[FIND_WARPS];
  const KVView& kv = a.kv;
  const int B = kv.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, M = kv.max_blocks, page = kv.block_size;
  int *row = find_smem, *same = row + B, *head = same + B;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  cluster_begin();
  pdl_wait();
  pdl_trigger();

  // ---- the rows with new tokens, in order ----
  const int per = (B + FIND_THREADS - 1) / FIND_THREADS, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto tokens = [&](int b) { return (long long)a.cu_new[b + 1] - a.cu_new[b]; };
  int mine = 0;
  for (int b = b0; b < b1; b++) mine += tokens(b) > 0;
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL_MASK, at, o);
    if (lane >= o) at += y;
  }
  if (lane == 31) wsum[warp] = at;
  __syncthreads();
  int n = 0;
  at -= mine;
  for (int w = 0; w < FIND_WARPS; w++) {
    if (w < warp) at += wsum[w];
    n += wsum[w];
  }
  for (int b = b0; b < b1; b++)
    if (tokens(b) > 0) row[at++] = b;
  __syncthreads();

  // ---- shared pages of neighbours, into the first CTA (once it has begun) ----
  cluster_begun();
  int* to = cluster.map_shared_rank(same, 0);
  for (int k = rank * FIND_WARPS + warp; k < n; k += ranks * FIND_WARPS) {
    const int b = row[k];
    int pages = 0;
    if (tokens(b) * (kv.Hq / kv.Hkv) >= GROUP_FULL) {
      pages = -1;
    } else if (k > 0 && kv.block_table != nullptr) {
      const int c = row[k - 1], most = min(seq_len(kv, b), seq_len(kv, c)) / page;
      const int32_t *x = kv.block_table + (long long)b * M, *y = kv.block_table + (long long)c * M;
      for (bool equal = true; equal && pages < most;) {
        int p[FIND_COLS], q[FIND_COLS];
#pragma unroll
        for (int i = 0; i < FIND_COLS; i++) {
          const int j = pages + 32 * i + lane;
          p[i] = j < most ? x[j] : 0;
          q[i] = j < most ? y[j] : 1;
        }
#pragma unroll
        for (int i = 0; i < FIND_COLS; i++) {
          const unsigned differ = __ballot_sync(FULL_MASK, p[i] != q[i]);
          if (equal) pages += differ == 0 ? 32 : __ffs(differ) - 1;
          equal &= differ == 0;
        }
      }
    }
    if (lane == 0) to[k] = pages;
  }
  cluster.sync();
  if (rank != 0) return;

  // ---- groups ----
  auto joins = [&](int k) {  // may the k-th join what is above it?
    return k > 0 && same[k] > 0 && same[k - 1] >= 0 && (long long)same[k] * page >= a.min_keys;
  };
  for (int k = tid; k < n; k += FIND_THREADS) {
    if (joins(k)) continue;
    int h = k, common = 0;
    head[k] = ~k;
    for (int i = k + 1; i < n && joins(i); i++) {
      const int rows = i - h, pages = rows == 1 ? same[i] : min(common, same[i]);
      if (rows == 1 || (long long)rows * pages >= (long long)(rows - 1) * common) {
        common = pages;
        head[i] = h;
        head[h] = ~i;
        same[i] = common;  // (joins(i) and joins(i + 1) say the same of it)
      } else {
        h = i;
        head[i] = ~i;
      }
    }
  }
  for (int b = tid; b < B; b += FIND_THREADS) a.shared[b] = make_int4(b, 1, 0, 0);
  __syncthreads();
  for (int k = tid; k < n; k += FIND_THREADS) {
    const int h = head[k] < 0 ? k : head[k], last = ~head[h];
    if (last > h) a.shared[row[k]] = make_int4(row[h], row[last] - row[h] + 1, same[last] * page, 0);
  }
}

cudaError_t launch_find_shared(const FindLaunch& a, cudaStream_t st) {
  const size_t smem = (size_t)a.kv.B * 3 * sizeof(int);
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(find_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  int cl = 1;
  while (cl < FIND_CLUSTER && a.kv.B > cl * FIND_WARPS) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl);
  cfg.blockDim = dim3(FIND_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.kv.pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, find_kernel, a);
}

}  // namespace prhs
