// Pages, slots, positions and tree masks of a batch of new tokens.
//
// Everything follows from two prefix sums over the sequences (new tokens; new
// pages), so every CTA of one cluster forms both for itself from the cached
// lengths (B values, a few loads per thread) and then takes an interleaved
// share of the tokens, of the new pages and of the trees, finding a token's
// sequence by a search in the shared prefix. The page counters may be updated
// in place: they are written after a cluster barrier behind the last read.
//
// A tree's masks are its ancestor sets, by pointer doubling: after round r a
// token knows its ancestors up to 2^r steps up, anc(j) |= anc(up(j)), up(j) =
// up(up(j)), so a tree of depth D takes ceil(log2 D) rounds of one warp, four
// tokens a lane, instead of a walk of D dependent reads per token.
//
// The bound is latency: a few KB in and out and three dependent round trips
// (lengths, page entries, stores).
#include <cooperative_groups.h>

#include "tokens.h"

namespace prhs {

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_CLUSTER = 8;

struct PlanTree {  // one warp's tree
  uint4 anc[PRHS_TREE_MAX];
  int16_t up[PRHS_TREE_MAX];
};

// Exclusive block scan of one value per thread (64-bit); *total gets the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* wsum, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(FULL_MASK, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < PLAN_WARPS; w++) {
    const long long s = wsum[w];
    if (w < warp) before += s;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ uint4 or4(uint4 a, uint4 b) {
  return make_uint4(a.x | b.x, a.y | b.y, a.z | b.z, a.w | b.w);
}

// Index of the last entry of the ascending list v[0..n) that is <= x (v[0] <= x).
__device__ __forceinline__ int last_le(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const PlanLaunch a) {
  extern __shared__ __align__(16) uint8_t plan_smem[];
  __shared__ long long wsum[PLAN_WARPS];
  __shared__ int sh_taken;
  const KVView& kv = a.kv;
  const int B = kv.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // cu [B + 1], page prefix [B + 1], then (with parents) one tree per warp
  int* cu = reinterpret_cast<int*>(plan_smem);
  int* pp = cu + B + 1;
  PlanTree* trees = reinterpret_cast<PlanTree*>(plan_smem + ((size_t)(2 * (B + 1)) * 4 + 15) / 16 * 16);
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();

  pdl_wait();
  pdl_trigger();
  const bool paged = a.block_table != nullptr, tree = a.parents != nullptr;
  const int head = paged ? a.free_head[0] : 0;
  const int per = (B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

  // ---- prefix of the new tokens ----
  long long mine = 0, total = 0;
  for (int b = b0; b < b1; b++) mine += max(0, a.n_new[b]);
  long long run = block_scan(mine, wsum, &total);
  for (int b = b0; b < b1; b++) {
    cu[b] = (int)min(run, (long long)a.T);
    run += max(0, a.n_new[b]);
  }
  if (tid == 0) {
    cu[B] = (int)min(total, (long long)a.T);
    sh_taken = 0;
  }
  const int T = (int)min(total, (long long)a.T);  // tokens that are not padding

  // ---- prefix of the new pages; a sequence that cannot be placed takes none ----
  auto pages_of = [&](int b, unsigned& bits) -> int {
    const int n = a.n_new[b], t = seq_len(kv, b);
    if (n < 0 || (tree && n > PRHS_TREE_MAX)) bits = PRHS_DEV_BAD_LEN;
    else if (n > 0 && ((long long)t + n > kv.t_max || (long long)cu[b] + n > a.T)) bits = PRHS_DEV_CAPACITY;
    if (!paged || n <= 0 || bits != 0) return 0;
    const int have = a.n_pages[b];
    if (have < 0 || have > kv.max_blocks || head < 0) {
      bits = PRHS_DEV_CAPACITY;
      return 0;
    }
    return max(0, (t + n + kv.block_size - 1) / kv.block_size - have);
  };
  mine = 0;
  for (int b = b0; b < b1; b++) {
    unsigned bits = 0;
    mine += pages_of(b, bits);
  }
  run = block_scan(mine, wsum, &total);
  for (int b = b0; b < b1; b++) {
    unsigned bits = 0;
    const int take = pages_of(b, bits);
    if (take > 0 && head + run + take > a.n_free) bits = PRHS_DEV_CAPACITY;
    // the sign bit marks a sequence that cannot be placed
    pp[b] = (int)min(run, 0x7fffffffll) | (bits == 0 ? 0 : (int)0x80000000);
    run += take;
    if (bits == 0 && take > 0) atomicMax(&sh_taken, (int)run);
    if (bits != 0 && rank == 0) raise_error(kv.err, bits);
  }
  __syncthreads();
  const int taken = sh_taken;
  const int step = ranks * PLAN_THREADS, first = rank * PLAN_THREADS + tid;

  for (int b = first; b <= B; b += step) a.cu_new[b] = cu[b];

  // ---- slots and positions ----
  for (int i = first; i < a.T; i += step) {
    int slot = -1, position = 0;
    if (i < T) {
      const int b = last_le(cu, B, i);
      const int t = seq_len(kv, b);
      position = t + (i - cu[b]);
      const int p = pp[b];
      if (p >= 0) {
        if (!paged) {
          slot = b * kv.t_max + position;
        } else {
          const int blk = position / kv.block_size, have = a.n_pages[b];
          const int page = blk < have ? a.block_table[(long long)b * kv.max_blocks + blk]
                                      : a.free_pages[head + p + blk - have];
          if ((unsigned)page < (unsigned)kv.num_blocks)
            slot = page * kv.block_size + (position - blk * kv.block_size);
          else
            raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
        }
      }
    }
    a.slots[i] = slot;
    if (!tree || i >= T) a.positions[i] = position;
    if (tree && i >= T) reinterpret_cast<uint4*>(a.tree_mask)[i] = make_uint4(0, 0, 0, 0);
  }

  // ---- new entries of the block tables ----
  if (paged)
    for (int g = first; g < taken; g += step) {
      int lo = 0, hi = B - 1;  // the last sequence whose page prefix is <= g
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((pp[mid] & 0x7fffffff) <= g) lo = mid; else hi = mid - 1;
      }
      const int p = pp[lo];
      if (p < 0) continue;
      const int page = a.free_pages[head + g];
      if ((unsigned)page >= (unsigned)kv.num_blocks) raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
      a.block_table[(long long)lo * kv.max_blocks + a.n_pages[lo] + (g - p)] = page;
    }

  // ---- trees: one warp per sequence ----
  if (tree) {
    PlanTree& tr = trees[warp];
    for (int b = rank * PLAN_WARPS + warp; b < B; b += ranks * PLAN_WARPS) {
      const int c0 = cu[b], n = cu[b + 1] - c0, t = seq_len(kv, b);
      if (n > PRHS_TREE_MAX) {  // refused above: no masks
        for (int j = lane; j < n; j += 32) {
          reinterpret_cast<uint4*>(a.tree_mask)[c0 + j] = make_uint4(0, 0, 0, 0);
          a.positions[c0 + j] = t + j;
        }
        continue;
      }
      constexpr int PL = PRHS_TREE_MAX / 32;
      uint4 anc[PL];
      int up[PL];
      bool more = false;
#pragma unroll
      for (int k = 0; k < PL; k++) {
        const int j = k * 32 + lane;
        up[k] = -1;
        anc[k] = make_uint4(k == 0 ? 1u << lane : 0, k == 1 ? 1u << lane : 0, k == 2 ? 1u << lane : 0,
                            k == 3 ? 1u << lane : 0);
        if (j < n) {
          const int p = a.parents[c0 + j];
          if (p < -1 || p >= j) raise_error(kv.err, PRHS_DEV_BAD_INDEX);
          else up[k] = p;
          tr.anc[j] = anc[k];
          tr.up[j] = (int16_t)up[k];
        }
        more |= up[k] >= 0;
      }
      __syncwarp();
      // ceil(log2(PRHS_TREE_MAX)) rounds at most: every parent is an earlier token
      for (int round = 0; round < 7 && __any_sync(FULL_MASK, more); round++) {
        more = false;
        int nu[PL];
#pragma unroll
        for (int k = 0; k < PL; k++) {
          nu[k] = up[k];
          if (up[k] >= 0) {
            anc[k] = or4(anc[k], tr.anc[up[k]]);
            nu[k] = tr.up[up[k]];
          }
          more |= nu[k] >= 0;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < PL; k++) {
          if (up[k] >= 0) {
            tr.anc[k * 32 + lane] = anc[k];
            tr.up[k * 32 + lane] = (int16_t)nu[k];
          }
          up[k] = nu[k];
        }
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < PL; k++) {
        const int j = k * 32 + lane;
        if (j < n) {
          reinterpret_cast<uint4*>(a.tree_mask)[c0 + j] = anc[k];
          a.positions[c0 + j] = t + __popc(anc[k].x) + __popc(anc[k].y) + __popc(anc[k].z) + __popc(anc[k].w) - 1;
        }
      }
      __syncwarp();
    }
  }

  // ---- counters: every CTA has read the old ones ----
  if (!paged) return;
  cluster.sync();
  if (rank != 0) return;
  for (int b = tid; b < B; b += PLAN_THREADS) {
    const int have = a.n_pages[b], t = seq_len(kv, b), n = a.n_new[b];
    const bool took = pp[b] >= 0 && n > 0;
    a.n_pages_out[b] = took ? max(have, (t + n + kv.block_size - 1) / kv.block_size) : have;
  }
  if (tid == 0) a.free_head_out[0] = head + taken;
}

cudaError_t launch_plan(const PlanLaunch& a, cudaStream_t st) {
  const size_t lists = ((size_t)2 * (a.kv.B + 1) * 4 + 15) / 16 * 16;
  const size_t smem = lists + (a.parents != nullptr ? PLAN_WARPS * sizeof(PlanTree) : 0);
  static int smem_set[SMEM_DEVICES];
  const cudaError_t e = allow_smem(plan_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  // one CTA for a decode or verification step; a cluster for prompts and for
  // batches with more trees than one CTA's warps
  const long long work = (long long)a.T / (2 * PLAN_THREADS);
  const long long trees = a.parents != nullptr ? (a.kv.B + PLAN_WARPS - 1) / PLAN_WARPS : 1;
  int cl = 1;
  while (cl < PLAN_CLUSTER && (work > cl || trees > cl)) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl);
  cfg.blockDim = dim3(PLAN_THREADS);
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
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace prhs
