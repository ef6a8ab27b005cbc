// Pages, slots, positions and tree masks of a batch of new tokens.
//
// Everything follows from two prefix sums over the sequences (new tokens; new
// pages), so every CTA of one cluster forms both for itself from the cached
// lengths (B values, a few loads per thread, one scan) and then takes its share
// of the tokens, of the new pages and of the trees. A warp takes 128 tokens of the
// chunks, whose sequence it finds by a search in the shared prefix (four tokens a
// thread, so that their page reads overlap); a tree is one warp's, its slots too. The
// page counters may be updated in place: they are written after a cluster
// barrier behind the last read.
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

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_CLUSTER = 16;  // above 8 by opt-in

struct PlanTree {  // one warp's tree
  uint4 anc[PRHS_TREE_MAX];
  int16_t up[PRHS_TREE_MAX];
};

// Exclusive block scan of two values per thread (64-bit); the sums into *tx, *ty.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, longlong2* wsum, long long* tx, long long* ty) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(FULL_MASK, x, o), v = __shfl_up_sync(FULL_MASK, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) wsum[warp] = make_longlong2(x, y);
  __syncthreads();
  // every warp scans the warps' sums for itself
  longlong2 s = lane < PLAN_WARPS ? wsum[lane] : make_longlong2(0, 0);
  long long bx = 0, by = 0, ax = s.x, ay = s.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ax += __shfl_xor_sync(FULL_MASK, ax, o);
    ay += __shfl_xor_sync(FULL_MASK, ay, o);
  }
  if (lane >= warp) s = make_longlong2(0, 0);
  bx = s.x;
  by = s.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    bx += __shfl_xor_sync(FULL_MASK, bx, o);
    by += __shfl_xor_sync(FULL_MASK, by, o);
  }
  x += bx - x0;
  y += by - y0;
  *tx = ax;
  *ty = ay;
}

__device__ __forceinline__ uint4 or4(uint4 a, uint4 b) {
  return make_uint4(a.x | b.x, a.y | b.y, a.z | b.z, a.w | b.w);
}

// Index of the last entry of the ascending list v[lo .. hi] that is <= x (v[lo] <= x).
__device__ __forceinline__ int last_le(const int* v, int lo, int hi, int x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const PlanLaunch a) {
  extern __shared__ __align__(16) uint8_t plan_smem[];
  __shared__ longlong2 wsum[PLAN_WARPS];
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

  if (tid == 0) sh_taken = 0;
  pdl_wait();
  pdl_trigger();
  const bool paged = a.block_table != nullptr, tree = a.parents != nullptr;
  const int head = paged ? a.free_head[0] : 0;
  const int per = (B + PLAN_THREADS - 1) / PLAN_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

  // New pages of sequence b, 0 (and the reason) when it cannot be placed.
  auto pages_of = [&](int b, int& n, unsigned& bits) -> int {
    n = a.n_new[b];
    const int t = seq_len(kv, b), have = paged ? a.n_pages[b] : 0;
    if (n < 0 || (tree && n > PRHS_TREE_MAX)) bits = PRHS_DEV_BAD_LEN;
    else if (n > 0 && ((long long)t + n > kv.t_max || have < 0 || have > kv.max_blocks || head < 0)) bits = PRHS_DEV_CAPACITY;
    if (!paged || n <= 0 || bits != 0) return 0;
    return max(0, (t + n + kv.block_size - 1) / kv.block_size - have);
  };

  // ---- prefixes of the new tokens and of the new pages ----
  // (A sequence cut by T takes no page, but those behind it are cut too, so the
  // prefix of every sequence that is placed is right without knowing.)
  long long sum_n = 0, sum_p = 0, total = 0, pages = 0;
  for (int b = b0; b < b1; b++) {
    int n;
    unsigned bits = 0;
    sum_p += pages_of(b, n, bits);
    sum_n += max(0, n);
  }
  block_scan2(sum_n, sum_p, wsum, &total, &pages);
  for (int b = b0; b < b1; b++) {
    int n;
    unsigned bits = 0;
    const int take = pages_of(b, n, bits);
    cu[b] = (int)min(sum_n, (long long)a.T);
    if (bits == 0 && n > 0 && sum_n + n > a.T) bits = PRHS_DEV_CAPACITY;
    if (bits == 0 && take > 0 && head + sum_p + take > a.n_free) bits = PRHS_DEV_CAPACITY;
    // the sign bit marks a sequence that cannot be placed
    pp[b] = (int)min(sum_p, 0x7fffffffll) | (bits == 0 ? 0 : (int)0x80000000);
    sum_n += max(0, n);
    sum_p += take;
    if (bits == 0 && take > 0) atomicMax(&sh_taken, (int)sum_p);
    if (bits != 0 && rank == 0) raise_error(kv.err, bits);
  }
  const int T = (int)min(total, (long long)a.T);  // tokens that are not padding
  if (tid == 0) cu[B] = T;
  __syncthreads();
  const int taken = sh_taken;
  const int step = ranks * PLAN_THREADS, first = rank * PLAN_THREADS + tid;

  const int shift = __ffs(kv.block_size) - 1;
  const bool pow2 = kv.block_size == 1 << shift;
  // Slot of position `pos` of sequence b (p: its entry of pp, have: its pages), -1 when there is none.
  auto slot_of = [&](int b, int pos, int p, int have) -> int {
    if (p < 0) return -1;
    if (!paged) return b * kv.t_max + pos;
    const int blk = pow2 ? pos >> shift : pos / kv.block_size;
    const int page = blk < have ? a.block_table[(long long)b * kv.max_blocks + blk] : a.free_pages[head + p + blk - have];
    if ((unsigned)page < (unsigned)kv.num_blocks) return page * kv.block_size + (pos - blk * kv.block_size);
    raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
    return -1;
  };

  // ---- trees: one warp per sequence ----
  if (tree) {
    PlanTree& tr = trees[warp];
    constexpr int PL = PRHS_TREE_MAX / 32;
    for (int b = rank * PLAN_WARPS + warp; b < B; b += ranks * PLAN_WARPS) {
      const int c0 = cu[b], n = cu[b + 1] - c0, p = pp[b], t = seq_len(kv, b);
      const int have = paged ? a.n_pages[b] : 0;
      if (n > PRHS_TREE_MAX) {  // refused above: no masks, no slots
        for (int j = lane; j < n; j += 32) {
          reinterpret_cast<uint4*>(a.tree_mask)[c0 + j] = make_uint4(0, 0, 0, 0);
          a.positions[c0 + j] = t + j;
          a.slots[c0 + j] = -1;
        }
        continue;
      }
      uint4 anc[PL];
      int up[PL], slot[PL];
      bool more = false;
#pragma unroll
      for (int k = 0; k < PL; k++) {
        const int j = k * 32 + lane;
        up[k] = -1;
        slot[k] = -1;
        anc[k] = make_uint4(k == 0 ? 1u << lane : 0, k == 1 ? 1u << lane : 0, k == 2 ? 1u << lane : 0,
                            k == 3 ? 1u << lane : 0);
        if (j < n) {
          const int par = a.parents[c0 + j];
          slot[k] = slot_of(b, t + j, p, have);
          if (par < -1 || par >= j) raise_error(kv.err, PRHS_DEV_BAD_INDEX);
          else up[k] = par;
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
          a.slots[c0 + j] = slot[k];
        }
      }
      __syncwarp();
    }
  } else {
    // ---- chunks: a warp takes 128 consecutive tokens, mostly of one sequence ----
    constexpr int TOKS = 4;
    for (int w0 = (rank * PLAN_WARPS + warp) * 32 * TOKS; w0 < T; w0 += ranks * PLAN_WARPS * 32 * TOKS) {
      const int bw = last_le(cu, 0, B - 1, w0);
      int b[TOKS], pos[TOKS], slot[TOKS];
#pragma unroll
      for (int u = 0; u < TOKS; u++) {
        const int i = min(w0 + u * 32 + lane, T - 1);
        b[u] = i < cu[bw + 1] ? bw : last_le(cu, bw + 1, B - 1, i);
        pos[u] = seq_len(kv, b[u]) + (i - cu[b[u]]);
      }
#pragma unroll
      for (int u = 0; u < TOKS; u++) slot[u] = slot_of(b[u], pos[u], pp[b[u]], paged ? a.n_pages[b[u]] : 0);
#pragma unroll
      for (int u = 0; u < TOKS; u++) {
        const int i = w0 + u * 32 + lane;
        if (i < T) {
          a.slots[i] = slot[u];
          a.positions[i] = pos[u];
        }
      }
    }
  }

  for (int b = first; b <= B; b += step) a.cu_new[b] = cu[b];
  for (int i = T + first; i < a.T; i += step) {  // padding
    a.slots[i] = -1;
    a.positions[i] = 0;
    if (tree) reinterpret_cast<uint4*>(a.tree_mask)[i] = make_uint4(0, 0, 0, 0);
  }

  // ---- new entries of the block tables, then the counters ----
  if (!paged) return;
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
  cluster.sync();  // every CTA has read the old counters
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
  cudaError_t e = allow_smem(plan_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  // one CTA for a decode or verification step; a cluster for prompts and for
  // batches with more trees than one CTA's warps
  const long long work = a.parents != nullptr ? 1 : (long long)a.T / (4 * PLAN_THREADS);
  const long long trees = a.parents != nullptr ? (a.kv.B + PLAN_WARPS - 1) / PLAN_WARPS : 1;
  int cl = 1;
  while (cl < PLAN_CLUSTER && (work > cl || trees > cl)) cl *= 2;
  if (cl > 8 && (e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
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
