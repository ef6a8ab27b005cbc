// Rows of the batch that become copies of other rows, end, or keep a part of
// their positions: page tables, holders of each page, the free list.
//
// A page's holders are the table rows that name it; shares[p] is their number
// less one. A row of the new table is columns of an old row (its parent's, or its
// own first ones), then pages from the free list; what its old row held beyond
// that is released. With +1 for each copied entry and -1 for each released one,
// the pages that end at -1 have no holder and go back in front of the free list.
// Sums do not depend on the order of the atomics. Which of several releases of
// one page counts as the one that frees it does: the first by (row, column), found
// by a second round of atomicMin on the same word (INT_MIN + the entry's number,
// below every count), so that the free list has one possible order.
//
// A call is carried out whole or not at all: rows are checked and pages counted
// before anything is written, and what shows later (a page outside the pool, no
// room in the free list) takes the counts back.
//
// One cluster of CTAs. The entries of the table are tasks of 256 columns of a
// row, a warp's tasks consecutive, so that a prefix over the warps' counts gives
// every freed page its place. Bound: latency, a few dependent passes through L2
// with a cluster barrier between two.
#include <cooperative_groups.h>

#include "pages.h"

namespace prhs {

namespace cg = cooperative_groups;

constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_CLUSTER = 16;           // above 8 by opt-in
constexpr int PG_COLS = 8;               // columns a lane
constexpr int PG_TASK = 32 * PG_COLS;    // columns of a task
constexpr int PG_KEEP = 1024;            // kept positions a warp checks at a time

// Exclusive prefix of x over the block's threads, the sum into *total.
__device__ __forceinline__ int block_scan(int x, int* wsum, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(FULL_MASK, y, o);
    if (lane >= o) y += u;
  }
  if (lane == 31) wsum[warp] = y;
  __syncthreads();
  int before = lane < warp ? wsum[lane] : 0, all = wsum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(FULL_MASK, before, o);
    all += __shfl_xor_sync(FULL_MASK, all, o);
  }
  *total = all;
  return before + y - x;
}

template <bool FORK>
__global__ void __launch_bounds__(PG_THREADS) pages_kernel(const __grid_constant__ PagesLaunch a) {
  extern __shared__ int pg_smem[];
  __shared__ int wsum[PG_WARPS];
  __shared__ int sh_most, sh_base[PG_WARPS];
  __shared__ unsigned sh_bits;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gw = rank * PG_WARPS + warp, gws = ranks * PG_WARPS;      // the warp among the cluster's
  const int gt = rank * PG_THREADS + tid, gts = ranks * PG_THREADS;
  const KVView& kv = a.kv;
  const int B = kv.B, M = kv.max_blocks, page = kv.block_size;
  const int32_t* table = kv.block_table;
  int* first = pg_smem;     // fork, [B]: the first child of each row that takes a part of its last page
  int* count = first + B;   //       [B]: its children
  int* late = a.sums + gws;

  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    sh_bits = 0;
    sh_most = 0;
  }
  if (gt == 0) *late = 0;
  if (a.shares_out != a.shares)
    for (int i = gt; i < kv.num_blocks; i += gts) a.shares_out[i] = a.shares[i];
  if (a.free_out != a.free_pages)
    for (int i = gt; i < a.n_free; i += gts) a.free_out[i] = a.free_pages[i];
  if (a.table_out != table)
    for (long long i = gt; i < (long long)B * M; i += gts) a.table_out[i] = table[i];
  const int head = a.free_head[0];

  // ---- what every row becomes ----
  if constexpr (FORK) {
    for (int b = tid; b < B; b += PG_THREADS) {
      first[b] = B;
      count[b] = 0;
    }
    __syncthreads();
    for (int b = tid; b < B; b += PG_THREADS) {
      const int p = a.parent[b];
      if (p == b || p < 0 || p >= B) continue;
      const int t = kv.seq_lens[p];
      atomicAdd(&count[p], 1);
      if (t > 0 && t % page != 0) atomicMin(&first[p], b);
    }
    __syncthreads();
  } else {
    const int chunks = (min(a.cap, kv.t_max) + PG_KEEP - 1) / PG_KEEP;
    for (int x = gw; x < B * chunks; x += gws) {
      const int b = x / chunks, m = a.keep_n[b], t = kv.seq_lens[b];
      const int32_t* keep = a.keep + (long long)b * a.cap;
      int same = 0;
      unsigned bits = m > a.cap || (m >= 0 && (t < 0 || t > kv.t_max || m > t)) ? PRHS_DEV_BAD_LEN : 0;
      const int i1 = bits != 0 ? 0 : min(m, (x % chunks + 1) * PG_KEEP);
#pragma unroll 4
      for (int i = x % chunks * PG_KEEP + lane; i < i1; i += 32) {
        const int k = keep[i], before = i > 0 ? keep[i - 1] : -1;
        if (k <= before || k < 0 || k >= t) bits |= PRHS_DEV_BAD_INDEX;
        else if ((unsigned)table[(long long)b * M + k / page] >= (unsigned)kv.num_blocks) bits |= PRHS_DEV_BAD_BLOCK;
        same += k == i;
      }
      same = __reduce_add_sync(FULL_MASK, same);
      bits = __reduce_or_sync(FULL_MASK, bits);
      if (lane == 0) a.part[x] = make_int2(same, (int)bits);
    }
    cluster.sync();
  }

  auto plan_row = [&](int b, unsigned& bits) {
    PageRow r = {b, 0, 0, 0, 0, -1, 0, -1};
    const int held = a.n_pages[b];
    if constexpr (FORK) {
      const int p = a.parent[b];
      if (p == b) return r;
      r.held = held;
      if (p < -1 || p >= B) bits |= PRHS_DEV_BAD_INDEX;
      if (held < 0 || held > M) bits |= PRHS_DEV_BAD_LEN;
      r.len = 0;
      if (p < 0 || p >= B) return r;
      const int t = kv.seq_lens[p], have = a.n_pages[p];
      if (t < 0 || t > kv.t_max || have < 0 || have > M || (t + page - 1) / page > have) {
        bits |= PRHS_DEV_BAD_LEN;
        return r;
      }
      r.from = p;
      r.len = t;
      r.blocks = r.keep = (t + page - 1) / page;
      if (t % page != 0) {
        const int last = table[(long long)p * M + r.blocks - 1];
        if ((unsigned)last >= (unsigned)kv.num_blocks) bits |= PRHS_DEV_BAD_BLOCK;
        else if (a.parent[p] == p || first[p] != b || a.shares[last] != 0) {
          r.keep--;
          r.last = last;
        }
      }
    } else {
      const int m = a.keep_n[b], t = kv.seq_lens[b];
      if (m < 0) return r;
      const int chunks = (min(a.cap, kv.t_max) + PG_KEEP - 1) / PG_KEEP;
      int same = 0;
      for (int c = 0; c < chunks; c++) {
        const int2 x = a.part[(long long)b * chunks + c];
        same += x.x;
        bits |= (unsigned)x.y;
      }
      if (held < 0 || held > M || t < 0 || t > kv.t_max || (t + page - 1) / page > held) bits |= PRHS_DEV_BAD_LEN;
      if (bits != 0) return r;
      r.len = m;
      r.held = held;
      r.blocks = (m + page - 1) / page;
      r.keep = same / page;
      if (same == m && m % page != 0 && a.shares[table[(long long)b * M + r.keep]] == 0) r.keep++;
      r.released = r.keep;
    }
    return r;
  };
  const int per = (B + PG_THREADS - 1) / PG_THREADS, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  unsigned bits = 0;
  int need = 0, most = 0, taken = 0;
  PageRow r0 = {};  // (the thread's only row of batches up to 1024)
  for (int b = b0; b < b1; b++) {
    r0 = plan_row(b, bits);
    need += r0.blocks - r0.keep;
    most = max(most, max(r0.held, r0.blocks));
    if constexpr (FORK)
      if (count[b] > 0) most = max(most, min(M, max(0, a.n_pages[b])));
  }
  need = block_scan(need, wsum, &taken);
  most = __reduce_max_sync(FULL_MASK, most);
  bits = __reduce_or_sync(FULL_MASK, bits);
  if (lane == 0) {
    atomicMax(&sh_most, most);
    atomicOr(&sh_bits, bits);
  }
  for (int b = b0; b < b1; b++) {
    unsigned ignored = 0;
    if (per > 1) r0 = plan_row(b, ignored);
    r0.taken = need;
    need += r0.blocks - r0.keep;
    if (b % ranks == rank) a.rows[b] = r0;
  }
  __syncthreads();
  bits = sh_bits;
  most = min(sh_most, M);
  if (bits == 0 && (head < 0 || head > a.n_free)) bits = PRHS_DEV_BAD_LEN;
  if (bits == 0 && taken > a.n_free - head) bits = PRHS_DEV_CAPACITY;
  cluster.sync();

  const int chunks = (most + PG_TASK - 1) / PG_TASK;
  const long long tasks = (long long)B * chunks;
  const long long x0 = tasks * gw / gws, x1 = tasks * (gw + 1) / gws;
  // A lane's released entries of a task (-2: none), and the number of its first entry.
  auto released = [&](long long x, auto&& act) {
    const int b = (int)(x / chunks), j0 = (int)(x % chunks) * PG_TASK + lane;
    const PageRow r = a.rows[b];
    int p[PG_COLS];
#pragma unroll
    for (int k = 0; k < PG_COLS; k++) {
      const int j = j0 + 32 * k;
      p[k] = j >= r.released && j < r.held && r.len >= 0 ? table[(long long)b * M + j] : -2;
    }
    act(p, b * M + j0);
  };
  auto in_pool = [&](int p) { return (unsigned)p < (unsigned)kv.num_blocks; };
  // Entries joined (sign 1) or given up again (sign -1), and releases.
  auto counts = [&](int sign, bool check) {
    for (long long x = x0; x < x1; x++) {
      unsigned bad = 0;
      released(x, [&](int(&p)[PG_COLS], int) {
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) {
          if (in_pool(p[k])) atomicAdd(&a.shares_out[p[k]], -sign);
          else if (p[k] != -2) bad = PRHS_DEV_BAD_BLOCK;
        }
      });
      if constexpr (FORK) {
        const int b = (int)(x / chunks), j0 = (int)(x % chunks) * PG_TASK + lane, n = count[b];
        if (n > 0) {
          const int whole = kv.seq_lens[b] / page;  // a last page in part is taken over below
          int p[PG_COLS];
#pragma unroll
          for (int k = 0; k < PG_COLS; k++) p[k] = j0 + 32 * k < whole ? table[(long long)b * M + j0 + 32 * k] : -2;
#pragma unroll
          for (int k = 0; k < PG_COLS; k++) {
            if (in_pool(p[k])) atomicAdd(&a.shares_out[p[k]], sign * n);
            else if (p[k] != -2) bad = PRHS_DEV_BAD_BLOCK;
          }
        }
        const PageRow r = a.rows[b];
        if (r.len > 0 && r.len % page != 0 && r.keep == r.blocks && lane == 0 && x % chunks == 0)
          atomicAdd(&a.shares_out[table[(long long)r.from * M + r.keep - 1]], sign);
      }
      if (check && bad != 0) atomicOr(late, (int)bad);
    }
  };
  // ---- counts; the new rows and the rows to copy, while the old table and the free list stand ----
  const long long cells = (long long)B * a.cap;
  auto copies = [&](bool refused) {
    for (long long i = gt; i < cells; i += gts) {
      const int b = (int)(i / a.cap), c = (int)(i - (long long)b * a.cap);
      int from = -1, to = -1;
      if (!refused) {
        const PageRow r = a.rows[b];
        if (FORK) {
          if (r.last >= 0 && c < r.len % page) {
            from = r.last * page + c;
            to = a.free_pages[head + r.taken] * page + c;
          }
        } else if (c >= r.keep * page && c < r.len) {
          const int k = a.keep[i];
          from = table[(long long)b * M + k / page] * page + k % page;
          to = a.free_pages[head + r.taken + c / page - r.keep] * page + c % page;
        }
      }
      a.src[i] = from;
      a.dst[i] = to;
    }
  };
  const bool early = bits != 0;  // refused before any count changed
  copies(early);
  int back = 0, before = 0, given = 0;  // pages that this warp, the warps before it, all warps give back
  if (!early) {
    counts(1, true);
    for (long long x = x0; x < x1; x++) {
      const int b = (int)(x / chunks), j0 = (int)(x % chunks) * PG_TASK + lane;
      const PageRow r = a.rows[b];
      if (r.len < 0) continue;
      const int end = max(r.held, r.blocks);
      int p[PG_COLS];
#pragma unroll
      for (int k = 0; k < PG_COLS; k++) {
        const int j = j0 + 32 * k;
        p[k] = -1;
        if (j < r.keep) p[k] = FORK ? table[(long long)r.from * M + j] : 0;
        else if (j < r.blocks) p[k] = a.free_pages[head + r.taken + j - r.keep];
        if (j >= r.keep && j < r.blocks && !in_pool(p[k])) atomicOr(late, PRHS_DEV_BAD_BLOCK);
      }
#pragma unroll
      for (int k = 0; k < PG_COLS; k++)
        if (j0 + 32 * k >= r.released && j0 + 32 * k < end) a.stage[(long long)b * M + j0 + 32 * k] = p[k];
    }
    cluster.sync();
    bits = *(volatile unsigned*)late;
  }

  // ---- the pages that nobody holds now, each by its first release ----
  if (bits == 0) {
    for (long long x = x0; x < x1; x++)
      released(x, [&](int(&p)[PG_COLS], int id) {
        int c[PG_COLS];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) c[k] = p[k] >= 0 ? __ldcg(&a.shares_out[p[k]]) : 0;
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (c[k] < 0) atomicMin(&a.shares_out[p[k]], INT32_MIN + id + 32 * k);
      });
    cluster.sync();
    // do(k, page) for the releases that free a page
    auto freeing = [&](long long x, auto&& act) {
      released(x, [&](int(&p)[PG_COLS], int id) {
        int c[PG_COLS];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) c[k] = p[k] >= 0 ? __ldcg(&a.shares_out[p[k]]) : 0;
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) act(c[k] == INT32_MIN + id + 32 * k, p[k]);
      });
    };
    for (long long x = x0; x < x1; x++) freeing(x, [&](bool mine, int) { back += mine; });
    back = __reduce_add_sync(FULL_MASK, back);
    if (lane == 0) a.sums[gw] = back;
    cluster.sync();
    const int sum = block_scan(tid < gws ? __ldcg(&a.sums[tid]) : 0, wsum, &given);
    if (tid / PG_WARPS == rank) sh_base[tid % PG_WARPS] = sum;
    __syncthreads();
    before = sh_base[warp];
    const int new_head = head + taken - given;
    if (new_head < 0) {  // no room in front of the free ones
      bits = PRHS_DEV_CAPACITY;
      for (long long x = x0; x < x1; x++)
        freeing(x, [&](bool mine, int p) {
          if (mine) __stcg(&a.shares_out[p], -1);
        });
      cluster.sync();
    } else {
      int at = new_head + before;
      for (long long x = x0; x < x1; x++) {
        if (back > 0)
          freeing(x, [&](bool mine, int p) {
            const unsigned all = __ballot_sync(FULL_MASK, mine);
            if (mine) {
              a.free_out[at + __popc(all & ((1u << lane) - 1))] = p;
              __stcg(&a.shares_out[p], 0);
            }
            at += __popc(all);
          });
        const int b = (int)(x / chunks), j0 = (int)(x % chunks) * PG_TASK + lane;
        const PageRow r = a.rows[b];
        if (r.len < 0) continue;
        const int end = max(r.held, r.blocks);
        int p[PG_COLS];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (j0 + 32 * k >= r.released && j0 + 32 * k < end) p[k] = a.stage[(long long)b * M + j0 + 32 * k];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (j0 + 32 * k >= r.released && j0 + 32 * k < end) a.table_out[(long long)b * M + j0 + 32 * k] = p[k];
      }
      for (int b = gt; b < B; b += gts) {
        const PageRow r = a.rows[b];
        a.lens_out[b] = r.len < 0 ? kv.seq_lens[b] : r.len;
        a.n_pages_out[b] = r.len < 0 ? a.n_pages[b] : r.blocks;
      }
      if (gt == 0) a.head_out[0] = new_head;
      return;
    }
  }

  // ---- refused: everything as it was, nothing to copy ----
  if (!early) {
    counts(-1, false);
    copies(true);
  }
  for (int b = gt; b < B; b += gts) {
    a.lens_out[b] = kv.seq_lens[b];
    a.n_pages_out[b] = a.n_pages[b];
  }
  if (gt == 0) {
    a.head_out[0] = head;
    raise_error(kv.err, bits);
  }
}

// -------------------------------------------------------------------------- //
// host side
// -------------------------------------------------------------------------- //
static size_t pages_up(size_t x) { return (x + 255) / 256 * 256; }
static size_t pages_chunks(const KVView& kv) { return ((size_t)kv.t_max + PG_KEEP - 1) / PG_KEEP; }
static size_t pages_bytes(const KVView& kv, size_t* at) {
  const size_t B = kv.B;
  at[0] = 0;
  at[1] = at[0] + pages_up(B * sizeof(PageRow));
  at[2] = at[1] + pages_up(B * kv.max_blocks * sizeof(int32_t));
  at[3] = at[2] + pages_up(B * pages_chunks(kv) * sizeof(int2));
  return at[3] + pages_up((PG_CLUSTER * PG_WARPS + 1) * sizeof(int));
}
size_t pages_workspace(const KVView& kv) {
  size_t at[4];
  return pages_bytes(kv, at);
}
void pages_split(PagesLaunch* a, void* ws) {
  size_t at[4];
  pages_bytes(a->kv, at);
  char* w = static_cast<char*>(ws);
  a->rows = reinterpret_cast<PageRow*>(w + at[0]);
  a->stage = reinterpret_cast<int32_t*>(w + at[1]);
  a->part = reinterpret_cast<int2*>(w + at[2]);
  a->sums = reinterpret_cast<int*>(w + at[3]);
}

template <bool FORK>
static cudaError_t pages_go(const PagesLaunch& a, cudaStream_t st) {
  auto k = pages_kernel<FORK>;
  const size_t smem = FORK ? (size_t)a.kv.B * 2 * sizeof(int) : 0;
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  // a CTA while its warps have a few tasks each
  const long long work = (long long)a.kv.B * a.kv.max_blocks + (long long)a.kv.B * a.cap;
  int cl = 1;
  while (cl < PG_CLUSTER && work > (long long)cl * PG_THREADS * PG_COLS) cl *= 2;
  if (cl > 8 && (e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cl);
  cfg.blockDim = dim3(PG_THREADS);
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
  return cudaLaunchKernelEx(&cfg, k, a);
}

cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t st) {
  return a.parent != nullptr ? pages_go<true>(a, st) : pages_go<false>(a, st);
}

}  // namespace prhs
