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
// The entries of the table are tasks of 128 columns of a row, a warp's tasks
// consecutive, so that a prefix over the warps' counts gives every freed page its
// place. One cluster of CTAs, or for large tables all SMs (a cooperative launch).
// Bound: latency, six or seven dependent passes through L2 with a barrier between two, 1 us
// each for a cluster, 2 for the grid; for large calls atomics on shared pages too. From a graph, 64 beams
// of 3.7 to 7.9K keys on 16-key pages trade places in 14.4 us (plans, sums and error bits through
// L2 instead of the CTAs' shared memory, new columns read back: 15.6), 512 rows of up to 2173
// pages in 41 (a cluster alone: 178; bytes 1.4), one row of 4096 positions is compacted in 14.5,
// 117 rows of up to 19.6K in 29 (53 with one cluster).
#include <cooperative_groups.h>

#include "pages.h"

namespace prhs {

namespace cg = cooperative_groups;

constexpr int PG_THREADS = 512;          // (a lane holds a task's entries over the passes)
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_CLUSTER = 16;           // above 8 by opt-in
constexpr int PG_GRID = 256;             // CTAs of a cooperative launch at most
constexpr int PG_COLS = 4;               // columns a lane (16: a pass's code is fetched once and used once, 18.5 -> 28.7 us for 64 rows)
constexpr int PG_TASK = 32 * PG_COLS;    // columns of a task
constexpr long long PG_ONE_CLUSTER = 1 << 16;  // entries up to which one cluster takes a call
constexpr int PG_KEEP = 128;             // kept positions a warp checks at a time
constexpr int PG_LOCAL = PG_THREADS;     // rows up to which every CTA of a cluster keeps all plans itself

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
  int before = lane < warp ? wsum[lane] : 0, all = lane < PG_WARPS ? wsum[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(FULL_MASK, before, o);
    all += __shfl_xor_sync(FULL_MASK, all, o);
  }
  *total = all;
  return before + y - x;
}

// n numbers copied by nt threads, four 16-byte pieces of each in flight where the arrays allow.
__device__ __forceinline__ void copy_ints(int32_t* dst, const int32_t* src, long long n, int t, int nt) {
  long long i = 0;
  if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src)) & 15) == 0) {
    i = n / 4 * 4;
    for (long long x0 = t; x0 < n / 4; x0 += 4ll * nt) {
      int4 v[4];
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (x0 + (long long)k * nt < n / 4) v[k] = reinterpret_cast<const int4*>(src)[x0 + (long long)k * nt];
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (x0 + (long long)k * nt < n / 4) reinterpret_cast<int4*>(dst)[x0 + (long long)k * nt] = v[k];
    }
  }
  for (i += t; i < n; i += nt) dst[i] = src[i];
}

template <bool FORK, bool GRID>
__global__ void __launch_bounds__(PG_THREADS, 1) pages_kernel(const __grid_constant__ PagesLaunch a) {
  extern __shared__ int pg_smem[];
  __shared__ int wsum[PG_WARPS];
  __shared__ int sh_most, sh_base[PG_WARPS];
  __shared__ unsigned sh_bits;
  // A cluster's CTAs write these into each other's: what the others would read through L2, at 0.7 us
  __shared__ __align__(16) PageRow sh_rows[GRID ? 1 : PG_LOCAL];
  __shared__ int sh_sums[GRID ? 1 : PG_CLUSTER * PG_WARPS];
  __shared__ unsigned sh_late;
  const int rank = blockIdx.x, ranks = gridDim.x;
  auto meet = [] {
    if constexpr (GRID) cg::this_grid().sync();
    else cg::this_cluster().sync();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gw = rank * PG_WARPS + warp, gws = ranks * PG_WARPS;      // the warp among the cluster's
  const int gt = rank * PG_THREADS + tid, gts = ranks * PG_THREADS;
  const KVView& kv = a.kv;
  const int B = kv.B, M = kv.max_blocks, page = kv.block_size;
  const int32_t* table = kv.block_table;
  int* first = pg_smem;     // fork, [B]: the first child of each row that takes a part of its last page
  int* count = first + B;   //       [B]: its children
  int* late = a.sums + gws;  // (all SMs)
  const bool local = !GRID && B <= PG_LOCAL;

  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    sh_bits = 0;
    sh_late = 0;
    sh_most = 0;
  }
  if (GRID && gt == 0) *late = 0;
  if (a.shares_out != a.shares) copy_ints(a.shares_out, a.shares, kv.num_blocks, gt, gts);
  if (a.free_out != a.free_pages) copy_ints(a.free_out, a.free_pages, a.n_free, gt, gts);
  if (a.table_out != table) copy_ints(a.table_out, table, (long long)B * M, gt, gts);
  const int head = a.free_head[0];

  // ---- what every row becomes ----
  if constexpr (FORK) {
    for (int b = tid; b < B; b += PG_THREADS) {
      first[b] = B;
      count[b] = 0;
      // (a row's last page and its holders beside its parent, not behind it)
      const int t = kv.seq_lens[b];
      if (t > 0 && t <= kv.t_max) {
        const int last = table[(long long)b * M + (t - 1) / page];
        if ((unsigned)last < (unsigned)kv.num_blocks) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.shares + last));
      }
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
    meet();
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
#pragma unroll 4
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
  PageRow r0 = {};  // (the thread's only row of batches up to PG_THREADS)
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
    if (local) sh_rows[b] = r0;
    else if (b % ranks == rank) a.rows[b] = r0;
  }
  __syncthreads();
  bits = sh_bits;
  most = min(sh_most, M);
  if (bits == 0 && (head < 0 || head > a.n_free)) bits = PRHS_DEV_BAD_LEN;
  if (bits == 0 && taken > a.n_free - head) bits = PRHS_DEV_CAPACITY;
  // Counts change when all CTAs have read what they plan by; with the plans at hand, what comes
  // before that does not wait.
  if constexpr (GRID) meet();
  else asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  auto planned = [] {
    if constexpr (!GRID) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  if (!local) planned();
  auto row_of = [&](int b) -> PageRow { return local ? sh_rows[GRID ? 0 : b] : a.rows[b]; };

  const int chunks = (most + PG_TASK - 1) / PG_TASK;
  const long long tasks = (long long)B * chunks;
  const long long x0 = tasks * gw / gws, x1 = tasks * (gw + 1) / gws;
  // A lane's share of a task: columns j0 + 32 k, and the entries released there (-2: none).
  struct Task {
    PageRow r;
    int b, j0, p[PG_COLS];
  };
  auto ask = [&](long long x) {
    Task t;
    t.b = (int)(x / chunks);
    t.j0 = (int)(x - (long long)t.b * chunks) * PG_TASK + lane;
    t.r = row_of(t.b);
#pragma unroll
    for (int k = 0; k < PG_COLS; k++) {
      const int j = t.j0 + 32 * k;
      t.p[k] = j >= t.r.released && j < t.r.held && t.r.len >= 0 ? table[(long long)t.b * M + j] : -2;
    }
    return t;
  };
  // The warp's tasks in order; the first one's entries stay in registers over the passes (most
  // calls have no more), the next one's come in behind the one that is worked on.
  Task own = {};
  if (x0 < x1) own = ask(x0);
  auto sweep = [&](auto&& act) {
    Task t = own;
    for (long long x = x0; x < x1; x++) {
      Task next;
      if (x + 1 < x1) next = ask(x + 1);
      act(t, x == x0);
      t = next;
    }
  };
  auto in_pool = [&](int p) { return (unsigned)p < (unsigned)kv.num_blocks; };
  // Entries joined (sign 1) or given up again (sign -1), and releases.
  auto counts = [&](const Task& t, int sign) {
    unsigned bad = 0;
#pragma unroll
    for (int k = 0; k < PG_COLS; k++) {
      if (in_pool(t.p[k])) atomicAdd(&a.shares_out[t.p[k]], -sign);
      else if (t.p[k] != -2) bad = PRHS_DEV_BAD_BLOCK;
    }
    if constexpr (FORK) {
      const int n = count[t.b];
      if (n > 0) {
        const int whole = kv.seq_lens[t.b] / page;  // a last page in part is taken over below
        int p[PG_COLS];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) p[k] = t.j0 + 32 * k < whole ? table[(long long)t.b * M + t.j0 + 32 * k] : -2;
#pragma unroll
        for (int k = 0; k < PG_COLS; k++) {
          if (in_pool(p[k])) atomicAdd(&a.shares_out[p[k]], sign * n);
          else if (p[k] != -2) bad = PRHS_DEV_BAD_BLOCK;
        }
      }
      if (t.r.len > 0 && t.r.len % page != 0 && t.r.keep == t.r.blocks && t.j0 == 0)
        atomicAdd(&a.shares_out[table[(long long)t.r.from * M + t.r.keep - 1]], sign);
    }
    return bad;
  };
  // Columns that change, and the rows to copy, while the old table and the free list stand.
  auto changes = [&](const Task& t, int k) {
    const int j = t.j0 + 32 * k;
    return t.r.len >= 0 && j >= t.r.released && j < max(t.r.held, t.r.blocks);
  };
  auto copies = [&](bool refused) {
    const int per_row = (a.cap + PG_TASK - 1) / PG_TASK;
    for (long long x = gw; x < (long long)B * per_row; x += gws) {
      const int b = (int)(x / per_row), c0 = (int)(x - (long long)b * per_row) * PG_TASK + lane;
      const PageRow r = row_of(b);
      int k[PG_COLS], from[PG_COLS], to[PG_COLS];
#pragma unroll
      for (int i = 0; i < PG_COLS; i++) {
        const int c = c0 + 32 * i;
        k[i] = -1;
        if (refused) continue;
        if (FORK) {
          if (r.last >= 0 && c < r.len % page) k[i] = c;
        } else if (c >= r.keep * page && c < r.len) {
          k[i] = a.keep[(long long)b * a.cap + c];
        }
      }
#pragma unroll
      for (int i = 0; i < PG_COLS; i++) {
        if (k[i] < 0) continue;
        from[i] = FORK ? r.last : table[(long long)b * M + k[i] / page];
        to[i] = a.free_pages[head + r.taken + (FORK ? 0 : (c0 + 32 * i) / page - r.keep)];
      }
#pragma unroll
      for (int i = 0; i < PG_COLS; i++) {
        const int c = c0 + 32 * i;
        if (c >= a.cap) break;
        a.src[(long long)b * a.cap + c] = k[i] < 0 ? -1 : from[i] * page + k[i] % page;
        a.dst[(long long)b * a.cap + c] = k[i] < 0 ? -1 : to[i] * page + c % page;
      }
    }
  };
  const bool early = bits != 0;  // refused before any count changed
  copies(early);
  if (local) planned();
  int kept[PG_COLS] = {};  // the first task's new columns, of which it frees `freed`
  unsigned freed = 0;
  int back = 0, before = 0, given = 0;  // pages that this warp, the warps before it, all warps give back
  if (!early) {
    sweep([&](const Task& t, bool own_task) {
      unsigned bad = counts(t, 1);
      int p[PG_COLS];
#pragma unroll
      for (int k = 0; k < PG_COLS; k++) {
        const int j = t.j0 + 32 * k;
        p[k] = -1;
        if (!changes(t, k)) continue;
        if (j < t.r.keep) p[k] = FORK ? table[(long long)t.r.from * M + j] : 0;
        else if (j < t.r.blocks) p[k] = a.free_pages[head + t.r.taken + j - t.r.keep];
      }
#pragma unroll
      for (int k = 0; k < PG_COLS; k++) {
        const int j = t.j0 + 32 * k;
        if (!changes(t, k)) continue;
        if (j >= t.r.keep && j < t.r.blocks && !in_pool(p[k])) bad |= PRHS_DEV_BAD_BLOCK;
        if (own_task) kept[k] = p[k];
        else a.stage[(long long)t.b * M + j] = p[k];
      }
      if (bad != 0) {
        if constexpr (GRID) atomicOr(late, (int)bad);
        else
          for (int r = 0; r < ranks; r++) atomicOr(cg::this_cluster().map_shared_rank(&sh_late, r), bad);
      }
    });
    meet();
    bits = GRID ? *(volatile unsigned*)late : *(volatile unsigned*)&sh_late;
  }

  // ---- the pages that nobody holds now, each by its first release ----
  if (bits == 0) {
    auto held_by = [&](const Task& t, int(&c)[PG_COLS]) {
#pragma unroll
      for (int k = 0; k < PG_COLS; k++) c[k] = t.p[k] >= 0 ? __ldcg(&a.shares_out[t.p[k]]) : 0;
    };
    auto frees = [&](const Task& t, int k, int count) { return count == INT32_MIN + t.b * M + t.j0 + 32 * k; };
    sweep([&](const Task& t, bool) {
      int c[PG_COLS];
      held_by(t, c);
#pragma unroll
      for (int k = 0; k < PG_COLS; k++)
        if (c[k] < 0) atomicMin(&a.shares_out[t.p[k]], INT32_MIN + t.b * M + t.j0 + 32 * k);
    });
    meet();
    sweep([&](const Task& t, bool own_task) {
      int c[PG_COLS];
      held_by(t, c);
#pragma unroll
      for (int k = 0; k < PG_COLS; k++) {
        const bool mine = frees(t, k, c[k]);
        back += mine;
        if (own_task && mine) freed |= 1u << k;
      }
    });
    back = __reduce_add_sync(FULL_MASK, back);
    if constexpr (GRID) {
      if (lane == 0) a.sums[gw] = back;
    } else if (lane < ranks) {
      cg::this_cluster().map_shared_rank(sh_sums, lane)[gw] = back;
    }
    meet();
    auto given_by = [&](int w) { return GRID ? __ldcg(&a.sums[w]) : sh_sums[GRID ? 0 : w]; };
    const int share = (gws + PG_THREADS - 1) / PG_THREADS, w0 = min(gws, tid * share), w1 = min(gws, w0 + share);
    int sum = 0;
    for (int w = w0; w < w1; w++) sum += given_by(w);
    sum = block_scan(sum, wsum, &given);
    for (int w = w0; w < w1; w++) {
      if (w / PG_WARPS == rank) sh_base[w % PG_WARPS] = sum;
      sum += given_by(w);
    }
    __syncthreads();
    before = sh_base[warp];
    const int new_head = head + taken - given;
    if (new_head < 0) {  // no room in front of the free ones
      bits = PRHS_DEV_CAPACITY;
      sweep([&](const Task& t, bool) {
        int c[PG_COLS];
        held_by(t, c);
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (frees(t, k, c[k])) __stcg(&a.shares_out[t.p[k]], -1);
      });
      meet();
    } else {
      int at = new_head + before;
      sweep([&](const Task& t, bool own_task) {
        int p[PG_COLS];
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (changes(t, k)) p[k] = own_task ? kept[k] : a.stage[(long long)t.b * M + t.j0 + 32 * k];
        if (back > 0) {
          int c[PG_COLS];
          if (!own_task) held_by(t, c);
#pragma unroll
          for (int k = 0; k < PG_COLS; k++) {
            const bool mine = own_task ? freed >> k & 1 : frees(t, k, c[k]);
            const unsigned all = __ballot_sync(FULL_MASK, mine);
            if (mine) {
              a.free_out[at + __popc(all & ((1u << lane) - 1))] = t.p[k];
              __stcg(&a.shares_out[t.p[k]], 0);
            }
            at += __popc(all);
          }
        }
#pragma unroll
        for (int k = 0; k < PG_COLS; k++)
          if (changes(t, k)) a.table_out[(long long)t.b * M + t.j0 + 32 * k] = p[k];
      });
      for (int b = gt; b < B; b += gts) {
        const PageRow r = row_of(b);
        a.lens_out[b] = r.len < 0 ? kv.seq_lens[b] : r.len;
        a.n_pages_out[b] = r.len < 0 ? a.n_pages[b] : r.blocks;
      }
      if (gt == 0) a.head_out[0] = new_head;
      return;
    }
  }

  // ---- refused: everything as it was, nothing to copy ----
  if (!early) {
    sweep([&](const Task& t, bool) { counts(t, -1); });
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
  return at[3] + pages_up((PG_GRID * PG_WARPS + 1) * sizeof(int));
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

template <bool FORK, bool GRID>
static cudaError_t pages_go(const PagesLaunch& a, int ctas, cudaStream_t st) {
  auto k = pages_kernel<FORK, GRID>;
  const size_t smem = FORK ? (size_t)a.kv.B * 2 * sizeof(int) : 0;
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(k, smem, smem_set);
  if (e != cudaSuccess) return e;
  if (!GRID && ctas > 8 && (e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(PG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  if (GRID) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  }
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.kv.pdl && !GRID ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

cudaError_t launch_pages(const PagesLaunch& a, int sms, cudaStream_t st) {
  // a CTA while its warps have a task each
  const long long work = (long long)a.kv.B * a.kv.max_blocks + (long long)a.kv.B * a.cap;
  int cl = 1;
  while (cl < PG_CLUSTER && work > (long long)cl * PG_THREADS * PG_COLS) cl *= 2;
  if (work <= PG_ONE_CLUSTER) return a.parent != nullptr ? pages_go<true, false>(a, cl, st) : pages_go<false, false>(a, cl, st);
  const long long most = (work + PG_THREADS * PG_COLS - 1) / (PG_THREADS * PG_COLS);
  int ctas = sms < PG_GRID ? sms : PG_GRID;
  if (most < ctas) ctas = (int)most;
  return a.parent != nullptr ? pages_go<true, true>(a, ctas, st) : pages_go<false, true>(a, ctas, st);
}

}  // namespace prhs
