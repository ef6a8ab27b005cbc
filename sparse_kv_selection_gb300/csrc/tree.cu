// Attention of a batch of new tokens over their sequences' caches and over
// each other (a tree by its masks, or a causal chunk), fp32 on the CUDA cores
// (the tensor cores' fp32 forms drop mantissa bits).
//
// The G query heads of one KV head see the same keys, so the rows of one
// (sequence, KV head) are its tokens times G (row = token * G + head of the
// group), cut into units of up to 8, 32 or 64 rows. A unit's keys are tiles of 32:
// the cache's, then the new tokens' (one word of a tree mask each). All tiles of
// all units are one list; every CTA takes an equal run of it, so long caches are
// split and short ones packed without a plan made on the host. A unit cut by a
// run's end leaves partial states in the workspace, which a second launch joins
// row by row.
//
// Inside a CTA the last warp walks the list and looks the pages of a tile up a
// tile before its copies start; all threads copy the next tiles (16-byte
// asynchronous copies, eight threads a key) while they work on the current one. A
// warp holds TY R rows: 32 / TY lanes share a row and take TY keys each for the
// logits, D TY / 32 columns each for the product with V, so that a row's maximum,
// sum and weights stay inside the warp. Products are packed pairs of fp32;
// everything is fp32. A warp without rows in a unit only copies.
//
// Bound: shared-memory reads. They move 128 bytes a clock into registers whether
// lanes share an address or not, and a lane's block of R rows by TY keys costs
// (R + TY) 16-byte reads for 4 R TY products, 4 (R + TY) / (R TY) times what the
// products take: 2 at 4 by 4, 3 at 2 by 4, 5 at 1 by 4 (the product with V has more
// columns a lane: 1.25 at 4 by 4). Hence the forms at the end of this file.
// Two causal chunks of 1024 tokens on 512 keys, 8 / 2 heads, d = 128: 227 us, 38
// TFLOP/s; single tokens of 16 heads over 69 206 keys, 4 KV heads, 16-key pages: 63
// us, 4.5 TB/s; 27 trees of 21 tokens over up to 1899 keys, 8 heads, d = 64: 63 us. With
// shared keys: 128 tokens in 8 groups, 4 KV heads, up to 1.4K keys, 112 us (bytes 43).
#include "tree_join.cuh"

namespace prhs {

constexpr int TK = 32;            // keys of a tile: a word of a tree mask
constexpr int FOLD = 32;          // tiles summed one by one
constexpr float T_LOG2E = 1.4426950408889634f;

// A tile of a CTA's run.
struct __align__(16) TreeStep {
  int e, kvh, block, tile;  // item, KV head, unit of theirs, tile of the unit
  int tiles, c0, n, t;      // the unit's tiles, first token, tokens, cached keys
  int b, base, part, pad;   // row of the cache, its first key here, where the state goes (TreeItem)
  int tile0, left, q, u;    // the unit's first tile in this run, tiles of the run behind this one, Q slot, tokens of a unit
};

template <int D, int TY, int R, int W, int CTAS>
struct TreeShape {
  static constexpr int TR = TY * R * W;          // rows of a unit
  static constexpr int TR_LOG2 = TR == 64 ? 6 : TR == 32 ? 5 : 3;
  static_assert(TR == 1 << TR_LOG2, "rows of a unit");
  static constexpr int THREADS = 32 * W;
  static constexpr int LD = D + 4;               // row stride of Q and K: eight rows' 16-byte reads hit distinct banks
  static constexpr int LP = TK + 4;              // row stride of the weights
  static constexpr int STAGE = TK * (LD + D);    // floats of a K and a V tile
  // Q slots: one a stage, so that the next units' Q comes with their first tiles, or one
  static constexpr int LIMIT = 228 * 1024 / CTAS - 1024 - 2560;  // a CTA's share, less what is reserved and static
  static constexpr int bytes(int stages, int slots) { return 4 * (stages * STAGE + slots * TR * LD + TR * LP); }
  static constexpr int STAGES = bytes(3, 3) <= LIMIT ? 3 : 2;
  static constexpr int STEPS = STAGES == 2 ? 4 : 8;  // tiles known at once: those in flight and two more
  static constexpr int QS = bytes(STAGES, STAGES) <= LIMIT ? STAGES : 1;
  static constexpr size_t SMEM = bytes(STAGES, QS);
  static_assert(bytes(STAGES, QS) <= LIMIT, "shared memory");
};

struct TreeSeq : TreeItem {  // one item's share of the list
  int u, blocks, cache_tiles;  // (u: tokens of a unit)
  long long tiles;  // of one KV head
};

// Tokens that unit `block` of u tokens may attend, and its tiles: a causal unit
// sees the tokens up to its own last one, a tree unit all of them, a unit over
// shared keys (part 1) none.
__device__ __forceinline__ int tree_keys(int n, int block, int u, bool causal) {
  const long long end = ((long long)block + 1) * u;
  return causal && end < n ? (int)end : n;
}
__device__ __forceinline__ int tree_tiles(int t, int n, int block, int u, bool causal, int part) {
  return (int)(((long long)t + TK - 1) / TK) +
         (part == 1 ? 0 : (int)(((long long)tree_keys(n, block, u, causal) + TK - 1) / TK));
}

// New-token tiles of the units before unit j.
constexpr int TREE_EVEN = 4;
__device__ __forceinline__ long long tree_new_before(const TreeSeq& s, long long j, int ul, bool causal) {
  const int all_tiles = tree_tiles(0, s.n, 0, s.n, false, s.part);
  if (!causal || s.part == 1) return j * all_tiles;
  long long sum = 0;
  if (s.blocks <= TREE_EVEN) {
    for (int i = 0; i < j; i++) sum += tree_tiles(0, s.n, i, s.u, true, s.part);
    return sum;
  }
  const bool all = j == s.blocks;
  const long long k = all ? j - 1 : j;  // units that end at their own last token, of 2^ul tokens
  if (ul >= 5) {
    sum = (k * (k + 1) / 2) << (ul - 5);
  } else {  // sum over i = 1 .. k of ceil(i / p), p = 2^(5 - ul)
    const int pl = 5 - ul;
    const long long q = k >> pl, r = k - (q << pl);
    sum = ((q * (q + 1) / 2) << pl) + r * (q + 1);
  }
  return all ? sum + all_tiles : sum;
}

// A sequence's units hold up to 2^ul tokens: equal shares where they are few or
// a tree's (9 tokens of 8 query heads in two units of 64 rows: 5 and 4 tokens, not
// 8 and 1, since the runs count tiles, not rows).
template <bool SHARED>
__device__ __forceinline__ TreeSeq tree_seq(const TreeLaunch& a, int e, int ul) {
  TreeSeq s;
  const bool causal = a.mask == nullptr;
  static_cast<TreeItem&>(s) = tree_item<SHARED>(a, !SHARED || a.items == TREE_BOTH ? e : 2 * e + (a.items == TREE_OWN));
  s.u = 1 << ul;
  s.blocks = (int)(((long long)s.n + s.u - 1) >> ul);
  s.cache_tiles = (int)(((long long)s.t + TK - 1) / TK);
  s.tiles = 0;
  if (s.blocks == 0) return s;
  if (s.blocks <= TREE_EVEN || !causal) {
    s.u = (s.n + s.blocks - 1) / s.blocks;
    s.blocks = (s.n + s.u - 1) / s.u;
  }
  s.tiles = (long long)s.blocks * s.cache_tiles + tree_new_before(s, s.blocks, ul, causal);
  return s;
}

// 16 bytes of global memory to shared memory, zeros when !have.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(have ? 16 : 0)
               : "memory");
}

template <int D, int TY, int R, int W, int CTAS, bool SHARED>
__global__ void __launch_bounds__(32 * W, CTAS) tree_kernel(const __grid_constant__ TreeLaunch a,
                                                                 const __grid_constant__ TreeRecords p) {
  using S = TreeShape<D, TY, R, W, CTAS>;
  constexpr int TR = S::TR, LD = S::LD, LP = S::LP, THREADS = S::THREADS, STEPS = S::STEPS;
  extern __shared__ __align__(16) float tree_smem[];
  float* sq0 = tree_smem + S::STAGES * S::STAGE;
  __shared__ TreeStep steps[STEPS];
  __shared__ long long key_row[STEPS][TK];  // a tile's keys: row of the cache, or the sequence's token; -1: none
  __shared__ uint32_t have_key[STEPS];      // those that exist
  __shared__ long long wsum[W], wgrouped[SHARED ? W : 1];  // (tokens of all groups)

  // Own keys beside the groups' (TREE_OWN): nothing here needs that launch, but the next one
  // needs both, so that this one's last CTA does nothing but wait for it.
  const int ctas = gridDim.x - (SHARED && a.items == TREE_OWN ? 1 : 0), cta = (SHARED ? p.cta0 : 0) + blockIdx.x;
  if (!SHARED || a.items != TREE_OWN || (int)blockIdx.x == ctas) pdl_wait();
  else __threadfence();  // (that launch has waited for all that was before it; no L1 keeps older lengths or tables)
  pdl_trigger();
  if (SHARED && (int)blockIdx.x == ctas) return;
  const KVView& kv = a.kv;
  const bool causal = a.mask == nullptr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gl = p.group_log2, ul = S::TR_LOG2 - gl;  // log2 of the group and of a unit's tokens

  // ---- this CTA's run of the list of all tiles ----
  const int items = SHARED && a.items == TREE_BOTH ? 2 * kv.B : kv.B;
  const int per_t = (items + THREADS - 1) / THREADS, e0 = tid * per_t;
  long long mine = 0, grouped = 0;
  bool back = false;  // offsets that step back: sequences would overlap, without bound
  for (int e = e0; e < min(items, e0 + per_t); e++) {
    const TreeSeq s = tree_seq<SHARED>(a, e, ul);
    mine += kv.Hkv * s.tiles;
    if (SHARED && s.part == 1) grouped += s.n;
    back |= a.cu_new[s.b + 1] < a.cu_new[s.b];
  }
  long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(FULL_MASK, run, o);
    if (lane >= o) run += y;
  }
  if constexpr (SHARED) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) grouped += __shfl_xor_sync(FULL_MASK, grouped, o);
    if (lane == 0) wgrouped[warp] = grouped;
  }
  if (lane == 31) wsum[warp] = run;
  back = __syncthreads_or(back);  // (flagged by tree_seq)
  if constexpr (SHARED) {
    grouped = 0;
#pragma unroll
    for (int w = 0; w < W; w++) grouped += wgrouped[w];
    if (groups_overlap(a, grouped, tid)) back = true;
    // (the groups' launch sees what there is to see)
    if (a.items != TREE_OWN && blockIdx.x == 0 && tid == 0) *a.part_ok = !back;
  }
  long long total = 0, before = run - mine;
#pragma unroll
  for (int w = 0; w < W; w++) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const long long per = (total + ctas - 1) / ctas, g0 = blockIdx.x * per;
  const int count = (int)(min(total, g0 + per) - g0);  // negative: none are left
  if (count <= 0 || back) {
    if (tid == 0) p.split[cta] = TreeSplit{};
    return;
  }
  if (g0 >= before && g0 < before + mine) {  // the run begins in this thread's items
    long long off = g0 - before;
    int e = e0;
    TreeSeq s = tree_seq<SHARED>(a, e, ul);
    while (off >= kv.Hkv * s.tiles) {
      off -= kv.Hkv * s.tiles;
      s = tree_seq<SHARED>(a, ++e, ul);
    }
    TreeStep x;
    x.e = e;
    x.b = s.b;
    x.base = s.base;
    x.part = s.part;
    x.kvh = (int)(off / s.tiles);
    off -= x.kvh * s.tiles;
    int lo = 0, hi = s.blocks - 1;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if ((long long)mid * s.cache_tiles + tree_new_before(s, mid, ul, causal) <= off) lo = mid; else hi = mid - 1;
    }
    x.block = lo;
    x.tile = x.tile0 = (int)(off - (long long)lo * s.cache_tiles - tree_new_before(s, lo, ul, causal));
    x.tiles = tree_tiles(s.t, s.n, lo, s.u, causal, s.part);
    x.c0 = s.c0;
    x.n = s.n;
    x.t = s.t;
    x.left = count - 1;
    x.q = 0;
    x.u = s.u;
    steps[0] = x;
  }
  __syncthreads();

  // The step behind `x` (x.left > 0): one thread; with shared keys a warp, since most items
  // may then have no tiles: 32 are looked at together.
  auto advance = [&](TreeStep x) {
    x.left--;
    if (++x.tile == x.tiles) {
      x.tile = x.tile0 = 0;
      x.q = x.q + 1 == S::QS ? 0 : x.q + 1;
      if ((long long)++x.block * x.u >= x.n) {
        x.block = 0;
        if (++x.kvh == kv.Hkv) {
          x.kvh = 0;
          TreeSeq s = {};
          if constexpr (SHARED) {
            unsigned some = 0;
            int e = x.e + 1 + lane;
            for (;; e += 32) {
              if (e < items) s = tree_seq<SHARED>(a, e, ul); else s.n = 0;
              some = __ballot_sync(FULL_MASK, s.n > 0);
              if (some != 0 || e - lane + 32 >= items) break;
            }
            const int from = some != 0 ? __ffs(some) - 1 : 0;
            x.e = e - lane + from;
            s.b = __shfl_sync(FULL_MASK, s.b, from);
            s.base = __shfl_sync(FULL_MASK, s.base, from);
            s.part = __shfl_sync(FULL_MASK, s.part, from);
            s.c0 = __shfl_sync(FULL_MASK, s.c0, from);
            s.n = __shfl_sync(FULL_MASK, s.n, from);
            s.t = __shfl_sync(FULL_MASK, s.t, from);
            s.u = __shfl_sync(FULL_MASK, s.u, from);
          } else {
            while (s.n == 0 && ++x.e < items) s = tree_seq<SHARED>(a, x.e, ul);
          }
          x.b = s.b;
          x.base = s.base;
          x.part = s.part;
          x.c0 = s.c0;
          x.n = s.n;
          x.t = s.t;
          x.u = s.u;
        }
      }
      x.tiles = tree_tiles(x.t, x.n, x.block, x.u, causal, x.part);
    }
    return x;
  };
  // All threads: a unit's Q rows (zeros behind its last), and a tile's K and V.
  auto copy_q = [&](const TreeStep& x) {
    float* sq = sq0 + (S::QS > 1 ? x.q : 0) * TR * LD;
#pragma unroll
    for (int i = 0; i < TR * D / 4 / THREADS; i++) {
      const int y = tid + i * THREADS, r = y / (D / 4), c = y % (D / 4) * 4;
      const int jj = r >> gl;
      const long long j = (long long)x.block * x.u + jj;
      const bool have = jj < x.u && j < x.n;
      copy16(sq + r * LD + c,
             static_cast<const float*>(a.q) +
                 (have ? ((x.c0 + j) * kv.Hq + (x.kvh << gl) + (r & ((1 << gl) - 1))) * D + c : 0),
             have);
    }
  };
  auto copy_tile = [&](const TreeStep& x, int stage, int slot) {
    float* sk = tree_smem + stage * S::STAGE;
    float* sv = sk + TK * LD;
    const int c = (tid & 7) * 4;
    const bool cached = x.tile < (int)(((long long)x.t + TK - 1) / TK);
    const float* kb = cached ? static_cast<const float*>(kv.k) : static_cast<const float*>(a.k_new) + x.c0 * a.ks + x.kvh * D;
    const float* vb = cached ? static_cast<const float*>(kv.v) : static_cast<const float*>(a.v_new) + x.c0 * a.vs + x.kvh * D;
    const long long ks = cached ? D : a.ks, vs = cached ? D : a.vs;
#pragma unroll
    for (int key = tid >> 3; key < TK; key += THREADS / 8) {
      const long long row = key_row[slot][key];
      const bool have = row >= 0;
      const float *kp = kb + (have ? row * ks : 0) + c, *vp = vb + (have ? row * vs : 0) + c;
#pragma unroll
      for (int q = 0; q < D / 32; q++) {
        copy16(sk + key * LD + c + q * 32, kp + q * 32, have);
        copy16(sv + key * D + c + q * 32, vp + q * 32, have);
      }
    }
  };
  // One warp: where a tile's keys are, a key a lane.
  auto find = [&](const TreeStep& x) -> long long {
    const int ct = (int)(((long long)x.t + TK - 1) / TK);
    const bool cached = x.tile < ct;
    const int i = (cached ? x.tile : x.tile - ct) * TK + lane;
    if (i >= (cached ? x.t : tree_keys(x.n, x.block, x.u, causal))) return -1;
    return cached ? kv_row(kv, x.b, x.kvh, (SHARED ? x.base : 0) + i) : i;
  };
  auto found = [&](const TreeStep& x, int slot, long long row) {
    key_row[slot][lane] = row;
    const unsigned have = __ballot_sync(FULL_MASK, row >= 0);
    if (lane == 0) have_key[slot] = have;
    if (row < 0 && x.tile * TK + lane < x.t) raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
  };

  constexpr int AHEAD = S::STAGES;  // tiles that have been looked up when the loop begins
  if (warp == W - 1) {
    if (SHARED || lane == 0)
      for (int i = 1; i < min(AHEAD + 1, count); i++) {
        const TreeStep y = advance(steps[i - 1]);
        if (lane == 0) steps[i] = y;
        if (SHARED) __syncwarp();
      }
    __syncwarp();
    long long row[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; i++) row[i] = i < count ? find(steps[i]) : -1;
#pragma unroll
    for (int i = 0; i < AHEAD; i++)
      if (i < count) found(steps[i], i, row[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; i++) {
    if (i < count) {
      if (S::QS > 1 && steps[i].tile == steps[i].tile0) copy_q(steps[i]);
      copy_tile(steps[i], i, i);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  constexpr int TX = 32 / TY, KT = TK / TX, C4 = D / (4 * TX);  // lanes a row, keys and column groups a lane
  const int ty = lane / TX, tx = lane % TX;  // rows wrow + ty + TY i; keys tx + TX k; columns (tx + TX c) 4
  const int wrow = warp * TY * R;
  const float qs = a.scale * T_LOG2E;
  float* sp = sq0 + S::QS * TR * LD + wrow * LP;
  float m[R], l[R];
  uint64_t o[R][2 * C4];  // column pairs
  int stage = 0;
  for (int it = 0; it < count; it++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
    __syncthreads();  // the tile is here, and everyone is done with the one before it
    const TreeStep x = steps[it & (STEPS - 1)];
    {
      const int nx = it + S::STAGES - 1;
      if (S::QS == 1 && x.tile == x.tile0) {
        copy_q(x);
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncthreads();
      }
      if (nx < count) {
        const TreeStep& y = steps[nx & (STEPS - 1)];
        if (S::QS > 1 && y.tile == y.tile0) copy_q(y);
        copy_tile(y, stage == 0 ? S::STAGES - 1 : stage - 1, nx & (STEPS - 1));
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // the last warp looks the tile after those up (its page numbers come in
    // while it computes), and one lane walks on
    const int look = it + AHEAD;
    long long row = -1;
    if (warp == W - 1 && look < count) {
      row = find(steps[look & (STEPS - 1)]);
      if ((SHARED || lane == 0) && look + 1 < count) {
        const TreeStep y = advance(steps[look & (STEPS - 1)]);
        if (lane == 0) steps[(look + 1) & (STEPS - 1)] = y;
      }
    }
    const float* sk = tree_smem + stage * S::STAGE;
    const float* sv = sk + TK * LD;
    const float* sq = sq0 + (S::QS > 1 ? x.q : 0) * TR * LD;
    if (++stage == S::STAGES) stage = 0;
    const long long row0 = ((long long)x.block * x.u) << gl;
    const int rows = (int)min((long long)x.u << gl, ((long long)x.n << gl) - row0);
    if (wrow >= rows) {
      if (warp == W - 1 && look < count) found(steps[look & (STEPS - 1)], look & (STEPS - 1), row);
      continue;
    }

    if (x.tile == x.tile0) {
#pragma unroll
      for (int i = 0; i < R; i++) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 2 * C4; c++) o[i][c] = 0;
      }
    }
    // ---- logits ----
    uint64_t acc[R][KT];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
      for (int k = 0; k < KT; k++) acc[i][k] = 0;
#pragma unroll 8
    for (int e = 0; e < D; e += 4) {
      ulonglong2 q[R];
#pragma unroll
      for (int i = 0; i < R; i++) q[i] = *reinterpret_cast<const ulonglong2*>(sq + (wrow + ty + TY * i) * LD + e);
#pragma unroll
      for (int k = 0; k < KT; k++) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sk + (tx + TX * k) * LD + e);
#pragma unroll
        for (int i = 0; i < R; i++) acc[i][k] = fma2(q[i].y, y.y, fma2(q[i].x, y.x, acc[i][k]));
      }
    }
    // ---- weights ----
    const int ct = (int)(((long long)x.t + TK - 1) / TK), nt = x.tile - ct;  // nt: tile of the new tokens
    const uint32_t have = have_key[it & (STEPS - 1)];
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int r = wrow + ty + TY * i;
      const long long j = (row0 + r) >> gl;
      unsigned see = ~0u;
      if (nt >= 0) {
        if (!causal) {
          see = j < x.n ? a.mask[(x.c0 + j) * PRHS_TREE_WORDS + nt] : 0u;
        } else {
          const long long past = j - (long long)nt * TK;  // the last key seen
          see = past >= TK - 1 ? ~0u : past < 0 ? 0u : (2u << past) - 1u;
        }
      }
      float s[KT], mx = m[i];
#pragma unroll
      for (int k = 0; k < KT; k++) {
        float lo, hi;
        unf2(acc[i][k], lo, hi);
        const int key = tx + TX * k;
        s[k] = ((see & have) >> key) & 1u ? (lo + hi) * qs : -INFINITY;
        mx = fmaxf(mx, s[k]);
      }
#pragma unroll
      for (int d = TX / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, d));
      const float corr = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mx);
      // (maxima drop NaN: a row of nothing else has -inf, and its weights must be NaN)
      const float ref = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < KT; k++) {
        const float w = exp2f(s[k] - ref);
        sum += w;
        sp[(ty + TY * i) * LP + tx + TX * k] = w;
      }
      l[i] = l[i] * corr + sum;
      m[i] = mx;
      const uint64_t c2 = f2(corr, corr);
#pragma unroll
      for (int c = 0; c < 2 * C4; c++) o[i][c] = mul2(o[i][c], c2);
    }
    __syncwarp();
    // ---- product with V ----
#pragma unroll 4
    for (int key = 0; key < TK; key += 4) {
      float w[R][4];
#pragma unroll
      for (int i = 0; i < R; i++) {
        const float4 y = *reinterpret_cast<const float4*>(sp + (ty + TY * i) * LP + key);
        w[i][0] = y.x;
        w[i][1] = y.y;
        w[i][2] = y.z;
        w[i][3] = y.w;
      }
#pragma unroll
      for (int k = 0; k < 4; k++)
#pragma unroll
        for (int c = 0; c < C4; c++) {
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sv + (key + k) * D + (c * TX + tx) * 4);
#pragma unroll
          for (int i = 0; i < R; i++) {
            const uint64_t w2 = f2(w[i][k], w[i][k]);
            o[i][2 * c] = fma2(w2, y.x, o[i][2 * c]);
            o[i][2 * c + 1] = fma2(w2, y.y, o[i][2 * c + 1]);
          }
        }
    }
    __syncwarp();  // (the weights are rewritten in the next tile)
    if (warp == W - 1 && look < count) found(steps[look & (STEPS - 1)], look & (STEPS - 1), row);

    // ---- the unit's last tile here: its result, or a partial record (m, l and O
    // against m), which also takes the sums of every FOLD tiles on the way: thousands of
    // terms added one by one lose more than blocks of them do (10 tokens over 20K keys,
    // 64 heads: 1.15e-6 of the result against 6.1e-7; runs of hundreds of tiles take 1%
    // longer for it) ----
    const int done = x.tile - x.tile0 + 1;
    const bool last = x.tile + 1 == x.tiles || x.left == 0;
    if (!last && done % FOLD != 0) continue;
    const bool whole = last && x.tile0 == 0 && x.tile + 1 == x.tiles;
    if (x.left == 0 && tid == 0) {  // (then this is the last)
      TreeSplit y = {};
      if (x.tile + 1 < x.tiles) {
        const long long start = g0 + count - 1 - x.tile;  // the list's number of the unit's first tile
        y.rows = rows;
        y.kvh = x.kvh;
        y.tok = (int)(x.c0 + (long long)x.block * x.u);
        y.first = cta - (int)blockIdx.x + (int)(start / per);
        y.part = x.part;
        y.n_rec = (int)((start + x.tiles - 1) / per) - (int)(start / per) + 1;
      }
      p.split[cta] = y;
    }
    const long long rec = (2ll * cta + (x.tile0 == 0 ? 1 : 0)) * p.rows_max;
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int r = wrow + ty + TY * i;
      float sum = l[i];
#pragma unroll
      for (int d = TX / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
      if (r < rows && done > FOLD) {  // what has been folded before
        const float2 f = __ldcg(p.ml + rec + r);
        const float c1 = f.x == -INFINITY ? 0.f : exp2f(f.x - m[i]);
        const uint64_t c2 = f2(c1, c1);
        const float* src = reinterpret_cast<const float*>(p.o) + (rec + r) * D + tx * 4;
        sum = fmaf(f.y, c1, sum);
#pragma unroll
        for (int c = 0; c < C4; c++) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(src + c * TX * 4));
          o[i][2 * c] = fma2(f2(y.x, y.y), c2, o[i][2 * c]);
          o[i][2 * c + 1] = fma2(f2(y.z, y.w), c2, o[i][2 * c + 1]);
        }
      }
      __syncwarp();  // (read by all lanes of the row before one overwrites it)
      if (r >= rows) continue;
      const long long orow = (x.c0 + ((row0 + r) >> gl)) * kv.Hq + (x.kvh << gl) + (r & ((1 << gl) - 1));
      const bool result = whole && (!SHARED || x.part == 0);
      const long long prow = SHARED ? (long long)(x.part - 1) * a.T * kv.Hq + orow : 0;
      const float inv = result ? tree_inv(sum) : 1.f;
      float* dst = (result            ? static_cast<float*>(a.out) + orow * D
                    : SHARED && whole ? a.part_o + prow * D
                                      : reinterpret_cast<float*>(p.o) + (rec + r) * D) + tx * 4;
#pragma unroll
      for (int c = 0; c < C4; c++) {
        float4 y;
        unf2(o[i][2 * c], y.x, y.y);
        unf2(o[i][2 * c + 1], y.z, y.w);
        *reinterpret_cast<float4*>(dst + c * TX * 4) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      }
      if (tx == 0) {
        if (result) a.lse[orow] = tree_lse(m[i], sum);
        else if (SHARED && whole) a.part_ml[prow] = make_float2(m[i], sum);
        else p.ml[rec + r] = make_float2(m[i], sum);
      }
      if (last) continue;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * C4; c++) o[i][c] = 0;
    }
  }
}

// -------------------------------------------------------------------------- //
// host side
// -------------------------------------------------------------------------- //
// The forms, by the most rows a sequence may have (us of the three workloads named
// above: of the form, and of others).
//  8: single tokens and short drafts, bound by the copies: many small CTAs of two
//     warps; lanes of two rows by two keys 64, of one by four 70, one warp 83.
// 32: lanes of four rows by two keys in four warps 64; of one by four in eight 104.
//     At d = 64 four CTAs an SM 64, three 73.
// 64: lanes of four rows by four keys in four warps 237; of two by four in eight
//     311; of eight by two 265.
// CTAs an SM as shared memory and registers allow.
static int tree_rows(const KVView& kv, int max_new) {
  const long long r = (long long)max_new * (kv.Hq / kv.Hkv);
  return r <= 8 ? 8 : r <= 32 ? 32 : 64;
}
static constexpr int tree_ctas_sm(int d, int rows) {
  return d == 128 ? (rows == 8 ? 3 : 2) : (rows == 8 ? 5 : rows == 32 ? 4 : 3);
}
static int tree_ctas(const KVView& kv, int rows, int sms) { return tree_ctas_sm(kv.d, rows) * sms; }
size_t tree_workspace(const KVView& kv, int max_new, bool shared, int sms) {
  // (a call may take fewer rows than max_new names: the form for what its tokens leave;
  // shared keys: with the CTAs of another form for the own keys)
  size_t need = 0;
  for (int rows = tree_rows(kv, max_new); rows >= 8; rows = rows == 64 ? 32 : rows == 32 ? 8 : 0) {
    const size_t n = tree_record_bytes(kv.d, tree_ctas(kv, rows, sms) + (shared ? tree_ctas(kv, 8, sms) : 0), rows);
    need = n > need ? n : need;
  }
  return need;
}

template <int D, int TY, int R, int W, bool SHARED>
static cudaError_t tree_go(const TreeLaunch& a, const TreeRecords& p, int sms, cudaStream_t st, unsigned* ctas) {
  constexpr int CTAS = tree_ctas_sm(D, TY * R * W);
  using S = TreeShape<D, TY, R, W, CTAS>;
  auto k = tree_kernel<D, TY, R, W, CTAS, SHARED>;
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(k, S::SMEM, smem_set);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles that the longest caches would give
  const long long units = (((long long)(SHARED ? a.T : a.max_new) << p.group_log2) + S::TR - 1) / S::TR * a.kv.B * a.kv.Hkv;
  const long long tiles = (SHARED ? 2 : 1) * units * ((a.kv.t_max + TK - 1ll) / TK + (a.max_new + TK - 1ll) / TK);
  *ctas = (unsigned)(tiles < CTAS * sms ? tiles : CTAS * sms);
  const bool own = SHARED && a.items == TREE_OWN;
  e = launch_pdl(k, dim3(*ctas + own), dim3(S::THREADS), S::SMEM, st, own || a.kv.pdl, a, p);
  if (e == cudaSuccess) abi_count_launch();
  return e;
}

template <bool SHARED>
static cudaError_t tree_form(const TreeLaunch& a, const TreeRecords& p, int rows, int sms, cudaStream_t st, unsigned* ctas) {
  const bool wide = a.kv.d == 128;
  if (rows == 8)
    return wide ? tree_go<128, 2, 2, 2, SHARED>(a, p, sms, st, ctas) : tree_go<64, 2, 2, 2, SHARED>(a, p, sms, st, ctas);
  if (rows == 32)
    return wide ? tree_go<128, 2, 4, 4, SHARED>(a, p, sms, st, ctas) : tree_go<64, 2, 4, 4, SHARED>(a, p, sms, st, ctas);
  return wide ? tree_go<128, 4, 4, 4, SHARED>(a, p, sms, st, ctas) : tree_go<64, 4, 4, 4, SHARED>(a, p, sms, st, ctas);
}

cudaError_t launch_tree(const TreeLaunch& launch, int sms, void* ws, cudaStream_t st) {
  TreeLaunch a = launch;
  const KVView& kv = a.kv;
  const bool shared = a.shared != nullptr;
  const int G = kv.Hq / kv.Hkv, own = tree_rows(kv, a.max_new);
  // Groups may have many rows where their sequences have few: each in the form for its rows, in
  // launches that run beside one another. (128 sequences of one token, 4 rows a KV head, in
  // 8 groups of 3.7 to 5K keys: 733 us with the form of the few for all, 596 with the groups',
  // 415; 32 questions on one prefix of 131072 keys 3.7, 1.8, 1.8 ms.) The second launch takes
  // 6 to 25 us, so groups that are small whatever they share have the form of the few (14
  // sequences, 8 rows a KV head, 2K keys: 45 us and 70; 16 samples of 4096 keys 92 and 107).
  const long long most = (long long)a.T * G;  // rows of a group
  const int rows = shared && most > 64 && most * kv.Hkv * kv.t_max > 1 << 20 ? tree_rows(kv, a.T) : own;
  const int all = tree_ctas(kv, rows, sms) + (own != rows ? tree_ctas(kv, own, sms) : 0);
  TreeRecords p = tree_records(ws, G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3, all, rows);
  unsigned ctas = 0, more = 0;
  a.items = own == rows ? TREE_BOTH : TREE_GROUPS;
  cudaError_t e = shared ? tree_form<true>(a, p, rows, sms, st, &ctas) : tree_form<false>(a, p, rows, sms, st, &ctas);
  if (e == cudaSuccess && own != rows) {
    a.items = TREE_OWN;
    p.cta0 = ctas;
    e = tree_form<true>(a, p, own, sms, st, &more);
    ctas += more;
  }
  if (e != cudaSuccess) return e;
  return kv.d == 128 ? launch_tree_join<float, 128, true>(a, p, ctas, st) : launch_tree_join<float, 64, true>(a, p, ctas, st);
}

}  // namespace prhs
