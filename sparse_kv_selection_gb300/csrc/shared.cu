// The last launch of the attention that reads shared prefixes once. A token of a
// group has two states, one against the shared keys (one pass over them gave it for
// all the group's tokens) and one against its sequence's other keys:
//
//   m = max(m1, m2),  o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2)
//
// On bf16 caches this launch also computes the second state of sequences with few
// query rows on few keys (few_item): single tokens, drafts, short prompts. A unit of
// the tcgen05 kernel begins and ends in 3 to 4 us, whatever it holds, and a CTA has
// one at a time; here units of 8 or 16 rows are CTAs of four warps, several an SM.
//
// Inside: a warp takes 16 keys at a time. They are the 16 rows of mma.sync, query rows
// its 8 columns, so that a warp reads every key once and 8 rows cost 8 columns:
//   S^T = K Q^T,  P^T = exp2(S^T - m) in bf16 (transposed by movmatrix),  O^T += V^T P^T
// Every warp has its own ring in shared memory, which its first lane fills by TMA
// (128-byte swizzle), so that warps wait for nobody but their copies. (Loads by all
// lanes straight into the registers of the products: 540 MB of own keys 120 us, four
// times the instructions; with asynchronous 16-byte copies 173.) The warps' states meet in shared memory; a unit of many keys is shared by up
// to FEW_SPLIT CTAs, the last of which to arrive (a ticket) joins their states.
//
// Bound: HBM (the keys, once), and latency: lengths, page numbers, keys, states are
// four dependent reads. All but the last run before the launches it waits for end.
#include "tree_join.cuh"

namespace prhs {

// -------------------------------------------------------------------------- //
// fp32: two states of every token
// -------------------------------------------------------------------------- //
constexpr int SJ_THREADS = 256, SJ_PER = 4;

template <int D>
__global__ void __launch_bounds__(SJ_THREADS) shared_join_kernel(const __grid_constant__ TreeLaunch a) {
  constexpr int C4 = D / 4;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  const TreeItem x = tree_item<true>(a, 2 * b + 1);
  if (x.part != 2 || *a.part_ok == 0) return;
  const long long total = (long long)x.n * a.kv.Hq * C4, row0 = (long long)x.c0 * a.kv.Hq, other = (long long)a.T * a.kv.Hq;
  for (long long i0 = (long long)blockIdx.y * SJ_THREADS * SJ_PER + threadIdx.x; i0 < total;
       i0 += (long long)gridDim.y * SJ_THREADS * SJ_PER) {
    float2 ml[SJ_PER][2];
    float4 o[SJ_PER][2];
#pragma unroll
    for (int k = 0; k < SJ_PER; k++) {
      const long long i = min(i0 + k * SJ_THREADS, total - 1), row = row0 + i / C4;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        ml[k][h] = __ldcg(a.part_ml + row + h * other);
        o[k][h] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (row + h * other) * C4 + i % C4);
      }
    }
#pragma unroll
    for (int k = 0; k < SJ_PER; k++) {
      const long long i = i0 + k * SJ_THREADS, row = row0 + i / C4;
      if (i >= total) break;
      const float M = fmaxf(ml[k][0].x, ml[k][1].x);
      const float w0 = tree_weight(ml[k][0].x, M), w1 = tree_weight(ml[k][1].x, M);
      // (a state that holds NaN has it in its sum, whatever its maximum)
      const float L = fmaf(w1, ml[k][1].y, w0 * ml[k][0].y), inv = tree_inv(L);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      tree_fma(y, w0, o[k][0]);
      tree_fma(y, w1, o[k][1]);
      tree_put(static_cast<float*>(a.out) + row * D + i % C4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (i % C4 == 0) a.lse[row] = tree_lse(M, L);
    }
  }
}

// -------------------------------------------------------------------------- //
// bf16: few rows on few keys, and the join
// -------------------------------------------------------------------------- //
constexpr int FEW_WARPS = 8, FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_STEP = 16;        // keys of a warp's step: a box, never over a page's end
constexpr int FEW_RING = 24 << 10;  // bytes of a warp's ring: 3 steps at d = 128, 6 at 64
constexpr float FEW_LOG2E = 1.4426950408889634f;
constexpr float FEW_RESCALE = 8.f;  // growth of a maximum (base 2) that rescales, as in the tcgen05 kernel

// D += A B, 16 x 8 x 16, bf16.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t few_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float few_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four 8 x 8 matrices of 16-bit elements, a row's address a lane; as they are or transposed.
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The warp tasks of one sequence, KV head by KV head: units of RB query rows, each
// cut into `cuts` equal runs of its steps; or, where the other launch attended its
// keys, joins of 32 rows.
struct FewSeq {
  TreeItem x;
  int blocks, steps, tasks, cuts;  // units of a KV head, steps of the longest, tasks
  bool few;
};
template <int RB>
__device__ __forceinline__ int few_steps(const TreeLaunch& a, const TreeItem& x, int gl, int blk, int* fresh) {
  const int end = min(x.n << gl, (blk + 1) * RB);  // (causal: new tokens up to the unit's last one)
  *fresh = a.mask == nullptr ? ((end - 1) >> gl) + 1 : x.n;
  return (x.t + FEW_STEP - 1) / FEW_STEP + (*fresh + FEW_STEP - 1) / FEW_STEP;
}
template <int RB>
__device__ __forceinline__ FewSeq few_seq(const TreeLaunch& a, int b, int gl) {
  FewSeq s;
  s.x = tree_item<true>(a, 2 * b + 1, true);
  s.few = few_item(a, s.x.n, s.x.t);
  s.blocks = s.steps = s.tasks = 0;
  s.cuts = 1;
  if (s.few) {
    s.blocks = ((s.x.n << gl) + RB - 1) / RB;
    int fresh;
    if (s.blocks > 0) s.steps = few_steps<RB>(a, s.x, gl, s.blocks - 1, &fresh);
  } else if (s.x.part == 2) {
    s.blocks = ((s.x.n << gl) + 31) / 32;
  }
  return s;
}
// With runs of about `run` steps.
__device__ __forceinline__ void few_cut(FewSeq& s, int Hkv, int run) {
  if (s.few) s.cuts = max(1, (2 * s.steps + run) / (2 * run));
  s.tasks = Hkv * s.blocks * s.cuts;
}

template <int D, int NT>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ CUtensorMap knmap, const __grid_constant__ CUtensorMap vnmap,
               const __grid_constant__ TreeLaunch a) {
  // a step's K, then its V: SEGS column segments of 16 rows of 128 bytes
  constexpr int RB = 8 * NT, C4 = D / 4, SEGS = D / 64, SEG = FEW_STEP * 128, STAGE = 2 * SEGS * SEG, STAGES = FEW_RING / STAGE;
  static_assert(RB * D * 4 <= FEW_RING, "a warp's state takes its ring's place");
  extern __shared__ __align__(1024) uint8_t few_smem[];
  __shared__ uint64_t full[FEW_WARPS][STAGES];
  __shared__ int wsum[3][FEW_WARPS];
  __shared__ int tasks_to[FEW_THREADS], cut_to[FEW_THREADS];  // up to a thread's sequences: tasks, and those of cut units
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, gl = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int gw = blockIdx.x * FEW_WARPS + warp, gws = gridDim.x * FEW_WARPS;
  if (warp == 0 && lane < 4) prefetch_tmap(lane == 0 ? &kmap : lane == 1 ? &vmap : lane == 2 ? &knmap : &vnmap);
  if (lane == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(&full[warp][i], 1);
    fence_barrier_init();
  }

  // ---- the list of tasks: prefixes over the sequences, a run of them a thread ----
  const int per = (kv.B + FEW_THREADS - 1) / FEW_THREADS, b0 = min(kv.B, tid * per), b1 = min(kv.B, b0 + per);
  auto block_sum = [&](int v, int slot) {  // (inclusive prefix and sum over the block)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL_MASK, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) wsum[slot][warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < FEW_WARPS; w++) {
      const int y = wsum[slot][w];
      if (w < warp) before += y;
      all += y;
    }
    return make_int2(before + v, all);
  };
  FewSeq mine = {};
  int steps = 0;
  for (int b = b0; b < b1; b++) {
    mine = few_seq<RB>(a, b, gl);
    steps += kv.Hkv * mine.blocks * mine.steps;
  }
  steps = block_sum(steps, 0).y;
  // Runs of a third of a warp's share (so that warps end together), of 8 to 16 steps
  // where there are few. The cut units' tasks then number four a warp at most.
  const int run = max((steps + 3 * gws - 1) / (3 * gws), min(16, max(8, steps / gws)));
  int tasks = 0, cut = 0;
  for (int b = b0; b < b1; b++) {
    if (per > 1) mine = few_seq<RB>(a, b, gl);
    few_cut(mine, kv.Hkv, run);
    tasks += mine.tasks;
    cut += mine.cuts > 1 ? mine.tasks : 0;
  }
  const int2 t2 = block_sum(tasks, 1), c2 = block_sum(cut, 2);
  tasks_to[tid] = t2.x;
  cut_to[tid] = c2.x;
  __syncthreads();
  if ((smem_addr(few_smem) & 1023) != 0) {  // the swizzle needs it
    raise_error(kv.err, PRHS_DEV_CAPACITY);
    return;
  }

  const bool causal = a.mask == nullptr;
  const uint32_t ring = smem_addr(few_smem) + warp * FEW_RING;
  float4* staged = reinterpret_cast<float4*>(few_smem + warp * FEW_RING);  // [C4][RB]
  const float sc = a.scale * FEW_LOG2E;
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;
  for (int task = gw; task < t2.y && !dead; task += gws) {
    // ---- what it is ----
    int lo = 0, hi = FEW_THREADS - 1;  // the first thread whose sequences end behind it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tasks_to[mid] > task) hi = mid; else lo = mid + 1;
    }
    int off = task - (lo > 0 ? tasks_to[lo - 1] : 0), slot = lo > 0 ? cut_to[lo - 1] : 0, b = lo * per;
    FewSeq s = few_seq<RB>(a, b, gl);
    few_cut(s, kv.Hkv, run);
    while (off >= s.tasks) {
      off -= s.tasks;
      slot += s.cuts > 1 ? s.tasks : 0;
      s = few_seq<RB>(a, ++b, gl);
      few_cut(s, kv.Hkv, run);
    }
    const TreeItem x = s.x;
    slot += off;
    const int part_of = off % s.cuts, blk = off / s.cuts % s.blocks, kvh = off / s.cuts / s.blocks;
    if (!s.few) {  // only a join
      pdl_wait();
      if (*a.part_ok == 0) continue;
      const int r = blk * 32 + lane, tok = x.c0 + (r >> gl), h = r & (G - 1);
      if (r >= x.n << gl) continue;
      float2 ml[2];
#pragma unroll
      for (int k = 0; k < 2; k++) ml[k] = __ldcg(a.part_ml + part_row<__nv_bfloat16>(a, k + 1, tok, kvh, h, gl));
      const float M = fmaxf(ml[0].x, ml[1].x), w0 = tree_weight(ml[0].x, M), w1 = tree_weight(ml[1].x, M);
      const float L = fmaf(w1, ml[1].y, w0 * ml[0].y), inv = tree_inv(L);
      const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
#pragma unroll 4
      for (int c4 = 0; c4 < C4; c4++) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        tree_fma(y, w0, __ldcg(part_at<__nv_bfloat16, D>(a, 1, tok, kvh, h, c4, gl)));
        tree_fma(y, w1, __ldcg(part_at<__nv_bfloat16, D>(a, 2, tok, kvh, h, c4, gl)));
        tree_put(static_cast<__nv_bfloat16*>(a.out) + orow * D + c4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      }
      a.lse[orow] = tree_lse(M, L);
      continue;
    }
    int fresh;
    const int all_steps = few_steps<RB>(a, x, gl, blk, &fresh), cached = (x.t + FEW_STEP - 1) / FEW_STEP;
    const int s0 = all_steps * part_of / s.cuts, s1 = all_steps * (part_of + 1) / s.cuts;
    const int rows = min(RB, (x.n << gl) - blk * RB), tok0 = (blk * RB) >> gl;
  // Q as the products take it: rows g of each eight, columns 16 j + 2 c and 16 j + 8 + 2 c
  uint32_t q[NT][D / 16][2];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int r = blk * RB + 8 * t + g;
    const bool have = 8 * t + g < rows;
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) +
                               ((long long)(x.c0 + (have ? r >> gl : tok0)) * kv.Hq + (kvh << gl) + (have ? r & (G - 1) : 0)) * D;
#pragma unroll
    for (int j = 0; j < D / 16; j++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        q[t][j][h] = have ? *reinterpret_cast<const uint32_t*>(row + 16 * j + 8 * h + 2 * c) : 0u;
  }

  // Rows of the steps' first keys, 32 steps at a time, one a lane (-1: on no page).
  auto row_at = [&](int s) -> int {
    if (s >= min(s1, cached)) return 0;
    const int key = x.base + s * FEW_STEP;
    if (kv.block_table == nullptr) return (b * kv.Hkv + kvh) * kv.t_max + key;
    const int page = kv.block_table[(long long)b * kv.max_blocks + key / kv.block_size];
    if ((unsigned)page >= (unsigned)kv.num_blocks) {
      raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
      return -1;
    }
    return (page * kv.Hkv + kvh) * kv.block_size + key % kv.block_size;
  };
  int window = s0, at = row_at(window + lane);
  int counts = 0;  // keys of the ring's steps, five bits each
  auto load = [&](int s, int stage) {
    if (s >= window + 32) {
      window += 32;
      at = row_at(window + lane);
    }
    const int row = __shfl_sync(FULL_MASK, at, s - window), j = (s - cached) * FEW_STEP;
    const bool is_new = s >= cached;
    const int n = is_new ? min(FEW_STEP, fresh - j) : row < 0 ? 0 : min(FEW_STEP, x.t - s * FEW_STEP);
    counts = (counts & ~(31 << 5 * stage)) | n << 5 * stage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp][stage], STAGE);
      const CUtensorMap *km = is_new ? &knmap : &kmap, *vm = is_new ? &vnmap : &vmap;
      const int z = is_new ? kvh : max(row, 0), w = is_new ? x.c0 + j : 0;
#pragma unroll
      for (int i = 0; i < SEGS; i++) tma_load_4d(ring + stage * STAGE + i * SEG, km, 0, i, z, w, &full[warp][stage]);
#pragma unroll
      for (int i = 0; i < SEGS; i++) tma_load_4d(ring + stage * STAGE + (SEGS + i) * SEG, vm, 0, i, z, w, &full[warp][stage]);
    }
    __syncwarp();
  };

  float m[NT][2], l[NT][2], o[NT][D / 16][4];  // rows 8 t + 2 c, + 1; O's columns 16 e + g, + 8
#pragma unroll
  for (int t = 0; t < NT; t++) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; e++) o[t][e][0] = o[t][e][1] = o[t][e][2] = o[t][e][3] = 0.f;
  }
  for (int i = 0, to = stage; i < min(STAGES, s1 - s0); i++) {
    load(s0 + i, to);
    if (++to == STAGES) to = 0;
  }
  // a lane's row of the four matrices of a product's operand: K's rows lane % 16, columns 8 (lane / 16) ..;
  // V's the other way about (its matrices come in the order of d, then keys)
  const int krow = lane & 15, kcol = lane >> 4, vrow = (lane & 7) + (lane >> 4) * 8, vcol = lane >> 3 & 1;
  const uint32_t k_at = ring + krow * 128, v_at = ring + SEGS * SEG + vrow * 128;
  for (int s = s0; s < s1; s++) {
    dead = !__all_sync(FULL_MASK, mbar_wait(&full[warp][stage], phase, kv.err));
    if (dead) break;
    const int n = counts >> 5 * stage & 31;
    float p[NT][4];  // keys g: rows 2 c, 2 c + 1; keys g + 8
#pragma unroll
    for (int t = 0; t < NT; t++) p[t][0] = p[t][1] = p[t][2] = p[t][3] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
      uint32_t k[4];
      ldm4(k, k_at + stage * STAGE + j / 4 * SEG + (((j % 4 * 2 + kcol) ^ (krow & 7)) << 4));
#pragma unroll
      for (int t = 0; t < NT; t++) mma16(p[t], k[0], k[1], k[2], k[3], q[t][j][0], q[t][j][1]);
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int key0 = (s - cached) * FEW_STEP;  // (new tokens)
#pragma unroll
      for (int i = 0; i < 4; i++) p[t][i] *= sc;
      if (s >= cached || n < FEW_STEP) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int key = g + 8 * (i >> 1);
          bool see = key < n;
          if (s >= cached && see) {
            const int tok = min((blk * RB + 8 * t + 2 * c + (i & 1)) >> gl, x.n - 1);
            see = causal ? key0 + key <= tok
                         : (a.mask[(long long)(x.c0 + tok) * PRHS_TREE_WORDS + ((key0 + key) >> 5)] >> ((key0 + key) & 31)) & 1u;
          }
          if (!see) p[t][i] = -INFINITY;
        }
      }
      float mx[2] = {fmaxf(p[t][0], p[t][2]), fmaxf(p[t][1], p[t][3])};
      auto grows = [&](int r) { return mx[r] > m[t][r] + FEW_RESCALE || (m[t][r] == -INFINITY && mx[r] > -INFINITY); };
      if (__any_sync(FULL_MASK, grows(0) || grows(1))) {
#pragma unroll
        for (int r = 0; r < 2; r++) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(FULL_MASK, mx[r], d));
          const bool grow = grows(r);
          const float corr = grow ? few_ex2(m[t][r] - mx[r]) : 1.f;
          if (grow) m[t][r] = mx[r];
          l[t][r] *= corr;
#pragma unroll
          for (int e = 0; e < D / 16; e++) {
            o[t][e][r] *= corr;
            o[t][e][2 + r] *= corr;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float ref = m[t][i & 1] == -INFINITY ? 0.f : m[t][i & 1];
        p[t][i] = few_ex2(p[t][i] - ref);
        l[t][i & 1] += p[t][i];
      }
      pb[t][0] = transpose8(few_pack(p[t][0], p[t][1]));
      pb[t][1] = transpose8(few_pack(p[t][2], p[t][3]));
    }
    // rows of V that do not exist hold whatever was there, and 0 * inf is not 0
    const uint32_t keep0 = (2 * c < n ? 0xffffu : 0u) | (2 * c + 1 < n ? 0xffff0000u : 0u);
    const uint32_t keep1 = (2 * c + 8 < n ? 0xffffu : 0u) | (2 * c + 9 < n ? 0xffff0000u : 0u);
#pragma unroll
    for (int e = 0; e < D / 16; e++) {
      uint32_t v[4];  // columns 16 e + g, + 8: keys 2 c, + 1; then keys + 8
      ldm4_trans(v, v_at + stage * STAGE + e / 4 * SEG + (((e % 4 * 2 + vcol) ^ (vrow & 7)) << 4));
      if (n < FEW_STEP) {
        v[0] &= keep0;
        v[1] &= keep0;
        v[2] &= keep1;
        v[3] &= keep1;
      }
#pragma unroll
      for (int t = 0; t < NT; t++) mma16(o[t][e], v[0], v[1], v[2], v[3], pb[t][0], pb[t][1]);
    }
    __syncwarp();  // (the stage has been read)
    if (s + STAGES < s1) load(s + STAGES, stage);
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (dead) break;

  // ---- its state: columns by rows in the ring's place, then four columns a lane ----
  __syncwarp();
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int r = 0; r < 2; r++) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[t][r] += __shfl_xor_sync(FULL_MASK, l[t][r], d);
      const int row = 8 * t + 2 * c + r;
#pragma unroll
      for (int e = 0; e < D / 16; e++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          reinterpret_cast<float*>(staged + (4 * e + 2 * h + g / 4) * RB + row)[g % 4] = o[t][e][2 * h + r];
    }
  __syncwarp();
  // lane: row lane % 8 of each eight, columns 4 (lane / 8 + 4 k) ..
  const int sr = lane & 7, sq = lane >> 3;
  float2 ml[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {  // (row 8 t + 2 c + r is in lanes c of any g)
    const float m0 = __shfl_sync(FULL_MASK, m[t][0], sr >> 1), m1 = __shfl_sync(FULL_MASK, m[t][1], sr >> 1);
    const float l0 = __shfl_sync(FULL_MASK, l[t][0], sr >> 1), l1 = __shfl_sync(FULL_MASK, l[t][1], sr >> 1);
    ml[t] = sr & 1 ? make_float2(m1, l1) : make_float2(m0, l0);
  }
  float4 y[NT][C4 / 4];
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int k = 0; k < C4 / 4; k++) y[t][k] = staged[(sq + 4 * k) * RB + 8 * t + sr];
  __syncwarp();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the ring's next copies come behind these reads)

  pdl_wait();  // (the tickets are set, the states against the shared keys written by the launches in front)
  if (*a.part_ok == 0) continue;
  if (s.cuts > 1) {  // the last of a unit's tasks to arrive joins their states, in their order
    float4* states = static_cast<float4*>(a.few_states);  // [tasks][C4][RB], then (maximum, sum) [tasks][RB]
    float2* sums = reinterpret_cast<float2*>(states + (long long)a.few_most * C4 * RB);
    const int slot0 = slot - part_of;
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int k = 0; k < C4 / 4; k++) __stcg(states + ((long long)slot * C4 + sq + 4 * k) * RB + 8 * t + sr, y[t][k]);
      if (sq == 0) __stcg(sums + (long long)slot * RB + 8 * t + sr, ml[t]);
    }
    __threadfence();
    __syncwarp();
    int arrived = 0;
    if (lane == 0) arrived = atomicAdd(a.few_ticket + slot0, 1);
    if (__shfl_sync(FULL_MASK, arrived, 0) != s.cuts - 1) continue;
    __threadfence();
#pragma unroll
    for (int t = 0; t < NT; t++) {
      float M = -INFINITY, L = 0.f;
      for (int w = 0; w < s.cuts; w++) M = fmaxf(M, __ldcg(sums + (long long)(slot0 + w) * RB + 8 * t + sr).x);
#pragma unroll
      for (int k = 0; k < C4 / 4; k++) y[t][k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int w = 0; w < s.cuts; w++) {
        const float2 z = __ldcg(sums + (long long)(slot0 + w) * RB + 8 * t + sr);
        const float wt = tree_weight(z.x, M);
        L = fmaf(wt, z.y, L);
#pragma unroll
        for (int k = 0; k < C4 / 4; k++)
          tree_fma(y[t][k], wt, __ldcg(states + ((long long)(slot0 + w) * C4 + sq + 4 * k) * RB + 8 * t + sr));
      }
      ml[t] = make_float2(M, L);
    }
  }

  // ---- the result, with the state against the shared keys ----
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int r = blk * RB + 8 * t + sr, tok = x.c0 + (r >> gl), h = r & (G - 1);
    if (8 * t + sr >= rows) continue;
    float M = ml[t].x, L = ml[t].y, w1 = 1.f, w0 = 0.f;
    if (x.part == 2) {
      const float2 z = __ldcg(a.part_ml + part_row<__nv_bfloat16>(a, 1, tok, kvh, h, gl));
      M = fmaxf(M, z.x);
      w1 = tree_weight(ml[t].x, M);
      w0 = tree_weight(z.x, M);
      L = fmaf(w0, z.y, w1 * L);
    }
    const float inv = tree_inv(L);
    const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
#pragma unroll
    for (int k = 0; k < C4 / 4; k++) {
      float4 v = make_float4(y[t][k].x * w1, y[t][k].y * w1, y[t][k].z * w1, y[t][k].w * w1);
      if (x.part == 2) tree_fma(v, w0, __ldcg(part_at<__nv_bfloat16, D>(a, 1, tok, kvh, h, sq + 4 * k, gl)));
      tree_put(static_cast<__nv_bfloat16*>(a.out) + orow * D + (sq + 4 * k) * 4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    }
    if (sq == 0) a.lse[orow] = tree_lse(M, L);
  }
  }
  if (dead)  // nothing may still be in flight when the CTA ends
    for (int i = 0; i < STAGES; i++) mbar_wait(&full[warp][i], phase ^ (i < stage), kv.err);
  pdl_wait();  // (whatever it had to do: this launch does not end before those in front of it)
  pdl_trigger();
}

// -------------------------------------------------------------------------- //
// host side
// -------------------------------------------------------------------------- //
// Cut units have at most 4/3 as many tasks as runs of the steps' share, three a warp.
static long long few_most(const KVView& kv, int max_new, int sms) {
  const long long G = kv.Hq / kv.Hkv, rows = max_new * G, blocks = (rows + 15) / 16;
  const long long cuts = (FEW_KEYS / FEW_STEP + 3) / 8 + 1;  // (of runs of 8 steps)
  const long long unit_tasks = (long long)kv.B * kv.Hkv * (blocks < FEW_BLOCKS ? blocks : FEW_BLOCKS) * cuts;
  const long long most = 4ll * FEW_WARPS * sms;
  return unit_tasks < most ? unit_tasks : most;
}
void few_shape(TreeLaunch* a, int sms) {
  if (a->kv.dtype != PRHS_BF16) return;
  a->few_rows = (long long)a->max_new * (a->kv.Hq / a->kv.Hkv) <= 8 ? 8 : 16;
  a->few_most = (int)few_most(a->kv, a->max_new, sms);
}
size_t few_state_bytes(const KVView& kv, int max_new, int sms) {
  if (kv.dtype != PRHS_BF16) return 0;
  const size_t rows = (long long)max_new * (kv.Hq / kv.Hkv) <= 8 ? 8 : 16;
  return few_most(kv, max_new, sms) * rows * (kv.d * sizeof(float) + sizeof(float2));
}
size_t few_ticket_bytes(const KVView& kv, int max_new, int sms) {
  return kv.dtype != PRHS_BF16 ? 0 : few_most(kv, max_new, sms) * sizeof(int);
}

template <int D, int NT>
static cudaError_t few_go(const TreeLaunch& a, const CUtensorMap* maps, int sms, cudaStream_t st) {
  auto k = few_kernel<D, NT>;
  static int smem_set[SMEM_DEVICES];
  const cudaError_t e = allow_smem(k, FEW_WARPS * FEW_RING, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(sms), dim3(FEW_THREADS), FEW_WARPS * FEW_RING, st, true, maps[0],
                    maps[1], maps[2], maps[3], a);
}
cudaError_t launch_few(const TreeLaunch& a, const CUtensorMap* maps, int sms, cudaStream_t st) {
  if (a.few_rows == 8) return a.kv.d == 128 ? few_go<128, 1>(a, maps, sms, st) : few_go<64, 1>(a, maps, sms, st);
  return a.kv.d == 128 ? few_go<128, 2>(a, maps, sms, st) : few_go<64, 2>(a, maps, sms, st);
}

cudaError_t launch_shared_join(const TreeLaunch& a, cudaStream_t st) {
  const long long pass = (long long)SJ_THREADS * SJ_PER, y = ((long long)a.max_new * a.kv.Hq * a.kv.d / 4 + pass - 1) / pass;
  const dim3 grid(a.kv.B, (unsigned)(y < 64 ? y : 64));
  if (a.kv.d == 128) return launch_pdl(shared_join_kernel<128>, grid, dim3(SJ_THREADS), 0, st, true, a);
  return launch_pdl(shared_join_kernel<64>, grid, dim3(SJ_THREADS), 0, st, true, a);
}

}  // namespace prhs
