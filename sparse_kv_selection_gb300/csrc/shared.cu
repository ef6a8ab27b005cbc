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
// Inside: a warp takes 16 keys at a time, straight from the cache into the registers
// of mma.sync (keys are its 16 rows, query rows its 8 columns, so that a warp holds
// every key once and 8 rows cost 8 columns):
//   S^T = K Q^T,  P^T = exp2(S^T - m) in bf16 (transposed by movmatrix),  O^T += V^T P^T
// The order of d within a product is free, so a lane's 16-byte piece of a K row feeds
// two instructions as it is, and O's columns are permuted so that V's pieces do too
// (two rows interleaved). The next 16 keys are asked for as soon as the registers are
// free. The warps' states meet in shared memory; a unit of many keys is shared by up
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
constexpr int FEW_WARPS = 4, FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_STEP = 16;       // keys of a warp's step
constexpr int FEW_SPLIT = 4;       // CTAs of a unit at most
constexpr int FEW_STATES = 8192;   // CTAs of a launch with more than one a unit
constexpr int FEW_STEPS_MIN = 32;  // steps of a CTA before the next one takes a share
constexpr int FEW_BLOCKS = 16;     // CTAs of rows a KV head at most
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
__device__ __forceinline__ uint32_t reg_of(const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// A state of every row of the unit: of a warp, of a CTA.
template <int D, int NT>
struct FewState {
  float o[8 * NT][D];
  float2 ml[8 * NT];
};

template <int D, int NT>
__global__ void __launch_bounds__(FEW_THREADS, NT == 1 ? (D == 64 ? 4 : 3) : 2) few_kernel(const __grid_constant__ TreeLaunch a) {
  using State = FewState<D, NT>;
  constexpr int RB = 8 * NT, C4 = D / 4, KJ = D / 32, VI = D / 64;
  extern __shared__ __align__(16) uint8_t few_smem[];
  State* states = reinterpret_cast<State*>(few_smem);  // the warps'
  __shared__ int arrived;
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, gl = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int unit = blockIdx.x / a.few_split, rank = blockIdx.x % a.few_split;
  const int blk = unit % a.few_blocks, kvh = unit / a.few_blocks % kv.Hkv, b = unit / a.few_blocks / kv.Hkv;
  // (one CTA waits whatever it has to do, so that this launch does not end before those in front of it)
  if (blockIdx.x == 0) pdl_wait();
  const TreeItem x = tree_item<true>(a, 2 * b + 1, true);
  const int rows = min(RB, (x.n << gl) - blk * RB);  // of this unit
  const bool few = few_item(a, x.n, x.t);
  if (!few) {  // the other launch attended its keys: only the join, rows in turn
    if (x.part != 2) return;
    pdl_wait();
    if (*a.part_ok == 0) return;
    const int total = (x.n << gl) * C4, all = a.few_blocks * a.few_split * FEW_THREADS;
    for (int i = (blk * a.few_split + rank) * FEW_THREADS + tid; i < total; i += all) {
      const int row = i / C4, c4 = i % C4, tok = x.c0 + (row >> gl), h = row & (G - 1);
      float2 ml[2];
      float4 o[2];
#pragma unroll
      for (int k = 0; k < 2; k++) {
        ml[k] = __ldcg(a.part_ml + part_row<__nv_bfloat16>(a, k + 1, tok, kvh, h, gl));
        o[k] = __ldcg(part_at<__nv_bfloat16, D>(a, k + 1, tok, kvh, h, c4, gl));
      }
      const float M = fmaxf(ml[0].x, ml[1].x), w0 = tree_weight(ml[0].x, M), w1 = tree_weight(ml[1].x, M);
      const float L = fmaf(w1, ml[1].y, w0 * ml[0].y), inv = tree_inv(L);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      tree_fma(y, w0, o[0]);
      tree_fma(y, w1, o[1]);
      const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
      tree_put(static_cast<__nv_bfloat16*>(a.out) + orow * D + c4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      if (c4 == 0) a.lse[orow] = tree_lse(M, L);
    }
    return;
  }
  if (rows <= 0) return;

  // ---- this CTA's steps: the cache's, then the new tokens' ----
  const bool causal = a.mask == nullptr;
  const int tok0 = (blk * RB) >> gl;                                       // the unit's first token
  const int fresh = causal ? min(x.n, ((blk * RB + rows - 1) >> gl) + 1) : x.n;  // new tokens that its rows may see
  const int cached = (x.t + FEW_STEP - 1) / FEW_STEP, steps = cached + (fresh + FEW_STEP - 1) / FEW_STEP;
  const int split = min(a.few_split, (steps + FEW_STEPS_MIN - 1) / FEW_STEPS_MIN);
  if (rank >= split) return;
  const int s0 = steps * rank / split, s1 = steps * (rank + 1) / split;

  // Q rows as the products take them: row g of each eight, columns 32 j + 8 c ..
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q);
  uint4 q[NT][KJ];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int r = blk * RB + 8 * t + g;
    const bool have = 8 * t + g < rows;
    const __nv_bfloat16* row = qp + ((long long)(x.c0 + (have ? r >> gl : tok0)) * kv.Hq + (kvh << gl) + (have ? r & (G - 1) : 0)) * D;
#pragma unroll
    for (int j = 0; j < KJ; j++) q[t][j] = have ? *reinterpret_cast<const uint4*>(row + 32 * j + 8 * c) : make_uint4(0, 0, 0, 0);
  }

  // Rows of the steps' first keys, 32 steps of the warp at a time, one a lane.
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
  struct Step {  // where a step's keys are, and how many there are
    const __nv_bfloat16 *k, *v;
    long long ks, vs;
    int n;
  };
  int window = s0 + warp, at = row_at(window + lane * FEW_WARPS);
  auto step_of = [&](int s) -> Step {
    Step y;
    if (s >= window + 32 * FEW_WARPS) {
      window += 32 * FEW_WARPS;
      at = row_at(window + lane * FEW_WARPS);
    }
    const int row = __shfl_sync(FULL_MASK, at, (s - window) / FEW_WARPS);
    if (s < cached) {
      y.k = static_cast<const __nv_bfloat16*>(kv.k) + (long long)max(row, 0) * D;
      y.v = static_cast<const __nv_bfloat16*>(kv.v) + (long long)max(row, 0) * D;
      y.ks = y.vs = D;
      y.n = row < 0 ? 0 : min(FEW_STEP, x.t - s * FEW_STEP);
    } else {
      const int j = (s - cached) * FEW_STEP;
      y.k = static_cast<const __nv_bfloat16*>(a.k_new) + (long long)(x.c0 + j) * a.ks + kvh * D;
      y.v = static_cast<const __nv_bfloat16*>(a.v_new) + (long long)(x.c0 + j) * a.vs + kvh * D;
      y.ks = a.ks;
      y.vs = a.vs;
      y.n = s < s1 ? min(FEW_STEP, fresh - j) : 0;
    }
    return y;
  };
  uint4 kf[2][KJ], vf[4][VI];
  auto load_k = [&](const Step& y) {
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < KJ; j++)
        kf[i][j] = g + 8 * i < y.n ? ldg_stream(y.k + (g + 8 * i) * y.ks + 32 * j + 8 * c) : make_uint4(0, 0, 0, 0);
  };
  auto load_v = [&](const Step& y) {  // (rows that do not exist as zeros: 0 * inf is not 0)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int key = 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int j = 0; j < VI; j++)
        vf[i][j] = key < y.n ? ldg_stream(y.v + key * y.vs + 64 * j + 8 * g) : make_uint4(0, 0, 0, 0);
    }
  };

  const float sc = a.scale * FEW_LOG2E;
  float m[NT][2], l[NT][2], o[NT][4 * VI][4];  // rows 8 t + 2 c, + 1
#pragma unroll
  for (int t = 0; t < NT; t++) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * VI; e++) o[t][e][0] = o[t][e][1] = o[t][e][2] = o[t][e][3] = 0.f;
  }
  int s = s0 + warp;
  Step now = {};
  if (s < s1) {
    now = step_of(s);
    load_k(now);
    load_v(now);
  }
  for (; s < s1; s += FEW_WARPS) {
    const bool more = s + FEW_WARPS < s1;
    Step next = now;
    float p[NT][4];  // keys g: rows 2 c, 2 c + 1; keys g + 8
#pragma unroll
    for (int t = 0; t < NT; t++) p[t][0] = p[t][1] = p[t][2] = p[t][3] = 0.f;
#pragma unroll
    for (int j = 0; j < KJ; j++)
#pragma unroll
      for (int t = 0; t < NT; t++) {
        mma16(p[t], kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y, q[t][j].x, q[t][j].y);
        mma16(p[t], kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w, q[t][j].z, q[t][j].w);
      }
    if (more) {
      next = step_of(s + FEW_WARPS);
      load_k(next);
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int key0 = (s - cached) * FEW_STEP;  // (new tokens)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int key = g + 8 * (i >> 1);
        bool see = key < now.n;
        if (s >= cached && see) {
          const int tok = min((blk * RB + 8 * t + 2 * c + (i & 1)) >> gl, x.n - 1);
          see = causal ? key0 + key <= tok
                       : (a.mask[(long long)(x.c0 + tok) * PRHS_TREE_WORDS + ((key0 + key) >> 5)] >> ((key0 + key) & 31)) & 1u;
        }
        p[t][i] = see ? p[t][i] * sc : -INFINITY;
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
          for (int e = 0; e < 4 * VI; e++) {
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
#pragma unroll
    for (int j = 0; j < VI; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint32_t r0 = reg_of(vf[0][j], e), r1 = reg_of(vf[1][j], e), r2 = reg_of(vf[2][j], e), r3 = reg_of(vf[3][j], e);
        const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
        const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
        for (int t = 0; t < NT; t++) mma16(o[t][4 * j + e], a0, a1, a2, a3, pb[t][0], pb[t][1]);
      }
    if (more) load_v(next);
    now = next;
  }

  // ---- the warps' states meet ----
  {
    State& y = states[warp];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        float sum = l[t][r];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(FULL_MASK, sum, d);
        const int row = 8 * t + 2 * c + r;
        if (g == 0) y.ml[row] = make_float2(m[t][r], sum);
#pragma unroll
        for (int j = 0; j < VI; j++)
#pragma unroll
          for (int h = 0; h < 2; h++)
            *reinterpret_cast<float4*>(&y.o[row][64 * j + 8 * g + 4 * h]) =
                make_float4(o[t][4 * j + 2 * h][r], o[t][4 * j + 2 * h][2 + r], o[t][4 * j + 2 * h + 1][r], o[t][4 * j + 2 * h + 1][2 + r]);
      }
  }
  __syncthreads();
  constexpr int PER = RB * C4 / FEW_THREADS;
  float M[PER], L[PER];
  float4 O[PER];
#pragma unroll
  for (int k = 0; k < PER; k++) {
    const int i = tid + k * FEW_THREADS, row = i / C4, c4 = i % C4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < FEW_WARPS; w++) mm = fmaxf(mm, states[w].ml[row].x);
    M[k] = mm;
    L[k] = 0.f;
    O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < FEW_WARPS; w++) {
      const float wt = tree_weight(states[w].ml[row].x, mm);
      L[k] = fmaf(wt, states[w].ml[row].y, L[k]);
      tree_fma(O[k], wt, *reinterpret_cast<const float4*>(&states[w].o[row][c4 * 4]));
    }
  }
  pdl_wait();  // (the tickets are set, the states against the shared keys written by the launches in front)
  pdl_trigger();
  if (*a.part_ok == 0) return;
  if (split > 1) {  // the states of a unit's CTAs meet in the last one to arrive
    State* all = reinterpret_cast<State*>(a.few_states) + (long long)unit * a.few_split;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const int i = tid + k * FEW_THREADS, row = i / C4, c4 = i % C4;
      __stcg(reinterpret_cast<float4*>(&all[rank].o[row][c4 * 4]), O[k]);
      if (c4 == 0) __stcg(&all[rank].ml[row], make_float2(M[k], L[k]));
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) arrived = atomicAdd(a.few_ticket + unit, 1);
    __syncthreads();
    if (arrived != split - 1) return;
    __threadfence();
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const int i = tid + k * FEW_THREADS, row = i / C4, c4 = i % C4;
      // in the CTAs' order, whichever came last
      float2 ml[FEW_SPLIT];
      float4 y[FEW_SPLIT];
#pragma unroll
      for (int w = 0; w < FEW_SPLIT; w++) {
        const State& from = all[min(w, split - 1)];
        ml[w] = __ldcg(&from.ml[row]);
        y[w] = __ldcg(reinterpret_cast<const float4*>(&from.o[row][c4 * 4]));
      }
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < FEW_SPLIT; w++)
        if (w < split) mm = fmaxf(mm, ml[w].x);
      M[k] = mm;
      L[k] = 0.f;
      O[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < FEW_SPLIT; w++) {
        if (w >= split) continue;
        const float wt = tree_weight(ml[w].x, mm);
        L[k] = fmaf(wt, ml[w].y, L[k]);
        tree_fma(O[k], wt, y[w]);
      }
    }
  }

  // ---- the result, with the state against the shared keys ----
#pragma unroll
  for (int k = 0; k < PER; k++) {
    const int i = tid + k * FEW_THREADS, row = i / C4, c4 = i % C4;
    if (row >= rows) continue;
    const int r = blk * RB + row, tok = x.c0 + (r >> gl), h = r & (G - 1);
    float4 y = O[k];
    float mm = M[k], sum = L[k];
    if (x.part == 2) {
      const float2 ml = __ldcg(a.part_ml + part_row<__nv_bfloat16>(a, 1, tok, kvh, h, gl));
      const float4 z = __ldcg(part_at<__nv_bfloat16, D>(a, 1, tok, kvh, h, c4, gl));
      mm = fmaxf(M[k], ml.x);
      const float w1 = tree_weight(M[k], mm), w0 = tree_weight(ml.x, mm);
      sum = fmaf(w0, ml.y, w1 * sum);
      y = make_float4(y.x * w1, y.y * w1, y.z * w1, y.w * w1);
      tree_fma(y, w0, z);
    }
    const float inv = tree_inv(sum);
    const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
    tree_put(static_cast<__nv_bfloat16*>(a.out) + orow * D + c4 * 4, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
    if (c4 == 0) a.lse[orow] = tree_lse(mm, sum);
  }
}

// -------------------------------------------------------------------------- //
// host side
// -------------------------------------------------------------------------- //
void few_shape(TreeLaunch* a) {
  if (a->kv.dtype != PRHS_BF16) return;
  const long long rows = (long long)a->max_new * (a->kv.Hq / a->kv.Hkv);
  a->few_rows = rows <= 8 ? 8 : 16;
  const long long blocks = (rows + a->few_rows - 1) / a->few_rows;
  a->few_blocks = (int)(blocks < FEW_BLOCKS ? blocks : FEW_BLOCKS);
  const long long units = (long long)a->kv.B * a->kv.Hkv * a->few_blocks;
  a->few_split = units * FEW_SPLIT <= FEW_STATES ? FEW_SPLIT : units * 2 <= FEW_STATES ? 2 : 1;
  a->few_units = (int)units;
}
// The most CTAs that share units in any call of at most max_new tokens a sequence.
static long long few_most(const KVView& kv, int max_new) {
  const long long rows = (long long)max_new * (kv.Hq / kv.Hkv), blocks = (rows + 15) / 16;
  const long long ctas = FEW_SPLIT * (long long)kv.B * kv.Hkv * (blocks < FEW_BLOCKS ? blocks : FEW_BLOCKS);
  return ctas < FEW_STATES ? ctas : FEW_STATES;
}
size_t few_state_bytes(const KVView& kv, int max_new) {
  if (kv.dtype != PRHS_BF16) return 0;
  const size_t rows = (long long)max_new * (kv.Hq / kv.Hkv) <= 8 ? 8 : 16;
  return few_most(kv, max_new) * rows * (kv.d * sizeof(float) + sizeof(float2));
}
size_t few_ticket_bytes(const KVView& kv, int max_new) {
  return kv.dtype != PRHS_BF16 ? 0 : few_most(kv, max_new) * sizeof(int);
}

template <int D, int NT>
static cudaError_t few_go(const TreeLaunch& a, cudaStream_t st) {
  return launch_pdl(few_kernel<D, NT>, dim3((unsigned)(a.few_units * a.few_split)), dim3(FEW_THREADS),
                    FEW_WARPS * sizeof(FewState<D, NT>), st, true, a);
}

cudaError_t launch_shared_join(const TreeLaunch& a, cudaStream_t st) {
  if (a.kv.dtype == PRHS_BF16) {
    if (a.few_rows == 8) return a.kv.d == 128 ? few_go<128, 1>(a, st) : few_go<64, 1>(a, st);
    return a.kv.d == 128 ? few_go<128, 2>(a, st) : few_go<64, 2>(a, st);
  }
  const long long pass = (long long)SJ_THREADS * SJ_PER, y = ((long long)a.max_new * a.kv.Hq * a.kv.d / 4 + pass - 1) / pass;
  const dim3 grid(a.kv.B, (unsigned)(y < 64 ? y : 64));
  if (a.kv.d == 128) return launch_pdl(shared_join_kernel<128>, grid, dim3(SJ_THREADS), 0, st, true, a);
  return launch_pdl(shared_join_kernel<64>, grid, dim3(SJ_THREADS), 0, st, true, a);
}

}  // namespace prhs
