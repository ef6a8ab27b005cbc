// Attention of few query rows, on bf16 caches whose rows share leading
// keys: the part of the tcgen05 kernel's launch (tree_tc.cuh) that computes the states of
// single tokens and drafts against their sequences' own keys (few_item).
// A unit of the tcgen05 part begins and ends in 3 to 4 us, whatever it holds; here
// units are 8 or 16 rows of one KV head, and a warp takes a run of their steps of 16
// keys.
//
// Inside a step: the keys are the 16 rows of mma.sync, query rows its 8 columns, so that
// a warp reads every key once and 8 rows cost 8 columns:
//   S^T = K Q^T,  P^T = exp2(S^T - m) in bf16 (transposed by movmatrix),  O^T += V^T P^T
// Every warp has its own ring in shared memory, which its first lane fills by TMA
// (128-byte swizzle), so that warps wait for nobody but their copies. The ring runs
// ahead into the warp's next unit, and a unit's state is written without waiting for
// anything: states of cut units, and those that meet one against shared keys, are joined
// by the launch behind this one (shared.cu).
//
// Bound: HBM (the keys, once), and latency: lengths, page numbers, keys are dependent
// reads before a warp's first product. 32 sequences of up to 8 drafted tokens on 2048 shared
// and up to 2K own keys, 32 heads, 606 MB: this launch 104 to 114 us, 5.4 to 5.8 TB/s; with
// every unit as tiles 152. The same steps with the keys loaded into registers 120, by
// 16-byte asynchronous copies 173.
#pragma once

#include "tree_join.cuh"

namespace prhs {

constexpr int FEW_WARPS = 8;
constexpr int FEW_STEP = 16;        // keys of a warp's step: a box, never over a page's end
constexpr int few_ring(int d) { return d == 128 ? 16 << 10 : 12 << 10; }  // bytes of a warp's ring: 2 steps, 3 at d = 64
constexpr int FEW_TABLE = 384;      // sequences whose lengths are kept at hand
constexpr int FEW_REST = 4;         // steps that the list counts more behind each unit, which are nothing: what a unit takes beside its own
constexpr int FEW_RUN = 4;          // steps of a warp at least
// A warp's share: its ring, eight rows of a state, the next unit's Q (rows 16 bytes apart, so
// that eight rows' reads hit distinct banks). Behind the shares: the table.
constexpr int few_q(int d) { return few_ring(d) + 8 * d * 4; }
constexpr int few_warp_bytes(int d) { return (few_q(d) + 16 * (d * 2 + 16) + 1023) / 1024 * 1024; }
constexpr int few_smem_bytes(int d) { return FEW_WARPS * few_warp_bytes(d) + FEW_TABLE * 5 * (int)sizeof(int); }
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

// One sequence's share of the list of steps: a unit for each KV head, of steps over the
// cached keys, then the new tokens.
struct FewSeq {
  TreeItem x;
  int steps;  // of a unit (FEW_REST with them; 0: not here)
};
__device__ __forceinline__ int few_steps(const TreeItem& x) {
  return (x.t + FEW_STEP - 1) / FEW_STEP + (x.n + FEW_STEP - 1) / FEW_STEP;
}
__device__ __forceinline__ FewSeq few_seq(const TreeLaunch& a, const TreeItem& x) {
  return {x, x.part == 1 || x.n == 0 || !few_item(a, x.n, x.t) ? 0 : few_steps(x) + FEW_REST};
}

// A unit's steps in a warp's run of the list.
struct FewTask {
  TreeItem x;
  int kvh, s0, s1;         // KV head, steps here
  int cached;              // steps over the cache
  int first, cuts;         // the warp that begins the unit, the warps that have steps of it
  int window, page;        // pages of steps window .. window + 31, one a lane (not looked at before they are used)
  bool some;               // (none: the run is done)
};

struct FewAux {
  uint64_t full[FEW_WARPS][6];
  int steps_to[384];  // of the list, up to a thread's items
};
// The table: five arrays of FEW_TABLE numbers.
__device__ __forceinline__ void few_note(int* table, int b, const TreeItem& x) {
  table[b] = x.base;
  table[FEW_TABLE + b] = x.t;
  table[2 * FEW_TABLE + b] = x.c0;
  table[3 * FEW_TABLE + b] = x.n;
  table[4 * FEW_TABLE + b] = x.part;
}

// A CTA's part: warps 0 .. 7 of CTA `cta` of `ctas` take runs of the list of all_steps
// steps; a thread of the launch has per_t items (steps_to).
template <int D, int NT>
__device__ __forceinline__ void few_role(const TreeLaunch& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                         const CUtensorMap& knmap, const CUtensorMap& vnmap, uint8_t* few_smem, FewAux& aux,
                                         int per_t, int all_steps, int cta, int ctas, int gl) {
  // a step's K, then its V: SEGS column segments of 16 rows of 128 bytes
  constexpr int RB = 8 * NT, C4 = D / 4, SEGS = D / 64, SEG = FEW_STEP * 128, STAGE = 2 * SEGS * SEG, STAGES = few_ring(D) / STAGE;
  constexpr int WARP_SMEM = few_warp_bytes(D), QS = D * 2 + 16;  // (bytes from one row of Q to the next)
  static_assert(STAGES <= 6 && few_ring(D) % STAGE == 0 && WARP_SMEM % 1024 == 0, "ring");
  const KVView& kv = a.kv;
  const int G = 1 << gl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int gw = cta * FEW_WARPS + warp, gws = ctas * FEW_WARPS;
  auto& full = aux.full;
  if (warp == 0 && lane < 4) prefetch_tmap(lane == 0 ? &kmap : lane == 1 ? &vmap : lane == 2 ? &knmap : &vnmap);
  if (lane == 0) {
    for (int i = 0; i < STAGES; i++) mbar_init(&full[warp][i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  // Every warp takes an equal run. A unit cut by the end of one leaves states for the join; runs
  // of a step or two would cost more than they give.
  const int run = max((all_steps + gws - 1) / gws, FEW_RUN);
  int pos = min(all_steps, gw * run);
  const int end = min(all_steps, pos + run);

  const bool causal = a.mask == nullptr;
  const uint32_t ring = smem_addr(few_smem) + warp * WARP_SMEM;
  float4* staged = reinterpret_cast<float4*>(few_smem + warp * WARP_SMEM + few_ring(D));  // [C4][8]
  const float sc = a.scale * FEW_LOG2E;

  uint8_t* next_q = few_smem + warp * WARP_SMEM + few_q(D);
  const int* table = reinterpret_cast<const int*>(few_smem + FEW_WARPS * WARP_SMEM);
  auto seq_at = [&](int b) {
    if (kv.B > FEW_TABLE) return few_seq(a, tree_item<true>(a, 2 * b + 1, true));
    TreeItem x;
    x.b = b;
    x.base = table[b];
    x.t = table[FEW_TABLE + b];
    x.c0 = table[2 * FEW_TABLE + b];
    x.n = table[3 * FEW_TABLE + b];
    x.part = table[4 * FEW_TABLE + b];
    return few_seq(a, x);
  };
  auto look_up = [&](FewTask& t, int window) {
    t.window = window;
    const int s = window + lane;
    if (kv.block_table != nullptr && s < min(t.s1, t.cached))
      t.page = kv.block_table[(long long)t.x.b * kv.max_blocks + (t.x.base + s * FEW_STEP) / kv.block_size];
  };
  auto fetch = [&]() {  // at pos, which moves on
    FewTask t = {};
    FewSeq s = {};
    int kvh = 0, in = 0;
    for (;; pos += s.steps - in) {
      if (pos >= end) return t;
      int lo = 0, hi = 383;  // the first thread whose items end behind it
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (aux.steps_to[mid] > pos) hi = mid; else lo = mid + 1;
      }
      int off = pos - (lo > 0 ? aux.steps_to[lo - 1] : 0), b = (lo * per_t) >> 1;  // (items 2 b + 1 have steps)
      s = seq_at(b);
      for (int x; off >= (x = kv.Hkv * s.steps);) {
        off -= x;
        s = seq_at(++b);
      }
      kvh = off / s.steps;
      in = off - kvh * s.steps;
      if (in < s.steps - FEW_REST) break;
    }
    const int start = pos - in;
    t.x = s.x;
    t.kvh = kvh;
    const int taken = min(s.steps - in, end - pos);  // of the list
    pos += taken;
    t.some = true;
    t.first = start / run;
    t.cuts = (start + s.steps - FEW_REST - 1) / run - t.first + 1;
    const int all = s.steps - FEW_REST;
    t.cached = (t.x.t + FEW_STEP - 1) / FEW_STEP;
    t.s0 = min(in, all);
    t.s1 = min(in + taken, all);
    look_up(t, t.s0);
    // its Q rows, zeros behind its last
    __syncwarp();
#pragma unroll
    for (int i = 0; i < RB * D / 8 / 32; i++) {
      const int y = lane + 32 * i, r = y / (D / 8), piece = y % (D / 8);
      const bool have = r < t.x.n << gl;
      const __nv_bfloat16* from =
          static_cast<const __nv_bfloat16*>(a.q) +
          (have ? ((long long)(t.x.c0 + (r >> gl)) * kv.Hq + (t.kvh << gl) + (r & (G - 1))) * D + piece * 8 : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(next_q + y / (D / 8) * QS + piece * 16)),
                   "l"(from), "r"(have ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return t;
  };
  int counts = 0;  // keys of the ring's steps, five bits each
  auto load = [&](FewTask& t, int s, int stage) {
    if (s >= t.window + 32) look_up(t, t.window + 32);
    const int page = __shfl_sync(FULL_MASK, t.page, s - t.window), j = (s - t.cached) * FEW_STEP, key = t.x.base + s * FEW_STEP;
    const bool is_new = s >= t.cached;
    int row = (t.x.b * kv.Hkv + t.kvh) * kv.t_max + key;  // of the cache
    if (kv.block_table != nullptr) row = (page * kv.Hkv + t.kvh) * kv.block_size + key % kv.block_size;
    if (!is_new && kv.block_table != nullptr && (unsigned)page >= (unsigned)kv.num_blocks) {
      if (lane == 0) raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
      row = -1;
    }
    const int n = is_new ? min(FEW_STEP, t.x.n - j) : row < 0 ? 0 : min(FEW_STEP, t.x.t - s * FEW_STEP);
    counts = (counts & ~(31 << 5 * stage)) | n << 5 * stage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[warp][stage], STAGE);
      const CUtensorMap *km = is_new ? &knmap : &kmap, *vm = is_new ? &vnmap : &vmap;
      const int z = is_new ? t.kvh : max(row, 0), w = is_new ? t.x.c0 + j : 0;
#pragma unroll
      for (int i = 0; i < SEGS; i++) tma_load_4d(ring + stage * STAGE + i * SEG, km, 0, i, z, w, &full[warp][stage]);
#pragma unroll
      for (int i = 0; i < SEGS; i++) tma_load_4d(ring + stage * STAGE + (SEGS + i) * SEG, vm, 0, i, z, w, &full[warp][stage]);
    }
    __syncwarp();
  };
  // The copies run ahead of the products into the next task, which is known while this one is worked on.
  int fill = 0, held = 0, stage = 0;  // the stage to fill next, stages filled, the stage to use next
  uint32_t phase = 0;
  bool dead = false, in_next = false;
  FewTask cur = fetch(), nxt;
  int cursor = cur.s0;
  for (; cur.some; cur = nxt) {
    if (!in_next) cursor = cur.s0;
    in_next = false;
    bool known = false;
    const TreeItem x = cur.x;
    const int kvh = cur.kvh;
    const int rows = x.n << gl, cached = cur.cached;
    // Q as the products take it: rows g of each eight, columns 16 j + 2 c and 16 j + 8 + 2 c
    uint32_t q[NT][D / 16][2];
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int j = 0; j < D / 16; j++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          q[t][j][h] = *reinterpret_cast<const uint32_t*>(next_q + (8 * t + g) * QS + (16 * j + 8 * h + 2 * c) * 2);

    float m[NT][2], l[NT][2], o[NT][D / 16][4];  // rows 8 t + 2 c, + 1; O's columns 16 e + g, + 8
#pragma unroll
    for (int t = 0; t < NT; t++) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int e = 0; e < D / 16; e++) o[t][e][0] = o[t][e][1] = o[t][e][2] = o[t][e][3] = 0.f;
    }
    // a lane's row of the four matrices of a product's operand: K's rows lane % 16, columns 8 (lane / 16) ..;
    // V's the other way about (its matrices come in the order of d, then keys)
    const int krow = lane & 15, kcol = lane >> 4, vrow = (lane & 7) + (lane >> 4) * 8, vcol = lane >> 3 & 1;
    const uint32_t k_at = ring + krow * 128, v_at = ring + SEGS * SEG + vrow * 128;
    for (int s = cur.s0;; s++) {
      while (held < STAGES) {
        if (!in_next && cursor >= cur.s1) {
          if (!known || !nxt.some) break;
          in_next = true;
          cursor = nxt.s0;
        }
        if (in_next && cursor >= nxt.s1) break;
        load(in_next ? nxt : cur, cursor++, fill);
        fill = fill + 1 == STAGES ? 0 : fill + 1;
        held++;
      }
      if (!known) {
        nxt = fetch();
        known = true;
      }
      if (s >= cur.s1) break;
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
              const int tok = min((8 * t + 2 * c + (i & 1)) >> gl, x.n - 1);
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
      held--;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (dead) break;

    // ---- its state, four columns a lane: row lane % 8 of each eight, columns 4 (lane / 8 + 4 k) .. ----
    const int sr = lane & 7, sq = lane >> 3;
    float2 ml[NT];
    float4 y[NT][C4 / 4];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 2; r++) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][r] += __shfl_xor_sync(FULL_MASK, l[t][r], d);
#pragma unroll
        for (int e = 0; e < D / 16; e++)
#pragma unroll
          for (int h = 0; h < 2; h++)
            reinterpret_cast<float*>(staged + (4 * e + 2 * h + g / 4) * 8 + 2 * c + r)[g % 4] = o[t][e][2 * h + r];
      }
      __syncwarp();
      // (row 8 t + 2 c + r is in lanes c of any g)
      const float m0 = __shfl_sync(FULL_MASK, m[t][0], sr >> 1), m1 = __shfl_sync(FULL_MASK, m[t][1], sr >> 1);
      const float l0 = __shfl_sync(FULL_MASK, l[t][0], sr >> 1), l1 = __shfl_sync(FULL_MASK, l[t][1], sr >> 1);
      ml[t] = sr & 1 ? make_float2(m1, l1) : make_float2(m0, l0);
#pragma unroll
      for (int k = 0; k < C4 / 4; k++) y[t][k] = staged[(sq + 4 * k) * 8 + sr];
    }

    // a unit cut by the run's end, or with a state against shared keys, is for the join; nothing
    // here waits for what it writes (or for the launch in front)
    const bool cut = cur.cuts > 1, result = !cut && x.part == 0;
    float4* states = static_cast<float4*>(a.few_states);  // [2 warps][C4][RB], then (maximum, sum) [2 warps][RB]
    float2* sums = reinterpret_cast<float2*>(states + (long long)2 * a.few_warps * C4 * RB);
    const long long slot = 2ll * gw + (cur.first == gw);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int r = 8 * t + sr, tok = x.c0 + (r >> gl), h = r & (G - 1);
      if (r >= rows) continue;
      const long long prow = part_row<__nv_bfloat16>(a, 2, tok, kvh, h, gl), orow = (long long)tok * kv.Hq + (kvh << gl) + h;
      const float inv = tree_inv(ml[t].y);
#pragma unroll
      for (int k = 0; k < C4 / 4; k++) {
        const int c4 = sq + 4 * k;
        if (result)
          tree_put(static_cast<__nv_bfloat16*>(a.out) + orow * D + c4 * 4,
                   make_float4(y[t][k].x * inv, y[t][k].y * inv, y[t][k].z * inv, y[t][k].w * inv));
        else if (cut)
          __stcg(states + (slot * C4 + c4) * RB + 8 * t + sr, y[t][k]);
        else
          __stcg(part_at<__nv_bfloat16, D>(a, 2, tok, kvh, h, c4, gl), y[t][k]);
      }
      if (sq != 0) continue;
      if (result) a.lse[orow] = tree_lse(ml[t].x, ml[t].y);
      else if (cut) __stcg(sums + slot * RB + 8 * t + sr, ml[t]);
      else __stcg(a.part_ml + prow, ml[t]);
      // (warps that begin no step of a unit do not know its first)
      if (cur.first == gw) a.where[prow] = make_int2(cur.first, cur.cuts);
    }
  }
  if (dead)  // nothing may still be in flight when the CTA ends
    for (int i = 0; i < held; i++) {
      mbar_wait(&full[warp][stage], phase, kv.err);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
}

}  // namespace prhs
