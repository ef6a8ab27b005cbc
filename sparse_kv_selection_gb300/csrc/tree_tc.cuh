// Attention of a batch of new tokens over their sequences' caches and over
// each other, bf16, on the fifth-generation tensor cores.
//
// The G query heads of one KV head see the same keys, so the rows of one
// (sequence, KV head) are its tokens times G (row = token * G + head of the
// group), cut into units of UNIT_ROWS = 256 rows. A unit's keys are tiles of 128:
// the cache's, then the new tokens'. All tiles of all units are one list; every
// CTA (one per SM) takes an equal run of it, so long caches are split and short
// ones packed without a plan made on the host. A unit cut by a run's end leaves
// partial states in the workspace, which a second launch joins row by row (units
// of a few tiles are not cut).
//
// Inside a CTA: two warps load K and V tiles by TMA into a ring of 128-key
// slots (128-byte swizzle), half the boxes of each tile each (a tile on 16-key
// pages is 16 copies of 2 KB, more than one thread issues at HBM's rate: 658 us
// with one warp, 640 with two, for the batch below). The scheduler's warp walks
// the list for the others and loads the units' Q tiles into two more slots.
// One thread issues the matrix instructions, and two warpgroups do the
// softmax, one per stream. A stream is a logit tile S [128 rows][128 keys] and an
// output tile O [128][D] in tensor memory:
//   S = Q K^T      (both from shared memory, 8 or 4 instructions of 16 elements)
//   P = exp2(S - m) in bf16 over S's own columns, one row a thread
//   O += P V       (P from tensor memory, V read d-major from its slot)
// With more than 128 rows the streams are the unit's two row tiles and share
// every K and V tile; with fewer they take the even and the odd key tiles, so
// that one stream's products run under the other's softmax either way. The two
// outputs of the second form are joined when the unit ends: both warpgroups
// read both tiles, half the columns each.
//
// The reference m of a row follows its running maximum only when that has grown
// by more than 8 (a factor 256 in the weights): O is then rescaled in tensor
// memory, at a few tiles of a row instead of all. The weights stay below 2^8
// and sums are fp32, so nothing is lost: l and O carry the same factor.
//
// P is rounded to bf16 (by up to half a unit of the type the result is rounded
// to, and without bias over the keys); l is summed before that rounding, m, l
// and O are fp32.
//
// Bound: HBM while a KV head has up to about 256 query rows (K and V are read
// once: 512 bytes a key at d = 128 against 4 * 128 * rows flops): 32 sequences of
// 2K-16K keys on 16-key pages, 32 KV heads, trees of 1-32 tokens, 4.25 GB: 630 us,
// the measured copy bandwidth. Above that the tensor cores and the
// softmax between their products: 5250 causal tokens on cached prefixes, 32 / 8
// heads: 388-391 us from a graph, 1480-1490 TFLOP/s, 0.80 of the measured matrix rate;
// single calls back to back 414-420 us, 0.74, at the power cap's clocks (a step of a
// stream is 1550 clocks, its two products 1031; the rest is the wait of one
// product for the softmax, 1250 clocks of 128 exponentials a thread). Few tiles
// a CTA (4096 keys, 32 heads): latency, 2.3 us to the first copy, 3 us from it to
// the first weights, 3 us of joining.
#pragma once

#include "few.cuh"
#include "tree_join.cuh"

namespace prhs {

constexpr int TT = 128;                  // keys of a tile, rows of a stream
constexpr int UNIT_ROWS = 2 * TT;
constexpr int TC_WARPS = 12;             // 8 softmax, two K/V producers, matrix issuer, scheduler
// Registers a thread: the softmax warpgroups hold a row of logits each, so they
// take over part of the third one's. The three shares add up to what the block
// is launched with (checked before the launch: a larger sum would wait forever).
constexpr int TC_REGS_LAUNCH = 168, TC_REGS_SOFTMAX = 224, TC_REGS_REST = 56;
static_assert(2 * TC_REGS_SOFTMAX + TC_REGS_REST <= 3 * TC_REGS_LAUNCH, "register shares");
constexpr int TC_THREADS = TC_WARPS * 32;
constexpr int TC_AUX = 3 << 10;          // bytes of shared memory beside the tiles
constexpr float TC_LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.f;
constexpr int QUAD_ROWS = 32;
constexpr int UNCUT_TILES = 12;  // the most tiles of a unit in a list that is not cut

template <int D>
struct TcShape {
  static constexpr int SEGS = D / 64;             // 128-byte column segments of a row
  static constexpr int SEG = TT * 128;            // bytes of one segment of a tile
  static constexpr int TILE = SEGS * SEG;
  static constexpr int SLOTS = D == 128 ? 5 : 10; // K and V tiles in flight
  static constexpr int DATA = (SLOTS + 2) * TILE; // the ring and two Q tiles
  static constexpr size_t SMEM = (size_t)DATA + TC_AUX;
};

// One unit's tiles in a CTA's run, as the scheduler warp hands it to the others.
constexpr int TC_WORKS = 4;
struct __align__(16) TcWork {
  int b, kvh, c0, n;        // sequence, KV head, first token, tokens
  int t, tok0, rows, tile0; // cached keys, the unit's first token and rows, its first tile here
  int nt, cache_tiles, loads, qtiles;  // tiles here; K and V / Q tiles loaded before
  int whole, last;          // all of the unit's tiles are here; the run ends with it
  int base, part;           // the first cached key; where its state goes (TreeItem)
  int first, cuts, pad[2];  // the CTA that begins the unit, the CTAs that have tiles of it

  __device__ __forceinline__ bool single() const { return rows <= TT; }
  // steps of the unit: step x is stream x & 1 on tile tile0 + (single ? x : x / 2)
  __device__ __forceinline__ int steps() const { return single() ? nt : 2 * nt; }
  // Order of the loads: as the issuer first uses them (S of steps 0 and 1, then
  // O of step x and S of step x + 2).
  __device__ __forceinline__ int load_tile(int l, bool& is_v) const {
    if (!single()) {
      is_v = l & 1;
      return l >> 1;
    }
    const bool end = l == 2 * nt - 1;
    is_v = end || (l > 0 && (l & 1) == 0);
    return end ? nt - 1 : is_v ? (l - 2) >> 1 : (l + 1) >> 1;
  }
  __device__ __forceinline__ int load_v(int i) const { return loads + (single() ? min(2 * i + 2, 2 * nt - 1) : 2 * i + 1); }
};

// A place in the ring of SLOTS slots: the slot and the parity of its use.
template <int SLOTS>
struct TcRing {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ explicit TcRing(int g) : slot(g % SLOTS), phase((g / SLOTS) & 1) {}
  __device__ __forceinline__ void step(int n) {  // n < SLOTS
    slot += n;
    if (slot >= SLOTS) {
      slot -= SLOTS;
      phase ^= 1;
    }
  }
};

struct TcSeq : TreeItem {  // one item's share of the list
  int blocks;        // units of one KV head
  int cache_tiles;
  int tiles;         // tiles of one KV head
};

// What a tile of one and of two row tiles takes, in the few rows' steps: 9 and 12 are what
// ends both parts at about the same time (8 and 10, 10 and 14: 8 groups of 16 sequences 100
// and 98 us instead of 92).
constexpr int TC_COST_1 = 9, TC_COST_2 = 12;

struct TcBars {  // one mbarrier each
  uint64_t full[10], empty[10], qfull[2], qempty[2], sfull[2], pfull[2][2], ofull[2], done;
  uint64_t wfull[TC_WORKS], wempty[TC_WORKS];
};
struct TcAux {
  union {
    struct {
      float m[2][TT], l[2][TT];  // row states of the two streams
    };
    FewAux few;
  };
  TcWork work[TC_WORKS];
  TcBars bar;
  uint32_t tmem;
  int bad_page;
  int start_item, start_off;  // where the run begins
  int begin, end;          // the run
  int wsum[TC_WARPS], wmax[TC_WARPS];
  int fsum[TC_WARPS];      // (shared keys) steps of the few rows' list
  long long cost[TC_WARPS];  // what the tiles' list takes, in steps of the other
  long long grouped[TC_WARPS];  // tokens of all groups
};
static_assert(sizeof(TcAux) <= TC_AUX, "aux region");

struct TcLaunch {
  TreeLaunch a;
  TreeRecords rec;
  int box_log2;  // log2 of the rows of a cache TMA box
};

// -------------------------------------------------------------------------- //
// tensor-core primitives (inline PTX)
// -------------------------------------------------------------------------- //
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// A whole logit row: 128 columns in four loads.
__device__ __forceinline__ void tmem_ld_row(uint32_t (&r)[TT], uint32_t addr) {
#pragma unroll
  for (int c = 0; c < 4; c++) tmem_ld32(reinterpret_cast<uint32_t(&)[32]>(r[c * 32]), addr + c * 32);
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle: start address, the byte
// distances between 64-element repeats (lead) and between groups of 8 rows (step).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t step) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(step >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 operands, fp32 accumulator, M = 128; B is
// K-major (rows of K) or N-major (V, d contiguous).
__device__ constexpr uint32_t instr_desc(int n, bool b_nmajor) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_nmajor ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(TT >> 4) << 24);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (f2, unf2, fma2: two fp32 numbers in a register pair)
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Lanes that differ in bit B trade the second element of the lower for the first
// of the upper.
template <int B>
__device__ __forceinline__ void quad_swap(uint32_t (&x)[4], uint32_t (&y)[4]) {
  const bool up = threadIdx.x & B;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const uint32_t z = __shfl_xor_sync(FULL_MASK, up ? x[k] : y[k], B);
    x[k] = up ? z : x[k];
    y[k] = up ? y[k] : z;
  }
}

// The softmax warps meet: true where all of them are about to leave. A warp that has
// left its units (at the run's end, or early because a wait gave up) meets the others
// until that is so, so that none of them waits here for one that is gone. (An
// mbarrier and a bounded wait instead: 4096 keys 19.5 -> 20.0 us, causal chunks 387 -> 394.)
__device__ __forceinline__ bool softmax_meet(bool leaving) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)leaving), "n"(2 * TT)
      : "memory");
  return r != 0;
}

// -------------------------------------------------------------------------- //
// the list of tiles
// -------------------------------------------------------------------------- //
// New-token tiles of the units before unit j (1 << ul tokens each): a causal
// unit sees the tokens up to its own last one, a tree unit all of them (one tile).
__device__ __forceinline__ int new_tiles_before(int j, int blocks, int n, int ul, bool causal) {
  if (!causal) return j;
  const bool all = j == blocks;
  const int k = all ? j - 1 : j;  // units that end at their own last token
  int s;
  if (ul >= 7) {
    s = (k * (k + 1) / 2) << (ul - 7);
  } else {  // sum over i = 1 .. k of ceil(i / p), p = 2^(7 - ul)
    const int pl = 7 - ul, q = k >> pl, r = k - (q << pl);
    s = ((q * (q + 1) / 2) << pl) + r * (q + 1);
  }
  return all ? s + ((n + TT - 1) >> 7) : s;
}

// Tiles of the units of item s before unit j. With shared keys a batch may have many
// units of a tile or two beside long ones, and a unit takes 3 to 4 us beside its tiles:
// the list then counts REST tiles more behind each, which are nothing.
template <bool SHARED>
constexpr int REST = SHARED ? 2 : 0;
template <bool SHARED>
__device__ __forceinline__ int tiles_before(const TcSeq& s, int j, int ul, bool causal) {
  return j * (s.cache_tiles + REST<SHARED>) + (s.part == 1 ? 0 : new_tiles_before(j, s.blocks, s.n, ul, causal));
}
template <bool SHARED>
__device__ __forceinline__ TcSeq tc_seq(const TreeLaunch& a, int e, int ul) {
  TcSeq s;
  static_cast<TreeItem&>(s) = tree_item<SHARED>(a, e);
  s.blocks = (s.n + (1 << ul) - 1) >> ul;
  s.cache_tiles = (s.t + TT - 1) >> 7;
  s.tiles = s.blocks == 0 ? 0 : tiles_before<SHARED>(s, s.blocks, ul, a.mask == nullptr);
  return s;
}
// Tiles of unit `block`.
__device__ __forceinline__ int tc_unit_tiles(const TcSeq& s, int block, int ul, bool causal) {
  if (s.part == 1) return s.cache_tiles;
  return s.cache_tiles + (causal ? (min(s.n, (block + 1) << ul) + TT - 1) >> 7 : 1);
}
// The unit that holds tile `off` of an item's share: KV head, unit, the tile's
// number in it and the tiles from there to where a run that would begin there does: the
// next unit's first tile (0 from a first one), or, where units may be cut, the tile itself.
template <bool SHARED>
__device__ __forceinline__ int4 tc_unit_at(const TreeLaunch& a, int e, int off, int ul, bool uncut) {
  const bool causal = a.mask == nullptr;
  const TcSeq s = tc_seq<SHARED>(a, e, ul);
  const int kvh = off / s.tiles;
  off -= kvh * s.tiles;
  int block = 0, hi = s.blocks - 1;
  while (block < hi) {
    const int mid = (block + hi + 1) >> 1;
    if (tiles_before<SHARED>(s, mid, ul, causal) <= off) block = mid; else hi = mid - 1;
  }
  off -= tiles_before<SHARED>(s, block, ul, causal);
  const int tiles = tc_unit_tiles(s, block, ul, causal);
  if (SHARED && !uncut && off < tiles) return make_int4(kvh, block, off, 0);
  return make_int4(kvh, block, off, off == 0 ? 0 : tiles + REST<SHARED> - off);
}

// -------------------------------------------------------------------------- //
// the kernel
// -------------------------------------------------------------------------- //
// NT: 0, or (shared keys) eights of query rows of a unit of the few rows' list.
template <int D, int NT>
__global__ void __launch_bounds__(TC_THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ktail,
                   const __grid_constant__ CUtensorMap vtail, const __grid_constant__ CUtensorMap knmap,
                   const __grid_constant__ CUtensorMap vnmap, const __grid_constant__ TcLaunch p) {
  using S = TcShape<D>;
  constexpr bool SHARED = NT > 0;
  constexpr int NT1 = NT > 0 ? NT : 1;
  static_assert(!SHARED || few_smem_bytes(D) <= S::DATA, "the few rows' rings take the tiles' place");
  extern __shared__ __align__(1024) uint8_t tc_smem[];
  const TreeLaunch& a = p.a;
  const KVView& kv = a.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = SHARED ? 2 * kv.B : kv.B, gl = p.rec.group_log2, ul = 8 - gl;  // log2 of the group and of a unit's tokens
  const uint32_t base = smem_addr(tc_smem);
  uint8_t* data = tc_smem;
  TcAux& aux = *reinterpret_cast<TcAux*>(data + S::DATA);
  TcBars& bar = aux.bar;

  // ---- what needs nothing of earlier launches: barriers, tensor memory ----
  if (warp == 10 && lane == 0) {
    for (int i = 0; i < S::SLOTS; i++) {
      mbar_init(&bar.full[i], 2);  // one arrival of each producer
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&bar.qfull[i], 1);
      mbar_init(&bar.qempty[i], 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.pfull[i][0], TT);
      mbar_init(&bar.pfull[i][1], TT);
      mbar_init(&bar.ofull[i], 1);
    }
    for (int i = 0; i < TC_WORKS; i++) {
      mbar_init(&bar.wfull[i], 1);
      mbar_init(&bar.wempty[i], TC_WARPS - 1);
    }
    mbar_init(&bar.done, 1);
    fence_barrier_init();
    aux.bad_page = 0;
    if ((base & 1023) != 0) raise_error(kv.err, PRHS_DEV_CAPACITY);  // the swizzle needs it
  }
  if (warp == 8 && lane < 3) prefetch_tmap(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
  pdl_wait();
  pdl_trigger();
  // (the join of a CTA that gives up reads this)
  if (!SHARED && tid == 0) p.rec.split[blockIdx.x] = TreeSplit{};

  // ---- this CTA's run of the list of all tiles ----
  const int per_t = (items + TC_THREADS - 1) / TC_THREADS, e0 = tid * per_t;
  int mine = 0, most = 0;  // tiles of this thread's items, of their largest unit
  int steps = 0;           // of the few rows' list
  long long cost = 0, grouped = 0;
  bool back = false;       // offsets that step back: sequences would overlap, and counts pass 32 bits
  for (int e = e0; e < min(items, e0 + per_t); e++) {
    const TcSeq s = tc_seq<SHARED>(a, e, ul);
    back |= a.cu_new[s.b + 1] < a.cu_new[s.b];
    mine += kv.Hkv * s.tiles;
    if (s.blocks > 0) most = max(most, tc_unit_tiles(s, s.blocks - 1, ul, a.mask == nullptr) + REST<SHARED>);
    if constexpr (SHARED) {
      if (s.part == 1) grouped += s.n;
      cost += (long long)kv.Hkv * s.tiles * ((s.n << gl) > TT ? TC_COST_2 : TC_COST_1);
      if (e & 1) {
        const FewSeq f = few_seq(a, tree_item<true>(a, e, true));
        steps += kv.Hkv * f.steps;
      }
    }
  }
  most = __reduce_max_sync(FULL_MASK, most);
  int run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL_MASK, run, o);
    if (lane >= o) run += y;
  }
  if constexpr (SHARED) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL_MASK, steps, o);
      if (lane >= o) steps += y;
      cost += __shfl_xor_sync(FULL_MASK, cost, o);
      grouped += __shfl_xor_sync(FULL_MASK, grouped, o);
    }
    if (lane == 31) {
      aux.fsum[warp] = steps;
      aux.cost[warp] = cost;
      aux.grouped[warp] = grouped;
    }
  }
  if (lane == 31) {
    aux.wsum[warp] = run;
    aux.wmax[warp] = most;
  }
  back = __syncthreads_or(back);
  if constexpr (SHARED) {
    grouped = 0;
#pragma unroll
    for (int w = 0; w < TC_WARPS; w++) grouped += aux.grouped[w];
    if (groups_overlap(a, grouped, tid)) back = true;
    if (blockIdx.x == 0 && tid == 0) *a.part_ok = !back;
  }
  if (back) return;  // (flagged above)
  int total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < TC_WARPS; w++) {
    const int x = aux.wsum[w];
    if (w < warp) before += x;
    total += x;
    most = max(most, aux.wmax[w]);
  }
  before += run - mine;
  // With shared keys the first CTAs take runs of the tiles and the others of the few rows' steps,
  // as many as the two lists take: both begin at once. (Every CTA first one, then the other: 105 us
  // instead of 92, the second list's latencies come behind the first's.)
  int all_steps = 0, ctas = gridDim.x;
  if constexpr (SHARED) {
    cost = 0;
#pragma unroll
    for (int w = 0; w < TC_WARPS; w++) {
      const int x = aux.fsum[w];
      if (w < warp) steps += x;
      all_steps += x;
      cost += aux.cost[w];
    }
    if (all_steps > 0)
      ctas = cost == 0 ? 0 : max(1, min(ctas - 1, (int)((ctas * cost + (cost + all_steps) / 2) / (cost + all_steps))));
  }
  const bool tile_cta = (int)blockIdx.x < ctas;
  const int per = (total + max(ctas, 1) - 1) / max(ctas, 1);
  // Runs are [g0, g1), or, where cutting units costs more than it gives, they begin
  // at the unit that begins there or next. Joining takes about 4 us, a tile 0.8 or
  // (two row tiles) 1.6, so runs may be up to five tiles longer instead, on units so
  // short that they do not differ by more: 512 causal tokens on 512 keys, 32 / 8 heads,
  // 24.2 us (cut: 26.8); 4 chunks of 184 on 217 keys 19.6 (26.1); 32 drafts of 8 on 500
  // keys 23.3 (24.5). The search costs long caches 0.6 us at most.
  const int g0 = blockIdx.x * per, g1 = min(total, g0 + per);
  most = max(most, 1);
  const bool uncut = most <= UNCUT_TILES && (per + most - 1) / most * most - per <= min(2 * per, 5);
#pragma unroll 1
  for (int i = 0; i <= (int)uncut; i++) {
    const int g = i == 0 ? g0 : g1;
    if (g >= total || g < before || g >= before + mine) continue;  // not in this thread's items
    int off = g - before;
    for (int k = 0; k < per_t; k++) {
      const int e = tid * per_t + k, x = kv.Hkv * tc_seq<SHARED>(a, e, ul).tiles;
      if (off < x) {
        const int skip = uncut || (SHARED && i == 0) ? tc_unit_at<SHARED>(a, e, off, ul, uncut).w : 0;
        if (i == 0) {
          aux.start_item = e;
          aux.start_off = off + skip;  // (may lead to the next item)
          aux.begin = g + skip;
        }
        if (i == 1 || !uncut || g1 >= total) aux.end = i == 1 ? g + skip : g1;
        break;
      }
      off -= x;
    }
  }
  __syncthreads();
  tc_fence_after();
  const bool tiles_here = g0 < g1 && aux.begin < aux.end;
  if ((!SHARED && !tiles_here) || (base & 1023) != 0) return;
  const bool some = !SHARED || tiles_here;
  if (warp == 9 && some) {  // tensor memory: S0, S1 (128 columns each), O0, O1 (D each)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&aux.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = some ? aux.tmem : 0;
  // The tiles are done. A CTA with none of them has steps: everyone hands over how many its
  // items have, where the softmax warps' states would be.
  auto tiles_done = [&](auto between) {
    __syncthreads();
    if (warp == 9 && some) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if constexpr (SHARED) {
      aux.few.steps_to[tid] = steps;
      between();
      __syncthreads();
    }
  };

  // The next unit of the run, false when a wait gave up. Every warp but the
  // scheduler's takes each one once.
  int taken = 0;
  auto take = [&](TcWork& w) -> bool {
    const int i = taken & (TC_WORKS - 1);
    const bool ok = __all_sync(FULL_MASK, mbar_wait(&bar.wfull[i], (taken / TC_WORKS) & 1, kv.err));
    if (ok) w = aux.work[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.wempty[i]);
    taken++;
    return ok;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_REGS_REST));
    if (!some) {
    } else if (warp == 11) {
      // ---------------------- scheduler, and Q producer ---------------------- //
      const bool leader = elect_one();
      int item = aux.start_item, off = aux.start_off, left = aux.end - aux.begin, loads = 0, qtiles = 0;
      const bool causal = a.mask == nullptr;
      TcSeq s = tc_seq<SHARED>(a, item, ul);
      while (off >= kv.Hkv * s.tiles) {
        off -= kv.Hkv * s.tiles;
        s = tc_seq<SHARED>(a, ++item, ul);
      }
      // With shared keys most items may have no tiles here, and finding that out takes 0.6 us of
      // dependent reads: 32 are looked at together, one a lane (640 single tokens in 19 small
      // groups: 420 us one by one).
      TcSeq ahead = {};
      int ahead0 = 0, ahead_some = 0;  // item of lane 0; lanes whose items are still to come
      auto next_item = [&]() {
        if constexpr (SHARED) {
          while (ahead_some == 0 && item + 1 < items) {
            ahead0 = item + 1;
            ahead.blocks = 0;
            if (ahead0 + lane < items) ahead = tc_seq<SHARED>(a, ahead0 + lane, ul);
            ahead_some = __ballot_sync(FULL_MASK, ahead.blocks > 0);
            item = min(items, ahead0 + 32) - 1;
          }
          if (ahead_some == 0) return false;  // (there is one while tiles are left)
          const int from = __ffs(ahead_some) - 1;
          ahead_some &= ahead_some - 1;
          s.b = __shfl_sync(FULL_MASK, ahead.b, from);
          s.base = __shfl_sync(FULL_MASK, ahead.base, from);
          s.t = __shfl_sync(FULL_MASK, ahead.t, from);
          s.c0 = __shfl_sync(FULL_MASK, ahead.c0, from);
          s.n = __shfl_sync(FULL_MASK, ahead.n, from);
          s.part = __shfl_sync(FULL_MASK, ahead.part, from);
          s.blocks = __shfl_sync(FULL_MASK, ahead.blocks, from);
          s.cache_tiles = __shfl_sync(FULL_MASK, ahead.cache_tiles, from);
        } else {
          do s = tc_seq<SHARED>(a, ++item, ul);
          while (s.blocks == 0);
        }
        return true;
      };
      const int4 at = tc_unit_at<SHARED>(a, item, off, ul, false);
      int kvh = at.x, block = at.y;
      off = at.z;
      for (int k = 0;; k++) {
        const int tiles = tc_unit_tiles(s, block, ul, causal);
        const int nt = min(tiles - off, left);
        const int start = SHARED ? aux.end - left - off : 0;  // the list's number of the unit's first tile
        left -= nt;
        if (SHARED && off + nt == tiles) left -= min(left, REST<SHARED>);
        const int i = k & (TC_WORKS - 1);
        if (!__all_sync(FULL_MASK, mbar_wait(&bar.wempty[i], ((k / TC_WORKS) & 1) ^ 1, kv.err))) break;
        const int rows = min(UNIT_ROWS, (s.n - (block << ul)) << gl);
        if (lane == 0) {
          TcWork& w = aux.work[i];
          w.b = s.b;
          w.kvh = kvh;
          w.c0 = s.c0;
          w.n = s.n;
          w.t = s.t;
          w.tok0 = block << ul;
          w.rows = rows;
          w.tile0 = off;
          w.nt = nt;
          w.cache_tiles = s.cache_tiles;
          w.loads = loads;
          w.qtiles = qtiles;
          w.whole = nt == tiles;
          w.last = left == 0;
          if constexpr (SHARED) {
            w.base = s.base;
            w.part = s.part;
            w.first = nt == tiles ? (int)blockIdx.x : start / per;
            w.cuts = nt == tiles ? 1 : (start + tiles - 1) / per - w.first + 1;
          }
          mbar_arrive(&bar.wfull[i]);
          if (left == 0) {
            TreeSplit sp = {};
            if (!SHARED && off + nt < tiles) {
              const int start = aux.end - nt - off;  // the list's number of the unit's first tile
              sp.rows = rows;
              sp.kvh = kvh;
              sp.tok = s.c0 + (block << ul);
              sp.first = start / per;
              sp.n_rec = (start + tiles - 1) / per - sp.first + 1;
            }
            if (!SHARED) p.rec.split[blockIdx.x] = sp;
          }
        }
        __syncwarp();
        bool ok = true;
        const int q_end = qtiles + (rows <= TT ? 1 : 2);
        for (int j = 0; ok && qtiles < q_end; j++, qtiles++) {
          const int slot = qtiles & 1;
          ok = __all_sync(FULL_MASK, mbar_wait(&bar.qempty[slot], ((qtiles >> 1) & 1) ^ 1, kv.err));
          if (ok && leader) {
            mbar_arrive_expect_tx(&bar.qfull[slot], S::TILE);
#pragma unroll
            for (int sg = 0; sg < S::SEGS; sg++)
              tma_load_4d(base + (S::SLOTS + slot) * S::TILE + sg * S::SEG, &qmap, 0, sg, kvh << gl,
                          s.c0 + (block << ul) + (j << (7 - gl)), &bar.qfull[slot]);
          }
          __syncwarp();
        }
        if (!ok || left == 0) break;
        loads += 2 * nt;
        off = 0;
        if (++block == s.blocks) {
          block = 0;
          if (++kvh == kv.Hkv) {
            kvh = 0;
            if (!next_item()) break;
          }
        }
      }
      for (int qt = max(0, qtiles - 2); qt < qtiles; qt++)
        mbar_wait(&bar.qfull[qt & 1], (qt >> 1) & 1, kv.err);
    } else if (warp != 9) {
      // -------- K and V producers: a column segment each, or every second box -------- //
      const bool leader = elect_one();
      auto base_key = [](const TcWork& w) { return SHARED ? w.base : 0; };
      const int half = warp == 8 ? 0 : 1;
      const int br_log2 = p.box_log2, br = 1 << br_log2, per_log2 = 7 - br_log2;
      int last = -1;
      TcWork w;
      bool ok = take(w);
      while (ok) {
        // Rows of the cache's boxes, 32 boxes at a time, one a lane; the page of
        // the next 32 is read while these are used. V is up to two tiles behind K.
        auto page_of = [&](int box) -> int {
          const int key = box << br_log2;
          if (kv.block_table == nullptr || key >= w.t) return 0;
          return kv.block_table[(long long)w.b * kv.max_blocks + (base_key(w) + key) / kv.block_size];
        };
        auto row_of = [&](int page, int box) -> int {
          const int key = base_key(w) + (box << br_log2);
          if (kv.block_table == nullptr) return (w.b * kv.Hkv + w.kvh) * kv.t_max + key;
          if ((unsigned)page >= (unsigned)kv.num_blocks) {  // the softmax masks its keys
            raise_error(kv.err, PRHS_DEV_BAD_BLOCK);
            *reinterpret_cast<volatile int*>(&aux.bad_page) = 1;
            __threadfence_block();
            page = 0;
          }
          return (page * kv.Hkv + w.kvh) * kv.block_size + key % kv.block_size;
        };
        TcRing<S::SLOTS> at(w.loads);
        int win = (w.tile0 << per_log2) - 32, rows = 0, behind = 0, ahead = 0;
        if (w.tile0 < w.cache_tiles) ahead = page_of(win + 32 + lane);
        for (int l = 0; ok && l < 2 * w.nt; l++) {
          bool is_v;
          const int tile = w.tile0 + w.load_tile(l, is_v);
          const bool fresh = tile >= w.cache_tiles;
          const int key0 = (fresh ? tile - w.cache_tiles : tile) * TT;
          const int valid = min(TT, (fresh ? w.n : w.t) - key0);
          const int step_log2 = fresh || valid < TT ? 4 : br_log2;  // rows of a box
          const int boxes = (valid + (1 << step_log2) - 1) >> step_log2;
          if (!fresh && (tile << per_log2) >= win + 32) {
            win += 32;
            behind = rows;
            rows = row_of(ahead, win + lane);
            ahead = page_of(win + 32 + lane);
          }
          const int slot = at.slot;
          ok = __all_sync(FULL_MASK, mbar_wait(&bar.empty[slot], at.phase ^ 1, kv.err));
          if (!ok) break;
          at.step(1);
          // this warp's boxes: all of segment `half` (d = 128), or boxes half, half + 2, ...
          const int mine = S::SEGS == 2 ? boxes : (boxes + 1 - half) >> 1;
          if (leader) mbar_arrive_expect_tx(&bar.full[slot], (mine << step_log2) * 128);
          const CUtensorMap* map = fresh ? (is_v ? &vnmap : &knmap)
                                         : step_log2 == br_log2 ? (is_v ? &vmap : &kmap) : (is_v ? &vtail : &ktail);
          const uint32_t dst = base + slot * S::TILE;
          // the boxes' rows first, then all copies from one thread: a copy takes it
          // about 40 clocks that way, over 100 with a shuffle between two
          int z[8];
          const int from = (tile << per_log2) - win;
#pragma unroll
          for (int x = 0; x < 8; x++) {
            const int key = x << step_log2;  // within the tile
            const int bx = from + (key >> br_log2);
            z[x] = __shfl_sync(FULL_MASK, bx < 0 ? behind : rows, bx & 31) + (key & (br - 1));
            if (fresh) z[x] = w.kvh;
          }
          if (leader) {
            int y = fresh ? w.c0 + key0 : 0;
            const int y_step = fresh ? 16 : 0;
            uint32_t to = dst + (S::SEGS == 2 ? half * S::SEG : 0);
            const uint32_t to_step = 128u << step_log2;
#pragma unroll
            for (int x = 0; x < 8; x++) {
              if (x >= boxes) break;
              if (S::SEGS == 2 || (x & 1) == half) tma_load_4d(to, map, 0, S::SEGS == 2 ? half : 0, z[x], y, &bar.full[slot]);
              to += to_step;
              y += y_step;
            }
          }
          __syncwarp();
          last = w.loads + l;
        }
        if (!ok || w.last) break;
        ok = take(w);
      }
      // nothing may still be in flight when the CTA ends
      for (int g = max(0, last - S::SLOTS + 1); g <= last; g++)
        mbar_wait(&bar.full[g % S::SLOTS], (g / S::SLOTS) & 1, kv.err);
    } else {
      // ---------------------------- matrix issuer ---------------------------- //
      constexpr uint32_t QK = instr_desc(TT, false), PV = instr_desc(D, true);
      if (elect_one()) {
        uint32_t np = 0;  // parities of the softmax results taken, a bit a stream
        bool ok = true;
        for (int k = 0; ok; k++) {
          const int wi = k & (TC_WORKS - 1);
          if (!mbar_wait(&bar.wfull[wi], (k / TC_WORKS) & 1, kv.err)) break;
          const int rows = aux.work[wi].rows, nt = aux.work[wi].nt, loads = aux.work[wi].loads;
          const int qtiles = aux.work[wi].qtiles, last = aux.work[wi].last;
          mbar_arrive(&bar.wempty[wi]);
          const bool single = rows <= TT;
          const int steps = single ? nt : 2 * nt;
          // places of the next K to use, the next K to release, the next V
          TcRing<S::SLOTS> kr(loads), kd(loads), vr(loads + (single ? min(2, 2 * nt - 1) : 1));
          auto issue_qk = [&](int y) {  // S of step y; its K tile is loaded
            const int st = y & 1, qslot = (qtiles + (single ? 0 : st)) & 1;
            const uint64_t qd = smem_desc(base + (S::SLOTS + qslot) * S::TILE, 16, 1024);
            const uint64_t kdesc = smem_desc(base + kr.slot * S::TILE, 16, 1024);
#pragma unroll
            for (int j = 0; j < D / 16; j++) {
              const uint32_t off = ((j / 4) * S::SEG + (j % 4) * 32) >> 4;
              mma_ss(tmem + st * TT, qd + off, kdesc + off, QK, j > 0);
            }
            tc_commit(&bar.sfull[st]);
            if (single) tc_commit(&bar.empty[kr.slot]);
            if (single || st == 1) kr.step(single && y == 0 ? 1 : 2);
            if (single ? y == steps - 1 : y >= steps - 2) tc_commit(&bar.qempty[qslot]);
          };
          ok = mbar_wait(&bar.qfull[qtiles & 1], (qtiles >> 1) & 1, kv.err);
          // step x of the loop: O of step x, then S of step x + 2 in the same stream; with
          // two row tiles (bound by the products) every load they need is waited for
          // before the softmax, so that nothing comes between the two products, and K is
          // released behind the next product: this thread's polls of a barrier queue
          // behind what it has issued, releases included (495 -> 404 -> 398 us). Steps -2
          // and -1 are S of steps 0 and 1.
          for (int x = -2; ok && x < steps; x++) {
            const bool more = x + 2 < steps;
            if (more && !single && (x & 1) == 0) ok = ok && mbar_wait(&bar.full[kr.slot], kr.phase, kv.err);
            if (x == -1 && !single) ok = ok && mbar_wait(&bar.qfull[(qtiles + 1) & 1], ((qtiles + 1) >> 1) & 1, kv.err);
            if (x >= 0) {
              const int st = x & 1;
              if (single || st == 0) ok = ok && mbar_wait(&bar.full[vr.slot], vr.phase, kv.err);
              const uint64_t vd = smem_desc(base + vr.slot * S::TILE, S::SEG, 1024);
              // the first half of P's keys while the softmax computes the second
#pragma unroll
              for (int h = 0; h < 2; h++) {
                ok = ok && mbar_wait(&bar.pfull[st][h], (np >> st) & 1, kv.err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int j = h * 4; j < h * 4 + 4; j++)
                  mma_ts(tmem + 2 * TT + st * D, tmem + st * TT + j * 8, vd + (j * 2048 >> 4), PV, x > 1 || j > 0);
              }
              if (!ok) break;
              np ^= 1u << st;
            }
            if (!ok) break;
            if (!single && x >= 0 && (x & 1) == 0) {  // K of the tile whose S were issued before this product
              tc_commit(&bar.empty[kd.slot]);
              kd.step(2);
            }
            if (x >= 0 && (single || (x & 1))) {
              tc_commit(&bar.empty[vr.slot]);
              vr.step(single && x == steps - 2 ? 1 : 2);
            }
            // (with a tile to itself a step gives back V before it waits for the next K)
            if (more && single) ok = mbar_wait(&bar.full[kr.slot], kr.phase, kv.err);
            if (!ok) break;
            if (more) issue_qk(x + 2);
            else if (x >= 0) tc_commit(&bar.ofull[x & 1]);
          }
          if (last) break;
        }
        // nothing may still be in flight when tensor memory is freed
        tc_commit(&bar.done);
        mbar_wait(&bar.done, 0, kv.err);
      }
      __syncwarp();
    }
    if constexpr (SHARED) {
      // the sequences for the few rows' list, asked for before the barrier
      constexpr int OTHERS = TC_THREADS - 2 * TT, PER = FEW_TABLE / OTHERS;
      const bool noted = kv.B <= FEW_TABLE && !tile_cta;
      TreeItem x[PER];
#pragma unroll
      for (int i = 0; i < PER; i++)
        if (noted && tid - 2 * TT + i * OTHERS < kv.B) x[i] = tree_item<true>(a, 2 * (tid - 2 * TT + i * OTHERS) + 1, true);
      tiles_done([&] {
#pragma unroll
        for (int i = 0; i < PER; i++)
          if (noted && tid - 2 * TT + i * OTHERS < kv.B)
            few_note(reinterpret_cast<int*>(data + FEW_WARPS * few_warp_bytes(D)), tid - 2 * TT + i * OTHERS, x[i]);
      });
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TC_REGS_SOFTMAX));
    // ------------------------------- softmax ------------------------------- //
    const int st = warp >> 2;                     // stream
    const int row = (warp & 3) * 32 + lane;       // its row, and the V row it may zero
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + st * TT;
    const bool flip = a.scale < 0.f;
    // a zero scale keeps masked logits at -inf (0 * inf is not a number)
    const float sc = fmaxf(fabsf(a.scale) * TC_LOG2E, 1e-30f);
    bool dead = false;
    int ns = 0, no = 0;  // S tiles and O tiles taken
    TcWork w;
    for (bool more = some && take(w); more; more = !w.last && take(w)) {
      const bool single = w.single();
      const int steps = w.steps();
      const int ur = (single ? 0 : st * TT) + row;  // row of the unit
      const int tok = w.tok0 + (ur >> gl);          // token of the sequence
      const int tok_c = min(tok, w.n - 1);
      const int tok_first = w.tok0 + (single ? 0 : st << (7 - gl));
      // a warp without rows computes nothing: rows do not mix, so what its part of
      // S and O holds reaches no result
      const bool idle = (single ? 0 : st * TT) + (warp & 3) * 32 >= w.rows;
      float m = -INFINITY, l = 0.f;
      for (int x = st; x < steps; x += 2) {
        const int i = single ? x : x >> 1, tile = w.tile0 + i;
        const bool fresh = tile >= w.cache_tiles;
        const int key0 = (fresh ? tile - w.cache_tiles : tile) * TT;
        const int valid = (fresh ? w.n : w.t) - key0;   // keys of the tile, at least 1
        if (!dead) dead = !__all_sync(FULL_MASK, mbar_wait(&bar.sfull[st], ns & 1, kv.err));
        ns++;
        if (dead) continue;
        tc_fence_after();
        // keys that exist, the same for every row (their V rows are zeroed below)
        uint32_t have[4] = {~0u, ~0u, ~0u, ~0u};
        const bool bad = !fresh && kv.block_table != nullptr && *reinterpret_cast<volatile int*>(&aux.bad_page) != 0;
        const bool cut = valid < TT || bad;
        if (cut) {
          uint32_t ok16 = 0xff;  // 16-key groups on pages of the pool
          if (bad) {
            const int k = (lane & 7) * 16;
            ok16 = __ballot_sync(FULL_MASK, k >= valid || kv_row(kv, w.b, w.kvh, (SHARED ? w.base : 0) + key0 + k) >= 0) & 0xff;
          }
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int k = valid - c * 32;
            have[c] = k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1;
            have[c] &= ((ok16 >> (2 * c)) & 1 ? 0xffffu : 0u) | ((ok16 >> (2 * c + 1)) & 1 ? 0xffff0000u : 0u);
          }
          // V rows of keys that do not exist hold whatever was there, possibly not
          // finite, and 0 * inf would reach every row: they are set to 0 (each row from
          // another piece on, since the rows' equal pieces share their banks)
          const int g = w.load_v(i), slot = g % S::SLOTS;
          dead = !__all_sync(FULL_MASK, mbar_wait(&bar.full[slot], (g / S::SLOTS) & 1, kv.err));
          const uint32_t hw = row < 32 ? have[0] : row < 64 ? have[1] : row < 96 ? have[2] : have[3];
          if (!dead && !((hw >> (row & 31)) & 1u)) {
#pragma unroll
            for (int c = 0; c < 8 * S::SEGS; c++)
              *reinterpret_cast<uint4*>(data + slot * S::TILE + (c / 8) * S::SEG + row * 128 + ((c ^ row) % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (!idle) {
          uint32_t r[TT];
          tmem_ld_row(r, s_addr);
          tc_wait_ld();
          if (flip) {
#pragma unroll
            for (int e = 0; e < TT; e++) r[e] ^= 0x80000000u;
          }
          const bool by_row = fresh && (a.mask != nullptr || key0 + TT - 1 > tok_first);
          if (cut || by_row) {
            uint32_t see[4] = {have[0], have[1], have[2], have[3]};
            if (by_row) {
              if (a.mask != nullptr) {
                const uint4 t4 = reinterpret_cast<const uint4*>(a.mask)[w.c0 + tok_c];
                see[0] &= t4.x;
                see[1] &= t4.y;
                see[2] &= t4.z;
                see[3] &= t4.w;
              } else {
#pragma unroll
                for (int c = 0; c < 4; c++) {
                  const int k = tok_c + 1 - key0 - c * 32;
                  see[c] &= k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1;
                }
              }
            }
#pragma unroll
            for (int e = 0; e < TT; e++)
              if (!((see[e / 32] >> (e % 32)) & 1u)) r[e] = 0xff800000u;
          }
          float mx4[4];
#pragma unroll
          for (int c = 0; c < 4; c++) mx4[c] = fmaxf(__uint_as_float(r[c]), __uint_as_float(r[c + 4]));
#pragma unroll
          for (int e = 8; e < TT; e += 8)
#pragma unroll
            for (int c = 0; c < 4; c++) mx4[c] = max3(mx4[c], __uint_as_float(r[e + c]), __uint_as_float(r[e + c + 4]));
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
          const bool grow = mx > m + RESCALE_LOG2 || (m == -INFINITY && mx > m);
          if (__any_sync(FULL_MASK, grow)) {
            const float corr = grow ? ex2(m - mx) : 1.f;
            if (grow) m = mx;
            l *= corr;
            if (x >= 2) {  // O holds the stream's earlier tiles: S of this step came after them
#pragma unroll 1
              for (int c = 0; c < D / 32; c++) {
                uint32_t o[32];
                const uint32_t oa = tmem + lanes + 2 * TT + st * D + c * 32;
                tmem_ld32(o, oa);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st32(oa, o);
              }
            }
          }
          const float mm = m == -INFINITY ? 0.f : -m;
          const uint64_t sc2 = f2(sc, sc), mm2 = f2(mm, mm);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < 2; h++) {
            uint32_t q[32];
#pragma unroll
            for (int e = 0; e < 32; e++) {
              float v0, v1;
              unf2(fma2(f2(__uint_as_float(r[h * 64 + 2 * e]), __uint_as_float(r[h * 64 + 2 * e + 1])), sc2, mm2), v0, v1);
              v0 = ex2(v0);
              v1 = ex2(v1);
              sum[e & 1] = add2(sum[e & 1], f2(v0, v1));
              q[e] = pack2(v0, v1);
            }
            tmem_st32(s_addr + h * 32, q);
            if (h == 0) {
              tc_wait_st();
              tc_fence_before();
              mbar_arrive(&bar.pfull[st][0]);
            }
          }
          float s0, s1;
          unf2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        } else {
          tc_fence_before();
          mbar_arrive(&bar.pfull[st][0]);
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bar.pfull[st][1]);
      }

      // ---- the unit's end in this run: result or partial record ----
      const bool both = single;
      if (steps > st) {
        if (!dead) dead = !__all_sync(FULL_MASK, mbar_wait(&bar.ofull[st], no & 1, kv.err));
        no++;
      }
      float w0 = 1.f, w1 = 0.f, M = m, L = l;
      if (both) {
        aux.m[st][row] = m;
        aux.l[st][row] = l;
        tc_fence_before();
        softmax_meet(false);
        const float m0 = aux.m[0][row], m1 = aux.m[1][row];
        M = fmaxf(m0, m1);
        w0 = m0 == -INFINITY ? 0.f : ex2(m0 - M);
        w1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
        L = w0 * aux.l[0][row] + w1 * aux.l[1][row];
      }
      tc_fence_after();
      const bool live = ur < w.rows && !dead;
      const bool result = w.whole && (!SHARED || w.part == 0);
      if (result) {
        const float inv = tree_inv(L);
        w0 *= inv;
        w1 *= inv;
      }
      const int rec = 2 * blockIdx.x + (w.tile0 == 0 ? 1 : 0);
      auto out_row = [&](int r) {
        return (long long)(w.c0 + w.tok0 + (r >> gl)) * kv.Hq + (w.kvh << gl) + (r & ((1 << gl) - 1));
      };
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
      // Four lanes exchange their rows' 16-byte pieces, so that a store covers 64 bytes
      // of eight rows, not 16 of 32: it is issued line by line (causal chunks 398 -> 387
      // us). With few rows the exchange costs more than it saves.
      const bool quads = w.rows > QUAD_ROWS;
      // both warpgroups of a shared unit write half the columns each
      const int c_lo = both ? st * (D / 64) : 0, c_hi = both ? c_lo + D / 64 : D / 32;
      const bool two = both && steps > 1;
#pragma unroll 1
      for (int c = c_lo; c < c_hi; c++) {
        uint32_t o[32], o1[32];
        tmem_ld32(o, tmem + lanes + 2 * TT + (both ? 0 : st * D) + c * 32);
        if (two) tmem_ld32(o1, tmem + lanes + 2 * TT + D + c * 32);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e++) {
          const float v = __uint_as_float(o[e]) * w0;
          o[e] = __float_as_uint(two ? fmaf(__uint_as_float(o1[e]), w1, v) : v);
        }
        if (result) {
          uint32_t v[4][4];
#pragma unroll
          for (int e = 0; e < 4; e++)
#pragma unroll
            for (int k = 0; k < 4; k++)
              v[e][k] = pack2(__uint_as_float(o[8 * e + 2 * k]), __uint_as_float(o[8 * e + 2 * k + 1]));
          if (!quads) {
            uint4* dst = reinterpret_cast<uint4*>(out + out_row(ur) * D + c * 32);
            if (live)
#pragma unroll
              for (int e = 0; e < 4; e++) dst[e] = make_uint4(v[e][0], v[e][1], v[e][2], v[e][3]);
            continue;
          }
          quad_swap<1>(v[0], v[1]);
          quad_swap<1>(v[2], v[3]);
          quad_swap<2>(v[0], v[2]);
          quad_swap<2>(v[1], v[3]);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int r = (ur & ~3) + e;
            if (r < w.rows && !dead)
              *reinterpret_cast<uint4*>(out + out_row(r) * D + c * 32 + (lane & 3) * 8) =
                  make_uint4(v[e][0], v[e][1], v[e][2], v[e][3]);
          }
        } else if (SHARED && w.whole) {
          float4* dst = part_at<__nv_bfloat16, D>(a, w.part, w.c0 + tok, w.kvh, ur & ((1 << gl) - 1), c * 8, gl);
          if (live)
#pragma unroll
            for (int e = 0; e < 8; e++)
              *reinterpret_cast<uint4*>(dst + e * ((long long)a.T << gl)) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else if (live) {
          uint4* dst = reinterpret_cast<uint4*>(p.rec.o) + (rec * (D / 4) + c * 8) * p.rec.rows_max + ur;
#pragma unroll
          for (int e = 0; e < 8; e++)
            dst[e * p.rec.rows_max] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (live && (!both || st == 0)) {
        if (result) a.lse[out_row(ur)] = tree_lse(M, L);
        else if (SHARED && w.whole) a.part_ml[part_row<__nv_bfloat16>(a, w.part, w.c0 + tok, w.kvh, ur & ((1 << gl) - 1), gl)] = make_float2(M, L);
        else p.rec.ml[rec * p.rec.rows_max + ur] = make_float2(M, L);
        if (SHARED && w.tile0 == 0)
          a.where[part_row<__nv_bfloat16>(a, w.part == 1 ? 1 : 2, w.c0 + tok, w.kvh, ur & ((1 << gl) - 1), gl)] =
              make_int2(w.first, w.cuts);
      }
      tc_fence_before();
      if (both && !w.last) softmax_meet(false);  // both outputs and the row states are read (the last: below)
    }
    while (some && !softmax_meet(true)) {
    }
    if constexpr (SHARED) {
      tiles_done([] {});
      if (!tile_cta)
        few_role<D, NT1>(a, ktail, vtail, knmap, vnmap, tc_smem, aux.few, per_t, all_steps, (int)blockIdx.x - ctas,
                         (int)gridDim.x - ctas, gl);
    }
  }
  if constexpr (!SHARED) tiles_done([] {});
}

// -------------------------------------------------------------------------- //
// host side
// -------------------------------------------------------------------------- //
inline int tc_rows_max(const KVView& kv, int max_new) {
  const long long r = (long long)max_new * (kv.Hq / kv.Hkv);
  return (int)(r < UNIT_ROWS ? r : UNIT_ROWS);
}

// Rows of a TMA box of the cache's whole tiles: the most that a page holds whole
// boxes of. The tile at a cache's end is copied in boxes of 16.
inline int tc_box_log2(const KVView& kv) {
  int r = 4;
  while ((1 << r) < TT && (kv.block_table == nullptr || kv.block_size % (2 << r) == 0)) r++;
  return r;
}

template <int D, int NT>
static cudaError_t tc_go(const TcLaunch& p, const CUtensorMap* maps, int sms, cudaStream_t st) {
  using S = TcShape<D>;
  auto k = tree_tc_kernel<D, NT>;
  // the register shares need what the kernel was compiled with, asked once
  static const int regs = [k] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, k) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < TC_REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  static int smem_set[SMEM_DEVICES];
  cudaError_t e = allow_smem(k, S::SMEM, smem_set);
  if (e != cudaSuccess) return e;
  // (with shared keys always early: calls back to back 127.7 -> 125.0 us for 913 prompt tokens, 115 -> 113.3
  // for 131072 keys)
  e = launch_pdl(k, dim3(sms), dim3(TC_THREADS), S::SMEM, st, NT > 0 || p.a.kv.pdl, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5],
                 maps[6], p);
  if (e == cudaSuccess) abi_count_launch();
  return e;
}

// The launch's arguments and descriptors: q; cache K and V; their partial tiles; new K and V.
inline prhs_status tc_prepare(const TreeLaunch& a, int sms, void* ws, TcLaunch* launch, CUtensorMap* maps) {
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv;
  TcLaunch& p = *launch;
  p.a = a;
  p.rec = tree_records(ws, G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3, sms, tc_rows_max(kv, tree_most_new(a)));
  p.box_log2 = tc_box_log2(kv);

  const uint64_t d = kv.d, row = d * 2, segs = d / 64;
  const uint64_t cache_rows = kv.block_table != nullptr ? (uint64_t)kv.num_blocks * kv.Hkv * kv.block_size
                                                        : (uint64_t)kv.B * kv.Hkv * kv.t_max;
  const uint64_t qd[4] = {64, segs, (uint64_t)kv.Hq, (uint64_t)a.T}, qs[3] = {128, row, row * kv.Hq};
  const uint32_t qb[4] = {64, 1, (uint32_t)G, (uint32_t)(TT / G)};
  // the cache's rows with a fourth dimension of one, so that one copy serves both
  const uint64_t cd[4] = {64, segs, cache_rows, 1}, cs[3] = {128, row, row * cache_rows};
  const uint32_t cb[4] = {64, 1, 1u << p.box_log2, 1}, tb[4] = {64, 1, 16, 1};
  const uint64_t nd[4] = {64, segs, (uint64_t)kv.Hkv, (uint64_t)a.T};
  const uint64_t ks[3] = {128, row, (uint64_t)a.ks * 2}, vs[3] = {128, row, (uint64_t)a.vs * 2};
  const uint32_t nb[4] = {64, 1, 1, 16};
  prhs_status s;
  if ((s = abi_encode_bf16(&maps[0], a.q, 4, qd, qs, qb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[1], kv.k, 4, cd, cs, cb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[2], kv.v, 4, cd, cs, cb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[3], kv.k, 4, cd, cs, tb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[4], kv.v, 4, cd, cs, tb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[5], a.k_new, 4, nd, ks, nb)) != PRHS_OK) return s;
  if ((s = abi_encode_bf16(&maps[6], a.v_new, 4, nd, vs, nb)) != PRHS_OK) return s;
  return PRHS_OK;
}

}  // namespace prhs
