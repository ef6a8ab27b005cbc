// Internal launch interface of the token-batch operators (several new tokens
// per sequence in one step).
#pragma once

#include "kernels.h"

namespace prhs {

struct PlanLaunch {
  KVView kv;
  const int32_t* n_new;
  int T;
  const int32_t* parents;
  const int32_t* free_pages;
  int n_free;
  const int32_t* free_head;
  const int32_t* n_pages;
  int32_t* block_table;  // null: contiguous cache
  int32_t* cu_new;
  int32_t* positions;
  int32_t* slots;
  uint32_t* tree_mask;
  int32_t* free_head_out;
  int32_t* n_pages_out;
};
cudaError_t launch_plan(const PlanLaunch& a, cudaStream_t s);

struct RopeLaunch {
  KVView kv;
  int T;
  int rot_dim;
  int interleaved;
  const uint64_t* turns;
  float mscale;
  const int32_t* positions;
  const int32_t* slots;  // null: the cache is not written
  const void* q;
  const void* k;
  const void* v;
  long long qs, ks, vs;  // token strides, elements
  void* q_out;
  void* k_out;           // nullable
};
cudaError_t launch_rope(const RopeLaunch& a, int sms, cudaStream_t s);

struct CommitLaunch {
  KVView kv;
  int T;
  const int32_t* cu_new;
  const int32_t* slots;  // null: the block table alone says where the rows go
  const int32_t* accept_idx;
  int accept_cap;
  const int32_t* accept_n;
  const void* k_new;     // both null: lengths only
  const void* v_new;
  long long ks, vs;
  int32_t* new_lens;
};
cudaError_t launch_commit(const CommitLaunch& a, int sms, cudaStream_t s);

// What a launch with shared keys takes of a batch: the groups' shared keys, the sequences' others, or both.
enum : int { TREE_BOTH, TREE_GROUPS, TREE_OWN };
struct TreeLaunch {
  KVView kv;
  const void* q;
  const void* k_new;
  const void* v_new;
  long long ks, vs;
  float scale;
  int T;
  const int32_t* cu_new;
  int max_new;
  const uint32_t* mask;  // null: causal
  void* out;             // the cache's element type
  float* lse;
  // rows that share leading keys (shared_attn; null: none do), and the partial
  // states of tokens that have two: against the shared keys, against the others
  // (fp32: [2][T * Hq][d] and [2][T * Hq]; bf16: [2][Hkv][d / 4][T * G] of four columns
  // and [2][Hkv][T * G])
  const int4* shared;
  int items;        // (fp32) TREE_BOTH, ..
  float* part_o;    // against the state's maximum
  float2* part_ml;  // maximum (base 2) and sum
  int* part_ok;     // 0: the offsets step back, there are no states
  // bf16: which CTAs or warps have pieces of a row's states, [2][Hkv][T * G]: the first, how many
  int2* where;
  // and the few rows' part of the launch (few_item)
  int few_rows;      // query rows of a unit
  int few_warps;     // warps that it may have
  void* few_states;  // [2 few_warps] states of units that several warps share, two a warp
};
// Whether a sequence's own t keys with its n tokens go to that part: few keys, and one
// unit of few_rows query rows a KV head. Two units read the keys twice: 386 sequences of 10
// tokens, two heads a KV head, up to 1360 keys, take 201 us there and 123 as tiles, 16 of 17 to
// 20 rows on up to 16K keys 679 and 351; only next to no own keys are better off (44 sequences
// of 9 tokens that share all but 6 keys: 41 and 64), and a few such among longer ones hold the
// others up (128 sequences of up to 3K keys 166 us, 187 to 221 with those below 256 there).
// (At most 16384 rows of KV heads: 2^26 steps.)
constexpr int FEW_KEYS = 32768;
__device__ __forceinline__ bool few_item(const TreeLaunch& a, int n, int t) {
  return t + n <= FEW_KEYS && (long long)n * (a.kv.Hq / a.kv.Hkv) <= a.few_rows;
}
// fp32: two launches (three with shared keys), all but the last counted by the callee; ws
// holds tree_workspace(kv, max_new, shared, sms) bytes.
cudaError_t launch_tree(const TreeLaunch& a, int sms, void* ws, cudaStream_t s);
size_t tree_workspace(const KVView& kv, int max_new, bool shared, int sms);  // (max_new: tree_most_new)
// bf16: two launches, the first counted by the callee; *err is the launches'
// result when the descriptors could be made. Workspace bytes of a call.
prhs_status launch_tree_tc(const TreeLaunch& a, int sms, void* ws, cudaStream_t s, cudaError_t* err);
size_t tree_tc_workspace(const KVView& kv, int max_new, int sms);

// With shared keys: fp32 launch_tree, then the join; bf16 one launch (counted) and the
// join. rec: (bf16) the partial states of the launch's CTAs, one an SM.
struct TreeRecords;
prhs_status launch_shared_tc(const TreeLaunch& a, int sms, void* ws, cudaStream_t s, cudaError_t* err);
cudaError_t launch_shared_join(const TreeLaunch& a, const TreeRecords& rec, int sms, cudaStream_t s);
void few_shape(TreeLaunch* a, int sms);
size_t few_state_bytes(const KVView& kv, int sms);
size_t shared_where_bytes(const KVView& kv, int T);
// The most tokens that a unit's rows may come from.
inline int tree_most_new(const TreeLaunch& a) { return a.shared != nullptr ? a.T : a.max_new; }

// TMA descriptor of a bf16 tensor with the 128-byte swizzle (dims and box
// innermost first, strides in bytes from dimension 1 on).
prhs_status abi_encode_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                            const uint64_t* strides, const uint32_t* box);

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
// One lane of a converged warp. (A lane chosen by its number compiles to a loop
// over the lanes around every instruction that takes uniform operands.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Two fp32 numbers in one 64-bit register pair, and operations on both.
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Tokens [c0, c0 + n) of sequence b; none (flagged) when cu_new is not
// ascending within [0, T] or the sequence has more than max_new.
__device__ __forceinline__ int seq_tokens(const int32_t* cu_new, int b, int T, int max_new,
                                          unsigned* err, int* c0) {
  const int lo = cu_new[b], hi = cu_new[b + 1];
  *c0 = lo;
  if (lo < 0 || hi < lo || hi > T || hi - lo > max_new) {
    raise_error(err, PRHS_DEV_BAD_LEN);
    return 0;
  }
  return hi - lo;
}

// Leading keys that sequence b, of t cached keys, shares with its group, 0 if it is
// alone. An entry that does not fit (other than its group's first row's, a length below
// the shared keys) is flagged and read as alone. Whole pages only.
__device__ __forceinline__ int shared_keys(const KVView& kv, const int4* shared, int b, int t) {
  const int4 s = shared[b];
  if (s.x == b && (s.y <= 1 || s.z == 0)) return 0;
  bool ok = s.x >= 0 && s.x <= b;
  const int4 g = ok ? shared[s.x] : s;
  const int keys = kv.block_table != nullptr ? g.z / kv.block_size * kv.block_size : g.z;
  ok = ok && g.x == s.x && g.y == s.y && g.z == s.z && b - s.x < g.y && keys >= 0 && keys <= t && keys <= kv.seq_lens[s.x];
  if (ok) return keys;
  raise_error(kv.err, PRHS_DEV_BAD_INDEX);
  return 0;
}

// Groups are apart, so that all of them together have no more than T tokens. More are
// flagged and nothing is attended: work and counts would be without bound.
__device__ __forceinline__ bool groups_overlap(const TreeLaunch& a, long long tokens, int tid) {
  if (tokens > a.T && tid == 0) raise_error(a.kv.err, PRHS_DEV_BAD_INDEX);
  return tokens > a.T;
}

// What the rows of a launch attend, item by item: sequence b's tokens over its own
// cached keys from `base` on and over each other; or, for rows that share leading
// keys, an item in front of that of a group's first row: all its rows' tokens over
// the shared keys of that row. (Items 2 b and 2 b + 1; without sharing, item b.) Not
// those of the few rows' part, unless `all`.
struct TreeItem {
  int b, base, t;  // row of the cache; its first key here, keys
  int c0, n;       // tokens
  int part;        // the state is the result (0), the one against the shared keys (1) or the others (2)
};
template <bool SHARED>
__device__ __forceinline__ TreeItem tree_item(const TreeLaunch& a, int e, bool all = false) {
  TreeItem x;
  x.b = SHARED ? e >> 1 : e;
  x.base = x.part = 0;
  x.t = seq_len(a.kv, x.b);
  if constexpr (SHARED) {
    const int keys = shared_keys(a.kv, a.shared, x.b, x.t);
    if (!(e & 1)) {
      const int4 s = a.shared[x.b];
      x.c0 = x.n = 0;
      x.part = 1;
      x.t = keys;
      if (s.x != x.b || keys == 0) return x;
      // (rows that are not within [0, T] are flagged by their own items)
      x.c0 = max(0, a.cu_new[x.b]);
      x.n = max(0, min(a.T, a.cu_new[min((long long)a.kv.B, (long long)x.b + s.y)]) - x.c0);
      return x;
    }
    if (keys > 0) {
      x.base = keys;
      x.t -= keys;
      x.part = 2;
    }
  }
  x.n = seq_tokens(a.cu_new, x.b, a.T, a.max_new, a.kv.err, &x.c0);
  if (SHARED && !all && few_item(a, x.n, x.t)) x.n = 0;
  return x;
}

// Row of KV head 0 of cache slot `slot`, and the rows from one head to the
// next: slots count pages * block_size + row (contiguous: sequence * t_max + row).
__device__ __forceinline__ long long slot_row(const KVView& kv, int slot, int* head_rows) {
  const int per = kv.block_table != nullptr ? kv.block_size : kv.t_max;
  *head_rows = per;
  return (long long)(slot / per) * kv.Hkv * per + slot % per;
}

}  // namespace prhs
