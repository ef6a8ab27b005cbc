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
};
// fp32: two launches, the first counted by the callee; ws holds
// tree_workspace(kv, max_new, sms) bytes.
cudaError_t launch_tree(const TreeLaunch& a, int sms, void* ws, cudaStream_t s);
size_t tree_workspace(const KVView& kv, int max_new, int sms);
// bf16: two launches, the first counted by the callee; *err is the launches'
// result when the descriptors could be made. Workspace bytes of a call.
prhs_status launch_tree_tc(const TreeLaunch& a, int sms, void* ws, cudaStream_t s, cudaError_t* err);
size_t tree_tc_workspace(const KVView& kv, int max_new, int sms);

// TMA descriptor of a bf16 tensor with the 128-byte swizzle (dims and box
// innermost first, strides in bytes from dimension 1 on).
prhs_status abi_encode_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                            const uint64_t* strides, const uint32_t* box);

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

// Row of KV head 0 of cache slot `slot`, and the rows from one head to the
// next: slots count pages * block_size + row (contiguous: sequence * t_max + row).
__device__ __forceinline__ long long slot_row(const KVView& kv, int slot, int* head_rows) {
  const int per = kv.block_table != nullptr ? kv.block_size : kv.t_max;
  *head_rows = per;
  return (long long)(slot / per) * kv.Hkv * per + slot % per;
}

}  // namespace prhs
