// C ABI of the token-batch operators: argument checks and launches. The
// contract of every entry point is in include/prhs.h.
#include <cmath>

#include "tree_join.cuh"

using namespace prhs;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t esize(const prhs_kv& kv) { return kv.dtype == PRHS_BF16 ? 2 : 4; }

// A token stride in elements: at least the row, whole 16-byte pieces.
bool stride_ok(const prhs_kv& kv, long long stride, int heads) {
  return stride >= (long long)heads * kv.d && stride % (long long)(16 / esize(kv)) == 0 &&
         stride < (1ll << 38);  // bytes below the 2^40 of a TMA stride
}

prhs_status launched(cudaError_t e) {
  if (e == cudaSuccess) {
    abi_count_launch();
    return PRHS_OK;
  }
  return abi_fail(PRHS_ECUDA, cudaGetErrorString(e));
}

size_t tree_ws_bytes(const KVView& kv, int max_new, bool shared, int sms) {
  return kv.dtype == PRHS_BF16 ? tree_tc_workspace(kv, max_new, sms) : tree_workspace(kv, max_new, shared, sms);
}

// Checks shared by every entry point: descriptor, device, token count.
prhs_status begin(const prhs_kv* kv, int T, KVView* view, int* sms) {
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (T < 0) return abi_fail(PRHS_EINVAL, "T must be >= 0");
  // 32-bit task and row counts of the kernels
  if ((long long)T * (kv->Hq + 2 * kv->Hkv) >= (1ll << 31))
    return abi_fail(PRHS_EUNSUPPORTED, "T * (Hq + 2 Hkv) above 2^31 rows");
  unsigned* err = nullptr;
  if ((s = abi_device(&err, sms)) != PRHS_OK) return s;
  *view = abi_view(*kv, err);
  return PRHS_OK;
}

prhs_status check_new(const prhs_kv& kv, const void* k, long long ks, const void* v, long long vs,
                      const char* who) {
  if (!al16(k) || !al16(v)) return abi_fail(PRHS_EINVAL, who);
  if (!stride_ok(kv, ks, kv.Hkv) || !stride_ok(kv, vs, kv.Hkv))
    return abi_fail(PRHS_EINVAL, "k_stride and v_stride must be at least Hkv * d, in whole 16-byte pieces");
  return PRHS_OK;
}

}  // namespace

extern "C" {

prhs_status prhs_plan_tokens(const prhs_kv* kv, const int32_t* n_new, int T,
                             const int32_t* parents, const int32_t* free_pages, int n_free,
                             const int32_t* free_head, const int32_t* n_pages, int32_t* cu_new,
                             int32_t* positions, int32_t* slots, uint32_t* tree_mask,
                             int32_t* free_head_out, int32_t* n_pages_out, cudaStream_t stream) {
  PlanLaunch a = {};
  int sms = 0;
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (!n_new || !cu_new) return abi_fail(PRHS_EINVAL, "plan: n_new and cu_new must be non-null");
  if (T > 0 && (!positions || !slots)) return abi_fail(PRHS_EINVAL, "plan: positions and slots must be non-null");
  if ((parents == nullptr) != (tree_mask == nullptr))
    return abi_fail(PRHS_EINVAL, "plan: parents and tree_mask must be both set or both null");
  if (!al16(tree_mask)) return abi_fail(PRHS_EINVAL, "plan: tree_mask must be 16-byte aligned");
  const bool paged = kv->block_table != nullptr;
  if (paged && (!free_head || !n_pages || !free_head_out || !n_pages_out))
    return abi_fail(PRHS_EINVAL, "plan: a paged cache needs free_head, n_pages and their outputs");
  if (paged && (n_free < 0 || (n_free > 0 && !free_pages)))
    return abi_fail(PRHS_EINVAL, "plan: free_pages must hold n_free >= 0 pages");
  if ((s = begin(kv, T, &a.kv, &sms)) != PRHS_OK) return s;
  a.n_new = n_new;
  a.T = T;
  a.parents = parents;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.free_head = free_head;
  a.n_pages = n_pages;
  a.block_table = const_cast<int32_t*>(kv->block_table);
  a.cu_new = cu_new;
  a.positions = positions;
  a.slots = slots;
  a.tree_mask = tree_mask;
  a.free_head_out = free_head_out;
  a.n_pages_out = n_pages_out;
  return launched(launch_plan(a, stream));
}

prhs_status prhs_rope_turns(prhs_rope_kind kind, int rot_dim, double base, double factor,
                            double original, double low, double high, uint64_t* turns,
                            float* mscale) {
  if (!turns || !mscale) return abi_fail(PRHS_EINVAL, "rope: null pointer argument");
  if (rot_dim < 16 || rot_dim % 16 != 0) return abi_fail(PRHS_EINVAL, "rope: rot_dim must be a positive multiple of 16");
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
    return abi_fail(PRHS_EINVAL, "rope: base must be above 1 and factor at least 1");
  if (kind < PRHS_ROPE_PLAIN || kind > PRHS_ROPE_RAMP) return abi_fail(PRHS_EINVAL, "rope: unknown kind");
  const bool mixed = kind == PRHS_ROPE_BANDS || kind == PRHS_ROPE_RAMP;
  if (mixed && !(original > 0.0 && low > 0.0 && high > low && std::isfinite(original) && std::isfinite(high)))
    return abi_fail(PRHS_EINVAL, "rope: bands and ramp need original > 0 and high > low > 0");
  const double two_pi = 6.283185307179586476925286766559;
  const double b = kind == PRHS_ROPE_NTK ? base * std::pow(factor, (double)rot_dim / (rot_dim - 2)) : base;
  double first = 0.0, last = 0.0;
  if (kind == PRHS_ROPE_RAMP) {
    // the pair whose angle makes `x` turns over the original context
    auto pair_of = [&](double x) { return rot_dim * std::log(original / (x * two_pi)) / (2.0 * std::log(base)); };
    first = std::fmax(0.0, std::floor(pair_of(high)));
    last = std::fmin(rot_dim - 1.0, std::ceil(pair_of(low)));
  }
  for (int i = 0; i < rot_dim / 2; i++) {
    const double theta = std::pow(b, -2.0 * i / rot_dim);
    double x = theta;
    if (kind == PRHS_ROPE_LINEAR) {
      x = theta / factor;
    } else if (kind == PRHS_ROPE_BANDS) {
      const double keep = std::fmin(1.0, std::fmax(0.0, (original * theta / two_pi - low) / (high - low)));
      x = keep * theta + (1.0 - keep) * (theta / factor);
    } else if (kind == PRHS_ROPE_RAMP) {
      const double g = std::fmin(1.0, std::fmax(0.0, (i - first) / std::fmax(last - first, 0.001)));
      x = g * (theta / factor) + (1.0 - g) * theta;
    }
    // theta <= 1 radian, so the turn is below 1 / 6 and its fraction exact
    turns[i] = (uint64_t)std::ldexp(x / two_pi, 64);
  }
  *mscale = kind == PRHS_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return PRHS_OK;
}

prhs_status prhs_rope_append(const prhs_kv* kv, const prhs_rope* rope, int T,
                             const int32_t* positions, const int32_t* slots, const void* q,
                             long long q_stride, const void* k, long long k_stride, const void* v,
                             long long v_stride, void* q_out, void* k_out, cudaStream_t stream) {
  RopeLaunch a = {};
  int sms = 0;
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (!rope || !rope->turns) return abi_fail(PRHS_EINVAL, "rope_append: rope and its turns must be non-null");
  if (rope->rot_dim < 16 || rope->rot_dim % 16 != 0 || rope->rot_dim > kv->d)
    return abi_fail(PRHS_EINVAL, "rope_append: rot_dim must be a multiple of 16 in [16, d]");
  if ((reinterpret_cast<uintptr_t>(rope->turns) & 7u) != 0)
    return abi_fail(PRHS_EINVAL, "rope_append: turns must be 8-byte aligned");
  if (T > 0 && (!positions || !q || !k || !q_out))
    return abi_fail(PRHS_EINVAL, "rope_append: positions, q, k and q_out must be non-null");
  if (T > 0 && slots && !v) return abi_fail(PRHS_EINVAL, "rope_append: slots need v");
  if (!al16(q) || !al16(q_out) || !al16(k_out)) return abi_fail(PRHS_EINVAL, "rope_append: q, q_out and k_out must be 16-byte aligned");
  if (!stride_ok(*kv, q_stride, kv->Hq))
    return abi_fail(PRHS_EINVAL, "rope_append: q_stride must be at least Hq * d, in whole 16-byte pieces");
  if ((s = check_new(*kv, k, k_stride, slots ? v : nullptr, slots ? v_stride : k_stride,
                     "rope_append: k and v must be 16-byte aligned")) != PRHS_OK)
    return s;
  if ((q_out == q && q_stride != (long long)kv->Hq * kv->d) || (k_out == k && k && k_stride != (long long)kv->Hkv * kv->d))
    return abi_fail(PRHS_EINVAL, "rope_append: in-place results need packed rows");
  if ((s = begin(kv, T, &a.kv, &sms)) != PRHS_OK) return s;
  if (T == 0) return PRHS_OK;
  a.T = T;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.turns = rope->turns;
  a.mscale = rope->mscale;
  a.positions = positions;
  a.slots = slots;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.q_out = q_out;
  a.k_out = k_out;
  return launched(launch_rope(a, sms, stream));
}

size_t prhs_tree_workspace_size(const prhs_kv* kv, int max_new) {
  if (abi_check_kv(kv) != PRHS_OK) return 0;
  if (max_new <= 0) {
    abi_fail(PRHS_EINVAL, "tree: max_new must be positive");
    return 0;
  }
  unsigned* err = nullptr;
  int sms = 0;
  if (abi_device(&err, &sms) != PRHS_OK) return 0;
  return tree_ws_bytes(abi_view(*kv, err), max_new, false, sms);
}

}  // extern "C"

namespace {

// Workspace of shared attention: that of tree attention over units of up to T
// tokens, and two partial states of every token.
struct SharedWs {
  size_t part_o, part_ml, part_ok, states, where, total;
};
SharedWs shared_ws(const KVView& kv, int T, int max_new, int sms) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  SharedWs w;
  w.part_o = up(tree_ws_bytes(kv, T, true, sms));
  w.part_ml = w.part_o + up((size_t)2 * T * kv.Hq * kv.d * sizeof(float));
  w.part_ok = w.part_ml + up((size_t)2 * T * kv.Hq * sizeof(float2));
  w.states = w.part_ok + 256;
  w.where = w.states + up(few_state_bytes(kv, sms));
  w.total = w.where + up(shared_where_bytes(kv, T));
  return w;
}

prhs_status attend(const prhs_kv* kv, const void* q, const void* k_new, long long k_stride, const void* v_new,
                   long long v_stride, float scale, int T, const int32_t* cu_new, int max_new, const uint32_t* tree_mask,
                   const int32_t* shared, void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  TreeLaunch a = {};
  int sms = 0;
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (!cu_new) return abi_fail(PRHS_EINVAL, "tree: cu_new must be non-null");
  if (T > 0 && (!q || !k_new || !v_new || !out || !lse)) return abi_fail(PRHS_EINVAL, "tree: null pointer argument");
  if (max_new <= 0) return abi_fail(PRHS_EINVAL, "tree: max_new must be positive");
  if (tree_mask && max_new > PRHS_TREE_MAX)
    return abi_fail(PRHS_EINVAL, "tree: max_new above PRHS_TREE_MAX with tree_mask");
  if (!al16(q) || !al16(out) || !al16(tree_mask) || !al16(shared))
    return abi_fail(PRHS_EINVAL, "tree: q, out, tree_mask and shared must be 16-byte aligned");
  if ((s = check_new(*kv, k_new, k_stride, v_new, v_stride, "tree: k_new and v_new must be 16-byte aligned")) != PRHS_OK)
    return s;
  if ((s = begin(kv, T, &a.kv, &sms)) != PRHS_OK) return s;
  // 32-bit tile counts: units (256 rows of tokens times group) times their tiles
  const int G = kv->Hq / kv->Hkv;
  const long long units = ((long long)T * G / 256 + kv->B) * kv->Hkv * (shared ? 2 : 1);
  if (units * (a.kv.t_max / 128 + (max_new < T ? max_new : T) / 128 + (shared ? 4 : 2)) >= (1ll << 31))
    return abi_fail(PRHS_EUNSUPPORTED, "tree: too many key tiles for one call");
  if (!ws) return abi_fail(PRHS_EWORKSPACE, "workspace is null");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return abi_fail(PRHS_EWORKSPACE, "workspace must be 256-byte aligned");
  if (!shared && ws_bytes < tree_ws_bytes(a.kv, max_new, false, sms))
    return abi_fail(PRHS_EWORKSPACE, "workspace is smaller than prhs_tree_workspace_size()");
  if (T == 0) return PRHS_OK;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.ks = k_stride;
  a.vs = v_stride;
  a.scale = scale;
  a.T = T;
  a.cu_new = cu_new;
  a.max_new = max_new < T ? max_new : T;  // (a sequence above T is flagged either way)
  a.mask = tree_mask;
  a.out = out;
  a.lse = lse;
  if (shared) {
    const SharedWs w = shared_ws(a.kv, T, a.max_new, sms);
    if (ws_bytes < w.total) return abi_fail(PRHS_EWORKSPACE, "workspace is smaller than prhs_shared_workspace_size()");
    a.shared = reinterpret_cast<const int4*>(shared);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + w.part_o);
    a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + w.part_ml);
    a.part_ok = reinterpret_cast<int*>(static_cast<char*>(ws) + w.part_ok);
    a.few_states = static_cast<char*>(ws) + w.states;
    a.where = reinterpret_cast<int2*>(static_cast<char*>(ws) + w.where);
    few_shape(&a, sms);
  }
  cudaError_t e = cudaSuccess;
  if (kv->dtype == PRHS_BF16) {
    s = shared ? launch_shared_tc(a, sms, ws, stream, &e) : launch_tree_tc(a, sms, ws, stream, &e);
    return s != PRHS_OK ? s : launched(e);
  }
  e = launch_tree(a, sms, ws, stream);
  if (e != cudaSuccess || !shared) return launched(e);
  abi_count_launch();
  return launched(launch_shared_join(a, TreeRecords{}, sms, stream));
}

}  // namespace

extern "C" {

prhs_status prhs_tree_attn(const prhs_kv* kv, const void* q, const void* k_new, long long k_stride,
                           const void* v_new, long long v_stride, float scale, int T,
                           const int32_t* cu_new, int max_new, const uint32_t* tree_mask, void* out,
                           float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return attend(kv, q, k_new, k_stride, v_new, v_stride, scale, T, cu_new, max_new, tree_mask, nullptr, out, lse, ws,
                ws_bytes, stream);
}

size_t prhs_shared_workspace_size(const prhs_kv* kv, int T, int max_new) {
  KVView view;
  int sms = 0;
  if (T <= 0 || max_new <= 0) {
    abi_fail(PRHS_EINVAL, "shared: T and max_new must be positive");
    return 0;
  }
  if (begin(kv, T, &view, &sms) != PRHS_OK) return 0;
  return shared_ws(view, T, max_new < T ? max_new : T, sms).total;
}

prhs_status prhs_shared_attn(const prhs_kv* kv, const void* q, const void* k_new, long long k_stride,
                             const void* v_new, long long v_stride, float scale, int T,
                             const int32_t* cu_new, int max_new, const uint32_t* tree_mask,
                             const int32_t* shared, void* out, float* lse, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
  if (!shared) return abi_fail(PRHS_EINVAL, "shared: shared must be non-null");
  return attend(kv, q, k_new, k_stride, v_new, v_stride, scale, T, cu_new, max_new, tree_mask, shared, out, lse, ws,
                ws_bytes, stream);
}

static prhs_status commit(const prhs_kv* kv, int T, const int32_t* cu_new, const int32_t* slots,
                          const int32_t* accept_idx, int accept_cap, const int32_t* accept_n,
                          const void* k_new, long long k_stride, const void* v_new,
                          long long v_stride, int32_t* new_lens, cudaStream_t stream) {
  CommitLaunch a = {};
  int sms = 0;
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (!cu_new || !accept_n || !new_lens)
    return abi_fail(PRHS_EINVAL, "commit: cu_new, accept_n and new_lens must be non-null");
  if (accept_idx && accept_cap <= 0) return abi_fail(PRHS_EINVAL, "commit: accept_cap must be positive");
  if ((k_new == nullptr) != (v_new == nullptr))
    return abi_fail(PRHS_EINVAL, "commit: k_new and v_new must be both set or both null");
  if (k_new && (s = check_new(*kv, k_new, k_stride, v_new, v_stride,
                              "commit: k_new and v_new must be 16-byte aligned")) != PRHS_OK)
    return s;
  if ((s = begin(kv, T, &a.kv, &sms)) != PRHS_OK) return s;
  a.T = T;
  a.cu_new = cu_new;
  a.slots = slots;
  a.accept_idx = accept_idx;
  a.accept_cap = accept_cap;
  a.accept_n = accept_n;
  a.k_new = k_new;
  a.v_new = v_new;
  a.ks = k_stride;
  a.vs = v_stride;
  a.new_lens = new_lens;
  return launched(launch_commit(a, sms, stream));
}

prhs_status prhs_commit_tokens(const prhs_kv* kv, int T, const int32_t* cu_new,
                               const int32_t* accept_idx, int accept_cap, const int32_t* accept_n,
                               const void* k_new, long long k_stride, const void* v_new,
                               long long v_stride, int32_t* new_lens, cudaStream_t stream) {
  return commit(kv, T, cu_new, nullptr, accept_idx, accept_cap, accept_n, k_new, k_stride, v_new, v_stride, new_lens,
                stream);
}

prhs_status prhs_commit_planned(const prhs_kv* kv, int T, const int32_t* cu_new, const int32_t* slots,
                                const int32_t* accept_idx, int accept_cap, const int32_t* accept_n,
                                const void* k_new, long long k_stride, const void* v_new,
                                long long v_stride, int32_t* new_lens, cudaStream_t stream) {
  if (T > 0 && !slots) return abi_fail(PRHS_EINVAL, "commit: slots must be non-null");
  return commit(kv, T, cu_new, slots, accept_idx, accept_cap, accept_n, k_new, k_stride, v_new, v_stride, new_lens,
                stream);
}

}  // extern "C"
