// C ABI of the operators for sequences that share pages: argument checks and
// launches. The contract of every entry point is in include/prhs.h.
#include "pages.h"

using namespace prhs;

namespace {

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

prhs_status launched(cudaError_t e) {
  if (e == cudaSuccess) {
    abi_count_launch();
    return PRHS_OK;
  }
  return abi_fail(PRHS_ECUDA, cudaGetErrorString(e));
}

prhs_status check_paged(const prhs_kv* kv) {
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (kv->block_table == nullptr) return abi_fail(PRHS_EINVAL, "pages: the cache is not paged");
  if ((long long)kv->B * kv->max_blocks >= (1ll << 30))  // entries are numbered in 30 bits
    return abi_fail(PRHS_EUNSUPPORTED, "pages: B * max_blocks above 2^30 entries");
  if ((long long)kv->B * kv->max_blocks * kv->block_size >= (1ll << 36))  // 128 kept positions a task
    return abi_fail(PRHS_EUNSUPPORTED, "pages: B * max_blocks * block_size above 2^36 positions");
  return PRHS_OK;
}

// What fork and compact have in common.
prhs_status pages_call(const prhs_kv* kv, const prhs_pages* now, const prhs_pages* next, PagesLaunch a, void* ws,
                       size_t ws_bytes, cudaStream_t stream) {
  if (!now || !next) return abi_fail(PRHS_EINVAL, "pages: now and next must be non-null");
  if (!now->n_pages || !now->page_shares || !now->free_head || !next->n_pages || !next->page_shares || !next->free_head)
    return abi_fail(PRHS_EINVAL, "pages: n_pages, page_shares and free_head must be non-null");
  if (now->n_free < 0 || now->n_free != next->n_free || (now->n_free > 0 && (!now->free_pages || !next->free_pages)))
    return abi_fail(PRHS_EINVAL, "pages: free_pages must hold n_free >= 0 pages, as many before as after");
  if ((now->block_table && now->block_table != kv->block_table) || (now->seq_lens && now->seq_lens != kv->seq_lens))
    return abi_fail(PRHS_EINVAL, "pages: the table and the lengths before are the descriptor's");
  if (!a.src || !a.dst) return abi_fail(PRHS_EINVAL, "pages: src and dst must be non-null");
  if (!al4(a.src) || !al4(a.dst)) return abi_fail(PRHS_EINVAL, "pages: arrays must be aligned");
  unsigned* err = nullptr;
  int sms = 0;
  const prhs_status s = abi_device(&err, &sms);
  if (s != PRHS_OK) return s;
  a.kv = abi_view(*kv, err);
  if (!ws) return abi_fail(PRHS_EWORKSPACE, "workspace is null");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return abi_fail(PRHS_EWORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < pages_workspace(a.kv)) return abi_fail(PRHS_EWORKSPACE, "workspace is smaller than prhs_pages_workspace_size()");
  a.n_pages = now->n_pages;
  a.shares = now->page_shares;
  a.free_pages = now->free_pages;
  a.free_head = now->free_head;
  a.n_free = now->n_free;
  a.table_out = next->block_table ? next->block_table : const_cast<int32_t*>(kv->block_table);
  a.lens_out = next->seq_lens ? next->seq_lens : const_cast<int32_t*>(kv->seq_lens);
  a.n_pages_out = next->n_pages;
  a.shares_out = next->page_shares;
  a.free_out = next->free_pages;
  a.head_out = next->free_head;
  pages_split(&a, ws);
  return launched(launch_pages(a, sms, stream));
}

}  // namespace

extern "C" {

size_t prhs_pages_workspace_size(const prhs_kv* kv) {
  if (check_paged(kv) != PRHS_OK) return 0;
  return pages_workspace(abi_view(*kv, nullptr));
}

prhs_status prhs_fork_seqs(const prhs_kv* kv, const prhs_pages* now, const int32_t* parent, const prhs_pages* next,
                           int32_t* src, int32_t* dst, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const prhs_status s = check_paged(kv);
  if (s != PRHS_OK) return s;
  if (!parent) return abi_fail(PRHS_EINVAL, "fork: parent must be non-null");
  PagesLaunch a = {};
  a.parent = parent;
  a.src = src;
  a.dst = dst;
  a.cap = kv->block_size;
  return pages_call(kv, now, next, a, ws, ws_bytes, stream);
}

prhs_status prhs_compact_seqs(const prhs_kv* kv, const prhs_pages* now, const int32_t* keep, int cap,
                              const int32_t* keep_n, const prhs_pages* next, int32_t* src, int32_t* dst, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
  const prhs_status s = check_paged(kv);
  if (s != PRHS_OK) return s;
  if (!keep || !keep_n) return abi_fail(PRHS_EINVAL, "compact: keep and keep_n must be non-null");
  if (cap <= 0) return abi_fail(PRHS_EINVAL, "compact: cap must be positive");
  if (cap > 1 << 30) return abi_fail(PRHS_EUNSUPPORTED, "compact: cap above 2^30 positions");  // (a cache has fewer)
  PagesLaunch a = {};
  a.keep = keep;
  a.keep_n = keep_n;
  a.src = src;
  a.dst = dst;
  a.cap = cap;
  return pages_call(kv, now, next, a, ws, ws_bytes, stream);
}

prhs_status prhs_copy_rows(const prhs_kv* kv, const prhs_kv* source, int n, const int32_t* src, const int32_t* dst,
                           cudaStream_t stream) {
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (source == nullptr) source = kv;
  if ((s = abi_check_kv(source)) != PRHS_OK) return s;
  if (source->dtype != kv->dtype || source->Hkv != kv->Hkv || source->d != kv->d)
    return abi_fail(PRHS_EINVAL, "copy_rows: the caches differ in element type, KV heads or d");
  if (n < 0) return abi_fail(PRHS_EINVAL, "copy_rows: n must be >= 0");
  if (n > 0 && (!src || !dst)) return abi_fail(PRHS_EINVAL, "copy_rows: src and dst must be non-null");
  // 32-bit counts of thread blocks: 1024 16-byte pieces each
  if ((long long)n * 2 * kv->Hkv * kv->d * (kv->dtype == PRHS_BF16 ? 2 : 4) / 16 >= (1ll << 40))
    return abi_fail(PRHS_EUNSUPPORTED, "copy_rows: too many rows for one call");
  unsigned* err = nullptr;
  int sms = 0;
  if ((s = abi_device(&err, &sms)) != PRHS_OK) return s;
  if (n == 0) return PRHS_OK;
  CopyLaunch a = {};
  a.to = abi_view(*kv, err);
  a.from = abi_view(*source, err);
  a.n = n;
  a.src = src;
  a.dst = dst;
  return launched(launch_copy_rows(a, stream));
}

prhs_status prhs_find_shared(const prhs_kv* kv, const int32_t* cu_new, int min_keys, int32_t* shared, cudaStream_t stream) {
  prhs_status s = abi_check_kv(kv);
  if (s != PRHS_OK) return s;
  if (!cu_new || !shared) return abi_fail(PRHS_EINVAL, "find_shared: cu_new and shared must be non-null");
  if ((reinterpret_cast<uintptr_t>(shared) & 15u) != 0) return abi_fail(PRHS_EINVAL, "find_shared: shared must be 16-byte aligned");
  if (min_keys < 0) return abi_fail(PRHS_EINVAL, "find_shared: min_keys must be >= 0");
  unsigned* err = nullptr;
  int sms = 0;
  if ((s = abi_device(&err, &sms)) != PRHS_OK) return s;
  FindLaunch a = {};
  a.kv = abi_view(*kv, err);
  a.cu_new = cu_new;
  a.min_keys = min_keys;
  a.shared = reinterpret_cast<int4*>(shared);
  return launched(launch_find_shared(a, stream));
}

}  // extern "C"
