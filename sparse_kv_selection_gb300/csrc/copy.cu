// Cache rows copied from slot to slot: K and V of every KV head.
//
// A list entry is 2 * Hkv rows of d elements. Entries are cut into 16-byte pieces
// (K's, then V's, head by head) and a CTA takes COPY_PIECES consecutive ones: the
// rows of its entries are worked out once, in shared memory, and every thread has
// its loads in flight together. Entries without a copy cost one read of the list.
// Bound: HBM, each element read once and written once: 78 MB each way 26.6 us from a graph, 0.86
// of the measured copy bandwidth (eight pieces a thread 28.2; divisions by an entry's
// pieces instead of a product 30.8). 440 rows (the last
// pages of 32 sequences, 4 MB each way): 6.2 us, launch and latency.
#include "pages.h"

namespace prhs {

constexpr int COPY_THREADS = 256;
constexpr int COPY_PER = 4;
constexpr int COPY_PIECES = COPY_THREADS * COPY_PER;
constexpr int COPY_ENTRIES = COPY_PIECES / 8 + 1;  // (an entry has at least 16 pieces)

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ CopyLaunch a, int ppr_log2, int per_entry) {
  __shared__ long long from_row[COPY_ENTRIES], to_row[COPY_ENTRIES];
  pdl_wait();
  pdl_trigger();
  const long long x0 = (long long)blockIdx.x * COPY_PIECES, total = (long long)a.n * per_entry;
  const int n = (int)min((long long)COPY_PIECES, total - x0);
  const int e0 = (int)(x0 / per_entry), off0 = (int)(x0 - (long long)e0 * per_entry);
  const int entries = (off0 + n - 1) / per_entry + 1;
  int from_heads = 0, to_heads = 0;
  for (int e = threadIdx.x; e < entries; e += COPY_THREADS) {
    const int from = a.src[e0 + e], to = a.dst[e0 + e];
    auto slots = [](const KVView& kv) { return kv.block_table != nullptr ? kv.num_blocks * kv.block_size : kv.B * kv.t_max; };
    long long row = -1;
    if (from >= 0 && from < slots(a.from) && to >= 0 && to < slots(a.to)) {
      row = slot_row(a.from, from, &from_heads);
      to_row[e] = slot_row(a.to, to, &to_heads);
    } else if (from != -1 && to != -1) {
      raise_error(a.to.err, PRHS_DEV_BAD_INDEX);
    }
    from_row[e] = row;
  }
  from_heads = a.from.block_table != nullptr ? a.from.block_size : a.from.t_max;
  to_heads = a.to.block_table != nullptr ? a.to.block_size : a.to.t_max;
  __syncthreads();

  // y / per_entry rounded down: y + 1/2 (below 2^20 + 1024, entries have at most 2^20 pieces) is half a
  // piece or more from an entry's end, and two roundings move the quotient by less than (y + 1/2) 2^-22 of that
  const float inv = 1.f / per_entry;
  const int half = per_entry / 2, last = (1 << ppr_log2) - 1;
  uint4 c[COPY_PER];
  uint4* dst[COPY_PER];
#pragma unroll
  for (int u = 0; u < COPY_PER; u++) {
    const int x = threadIdx.x + u * COPY_THREADS;
    dst[u] = nullptr;
    if (x >= n) continue;
    const int y = off0 + x, e = __float2int_rd((y + 0.5f) * inv), z = y - e * per_entry;
    const long long row = from_row[e];
    if (row < 0) continue;
    const bool is_v = z >= half;
    const int h = (z - (is_v ? half : 0)) >> ppr_log2;
    c[u] = __ldcs(static_cast<const uint4*>(is_v ? a.from.v : a.from.k) +
                  ((row + (long long)h * from_heads) << ppr_log2) + (z & last));
    dst[u] = static_cast<uint4*>(const_cast<void*>(is_v ? a.to.v : a.to.k)) +
             ((to_row[e] + (long long)h * to_heads) << ppr_log2) + (z & last);
  }
#pragma unroll
  for (int u = 0; u < COPY_PER; u++)
    if (dst[u] != nullptr) __stcs(dst[u], c[u]);
}

cudaError_t launch_copy_rows(const CopyLaunch& a, cudaStream_t st) {
  const int es = a.to.dtype == PRHS_BF16 ? 2 : 4, ppr = a.to.d * es / 16;  // 8, 16 or 32
  const int per_entry = 2 * a.to.Hkv * ppr;
  const long long ctas = ((long long)a.n * per_entry + COPY_PIECES - 1) / COPY_PIECES;
  return launch_pdl(copy_kernel, dim3((unsigned)ctas), dim3(COPY_THREADS), 0, st, a.to.pdl, a,
                    ppr == 8 ? 3 : ppr == 16 ? 4 : 5, per_entry);
}

}  // namespace prhs
