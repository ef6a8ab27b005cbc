// The last launch of the attention that reads shared prefixes once. A token of a
// group has two states, one against the shared keys (one pass over them gave it for
// all the group's tokens) and one against its sequence's other keys:
//
//   m = max(m1, m2),  o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2)
//
// On bf16 each may lie in pieces, one for each CTA or warp of the launch before that had
// a run of its unit's keys (`where`: the first, how many). A warp takes eight rows and 32
// columns, a lane eight columns of a row; of up to four rows (WAYS) lanes share a row's pieces (16
// samples of 4096 keys 36.9 us, 38.7 without, 32 questions on 131072 115.7 and 119.7; 128 tokens
// of few pieces 90 and 88). Bound: latency, four dependent reads through L2
// (the sequence, its group; the pieces' places, the pieces), the first two of which do not wait
// for the launch in front: 10 us behind 32 drafts or 128 tokens, 25 behind 913 prompt tokens of
// 32 heads on one prefix (48 MB of states).
#include "tree_join.cuh"

namespace prhs {

constexpr int SJ_THREADS = 128, SJ_CTAS_SM = 8, SJ_PIECES = 4;  // (pieces in flight)

template <typename T, int D, bool WAYS>
__global__ void __launch_bounds__(SJ_THREADS, WAYS ? 5 : SJ_CTAS_SM) shared_join_kernel(const __grid_constant__ TreeLaunch a,
                                                                 const __grid_constant__ TreeRecords rec, int ctas) {
  constexpr int C4 = D / 4, CHUNKS = D / 32;
  const KVView& kv = a.kv;
  const int G = kv.Hq / kv.Hkv, gl = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3, b = blockIdx.x;
  // as tree_item reads them (the launch before has flagged what does not fit), through L2: what
  // was there before that launch may stand in an L1 that this one's wait has not passed
  const int4 mine = __ldcg(a.shared + b);
  const int len = __ldcg(kv.seq_lens + b), lo = __ldcg(a.cu_new + b), hi = __ldcg(a.cu_new + b + 1);
  if (blockIdx.x + blockIdx.y == 0) pdl_wait();  // (one waits whatever it has to do: this launch ends behind the one before)
  if (lo < 0 || hi <= lo || hi > a.T || hi - lo > a.max_new) return;
  const int t = max(0, min(len, kv.t_max)), n = hi - lo, head = max(0, min(mine.x, b));
  const bool grouped = mine.x == head && !(mine.x == b && (mine.y <= 1 || mine.z == 0));
  const int4 group = grouped ? __ldcg(a.shared + head) : make_int4(0, 0, 0, 0);
  const int head_len = grouped ? __ldcg(kv.seq_lens + head) : 0, group0 = grouped ? max(0, __ldcg(a.cu_new + head)) : 0;
  int keys = 0;  // that are shared
  if (grouped) {
    keys = kv.block_table != nullptr ? group.z / kv.block_size * kv.block_size : group.z;
    const bool same = group.x == head && group.y == mine.y && group.z == mine.z;
    if (!same || b - head >= group.y || keys < 0 || keys > t || keys > head_len) keys = 0;
  }
  const bool few[2] = {false, sizeof(T) == 2 && few_item(a, n, t - keys)};  // whose are the states?
  // all that was there before the launch in front; what it wrote from here on
  pdl_wait();
  pdl_trigger();
  if (*a.part_ok == 0) return;
  // eight lanes take the rows; of fewer rows (1, 2, 4) several take a part of the pieces each
  const int rows = n << gl, blocks = (rows + 7) / 8, lane = threadIdx.x & 31;
  const int span = !WAYS || rows > 4 ? 8 : rows == 3 ? 4 : rows, ways = WAYS ? 8 / span : 1, way = WAYS ? (lane & 7) / span : 0;
  const long long warps = (long long)gridDim.y * (SJ_THREADS / 32), total = (long long)kv.Hkv * blocks * CHUNKS;
  for (long long i = (long long)blockIdx.y * (SJ_THREADS / 32) + threadIdx.x / 32; i < total; i += warps) {
    const int chunk = (int)i % CHUNKS, hr = (int)(i / CHUNKS), kvh = hr / blocks, r = (hr - kvh * blocks) * 8 + (lane & 7) % span;
    const bool out_of = r >= rows;
    if (!WAYS && out_of) continue;
    const int rr = min(r, rows - 1), tok = lo + (rr >> gl), h = rr & (G - 1), c4 = chunk * 8 + (lane >> 3) * 2;
    int2 at[2] = {make_int2(0, 1), make_int2(0, 1)};  // of the states against the shared and the other keys
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 2; k++)
        if (k == 1 || keys > 0) at[k] = __ldcg(a.where + part_row<T>(a, k + 1, tok, kvh, h, gl));
    }
    const bool stands = keys == 0 && (sizeof(T) == 4 || at[1].y <= 1);  // its result is written
    if (WAYS ? __all_sync(FULL_MASK, stands || out_of) : stands) continue;
    float M = -INFINITY, L = 0.f;
    float4 y[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < 2; k++) {
      if (k == 0 && keys == 0) continue;
      const float2* ml = a.part_ml + part_row<T>(a, k + 1, tok, kvh, h, gl);
      const float4* o = part_at<T, D>(a, k + 1, tok, kvh, h, c4, gl);
      long long ml_step = 0, o_step = 0, next = sizeof(T) == 4 ? 1 : (long long)a.T << gl;  // to the next piece, the next columns
      int pieces = 1, first = 0;
      if (sizeof(T) == 2 && at[k].y > 1) {
        // a writer's second slot is of the unit that it begins, its first of one begun before
        const int writers = few[k] ? a.few_warps : ctas, unit = few[k] ? a.few_rows : 256, stride = few[k] ? unit : rec.rows_max;
        first = max(0, min(at[k].x, writers - 1));  // (whatever stands there after a launch that gave up)
        pieces = min(at[k].y, writers - first);
        const int row = (k == 0 ? ((tok - group0) << gl) + h : rr) & (unit - 1);
        const float4* states = static_cast<const float4*>(a.few_states);
        ml = (few[k] ? reinterpret_cast<const float2*>(states + 2ll * a.few_warps * C4 * unit) : rec.ml) + row;
        o = (few[k] ? states : rec.o) + (long long)c4 * stride + row;
        ml_step = stride;
        o_step = (long long)C4 * stride;
        next = stride;
      }
      for (int p0 = 0; p0 < pieces; p0 += SJ_PIECES * ways) {
        float2 s[SJ_PIECES];
        float4 x[SJ_PIECES][2];
#pragma unroll
        for (int p = 0; p < SJ_PIECES; p++) {
          s[p] = make_float2(-INFINITY, 0.f);
          x[p][0] = x[p][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          const int at_p = p0 + p * ways + way;
          if (at_p < pieces) {
            const long long slot = 2ll * (first + at_p) + (at_p == 0);
            s[p] = __ldcg(ml + slot * ml_step);
            x[p][0] = __ldcg(o + slot * o_step);
            x[p][1] = __ldcg(o + slot * o_step + next);
          }
        }
        float m = M;
#pragma unroll
        for (int p = 0; p < SJ_PIECES; p++) m = fmaxf(m, s[p].x);
        const float keep = tree_weight(M, m);
        L *= keep;
#pragma unroll
        for (int c = 0; c < 2; c++) y[c] = make_float4(y[c].x * keep, y[c].y * keep, y[c].z * keep, y[c].w * keep);
#pragma unroll
        for (int p = 0; p < SJ_PIECES; p++) {
          const float w = tree_weight(s[p].x, m);
          L = fmaf(w, s[p].y, L);  // (a state that holds NaN has it in its sum, whatever its maximum)
          tree_fma(y[0], w, x[p][0]);
          tree_fma(y[1], w, x[p][1]);
        }
        M = m;
      }
    }
    if constexpr (WAYS) {
      for (int d = span; d < 8; d <<= 1) {  // the ways' shares of a row meet
        const float other = __shfl_xor_sync(FULL_MASK, M, d), m = fmaxf(M, other);
        const float w0 = tree_weight(M, m), w1 = tree_weight(other, m);
        L = fmaf(w1, __shfl_xor_sync(FULL_MASK, L, d), w0 * L);
#pragma unroll
        for (int c = 0; c < 2; c++) {
          float* v = &y[c].x;
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] = fmaf(w1, __shfl_xor_sync(FULL_MASK, v[e], d), w0 * v[e]);
        }
        M = m;
      }
      if (stands || out_of || way != 0) continue;
    }
    const float inv = tree_inv(L);
    const long long orow = (long long)tok * kv.Hq + (kvh << gl) + h;
    T* out = static_cast<T*>(a.out) + orow * D + c4 * 4;
#pragma unroll
    for (int c = 0; c < 2; c++) tree_put(out + c * 4, make_float4(y[c].x * inv, y[c].y * inv, y[c].z * inv, y[c].w * inv));
    if (c4 == 0) a.lse[orow] = tree_lse(M, L);
  }
}

template <typename T, int D>
static cudaError_t join_go(const TreeLaunch& a, const TreeRecords& rec, int sms, cudaStream_t st) {
  const long long blocks = ((long long)a.max_new * (a.kv.Hq / a.kv.Hkv) + 7) / 8;
  long long y = (blocks * a.kv.Hkv * (D / 32) + SJ_THREADS / 32 - 1) / (SJ_THREADS / 32);
  // one wave, since each CTA looks its sequence up (24 prompts: two waves 127.5 us, one 128.6, half of one 143);
  // with WAYS, of which an SM holds 5 CTAs, 1.6. A sequence's rows are its own CTAs' alone: one of many rows
  // among many of few is joined by few CTAs
  const long long most = ((long long)SJ_CTAS_SM * sms + a.kv.B - 1) / a.kv.B;
  if (y > most) y = most;
  auto* kernel = sizeof(T) == 2 && a.max_new * (a.kv.Hq / a.kv.Hkv) <= 4 ? shared_join_kernel<T, D, sizeof(T) == 2> : shared_join_kernel<T, D, false>;
  return launch_pdl(kernel, dim3(a.kv.B, (unsigned)y), dim3(SJ_THREADS), 0, st, true, a, rec, sms);
}
cudaError_t launch_shared_join(const TreeLaunch& a, const TreeRecords& rec, int sms, cudaStream_t st) {
  if (a.kv.dtype == PRHS_BF16)
    return a.kv.d == 128 ? join_go<__nv_bfloat16, 128>(a, rec, sms, st) : join_go<__nv_bfloat16, 64>(a, rec, sms, st);
  return a.kv.d == 128 ? join_go<float, 128>(a, rec, sms, st) : join_go<float, 64>(a, rec, sms, st);
}

}  // namespace prhs
