// Operators on vocabulary rows, short rows (up to 16 KB): one warp a row, from the copy
// of the row into shared memory to its results. The serial work of a row's ends (the
// teacher, sums over lanes, logarithms: some microseconds, most of it latency) is as
// long as the rest here, so what counts is how many rows are under way: 10 to 32 an SM,
// by what shared memory holds, a block each (four rows a block, which end together:
// 37 us instead of 27.5 for a step of 3000 rows of 16 KB). On one GB300, passes replayed
// from a graph: a step of 4000 rows of 4096 bf16 entries 21.3 us (the long rows' kernel:
// 70), the loss of 3000 rows of 700 float32 entries 8.5 us (33), a step of 7 rows of 4096
// float32 entries 7.4 us. Bound by the latency of a row's chain of steps.
#include <algorithm>

#include "kernels.h"
#include "tc_ptx.cuh"
#include "vocab_rows.cuh"

namespace eg {
namespace vocab {
namespace {

constexpr int kWarps = 1;     // rows a block
constexpr int kVecs = 8;      // vectors a lane looks at together for alternatives
constexpr int kBatch = 4;     // and for sums

struct alignas(16) WarpScan {
  unsigned long long cand[kCand];
  Cut cut;
};
struct alignas(16) WarpDistill {
  Teacher t;
  Marks marks;
  Coef k;
};
template <int kMode> using WarpSmem = std::conditional_t<kMode == kLogprobs, WarpScan, WarpDistill>;

// The copy's end, for the whole warp. False if it does not come within the limit (the row's results are NaN then);
// a copy that is merely late still lands first (0.2 s more at most), as its place is the next block's afterwards.
__device__ __forceinline__ bool wait_copy(uint64_t* bar, unsigned long long ns) {
  bool ok = tc::mbar_try_wait(bar, 0);
  if (!ok && ns > 0) {
    const unsigned long long t0 = tc::globaltimer();
    while (!(ok = tc::mbar_try_wait(bar, 0)) && tc::globaltimer() - t0 <= ns) {
    }
  }
  if (__all_sync(kFull, ok)) return true;
#pragma unroll 1
  for (int tries = 0; tries < 100000 && !tc::mbar_try_wait(bar, 0); ++tries) {
  }
  return false;
}

template <typename T, bool kEntropy> __device__ __forceinline__ Sums sum_row(const uint4* v, int n, const Sums& edges, float c) {
  const int lane = threadIdx.x & 31;
  Acc<T, kEntropy, kBatch, 32> acc;
  acc.clear();
#pragma unroll 1
  for (int i = 0; i < n; i += kBatch * 32) acc.add(v + i, lane, min(n - i, kBatch * 32), c);
  Sums p = acc.total(c);
  if (lane == 1) p = edges;
  if (lane > 1) p = no_sums();
  return join_lanes<32, kEntropy>(p, c);
}

template <typename T>
__device__ void answer_row(WarpScan& x, const uint4* v, const Args& a, int64_t row, const Row<T>& z, int je, float ze) {
  const int lane = threadIdx.x & 31, k = a.t.k;
  int tok = -1;
  float zt = 0.f;
  if (a.t.logprob && lane == 0) {
    tok = a.t.tok[row];
    if (tok >= 0 && tok < z.n) zt = up(z.row[tok]);
  }
  const Sums p = sum_row<T, true>(v, z.nb, lane_sums<true>(ze, je >= 0, a.c.hi), a.c.hi);
  const Answer ans(p, a.c);
  if (lane == 0) store_answer(a.t, row, ans, p, tok, zt, z.n, a.c);
  if (k == 0) return;
  // the alternatives, as the scanning warps of a long row find them
#pragma unroll
  for (int i = 0; i < kCand / 32; ++i) x.cand[i * 32 + lane] = 0;
  if (lane == 0) x.cut = Cut{0, 0, 0};
  __syncwarp();
  int n_cand = 0, seen = 0;
#pragma unroll 1
  for (int v0 = 0; v0 < z.nb; v0 += kVecs * 32) {
    uint32_t bits = 0;
    if (seen == 0) {
      uint32_t o[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        o[i] = order_bits(v0 + i * 32 + lane < z.nb ? fmaxf(-INFINITY, vec_max<T>(v[v0 + i * 32 + lane])) : -INFINITY);
      bits = kth_bits(o, k);
      if (bits <= order_bits(-INFINITY)) bits = 0;
    } else if ((seen & (seen - 1)) == 0) {
      raise_cut<kCand>(x.cand, &x.cut, k);
    }
    ++seen;
    if (lane == 0 && bits) atomicMax(&x.cut.key, (unsigned long long)bits << 32);
    __syncwarp();
    const float value = cut_value<T>(*(volatile unsigned long long*)&x.cut.key);
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      hits |= (uint32_t)(reaches<T>(v[min(v0 + i * 32 + lane, z.nb - 1)], value) & (v0 + i * 32 + lane < z.nb)) << i;
    n_cand = scan_hits<T>(reinterpret_cast<const T*>(v + v0), hits, 32, 0, z.entry(v0), x.cand, n_cand, &x.cut, k);
    __syncwarp();
  }
  const uint32_t ons = __ballot_sync(kFull, ze > -INFINITY);
  if (n_cand + __popc(ons) > kCand) n_cand = compact(x.cand, &x.cut, k);
  if (ze > -INFINITY) x.cand[n_cand + __popc(ons & ((1u << lane) - 1))] = order_key(ze, je);
  __syncwarp();
  const int n = keep_best<kCand>(x.cand, *(volatile unsigned long long*)&x.cut.key, k);
  int* idx = a.t.idx + row * k;
  float* val = a.t.val + row * k;
  if (ans.good)
    rank_best(x.cand, n, k, [&](int at, unsigned long long key) {
      idx[at] = key_index(key);
      val[at] = ans.logprob(key_value(key), a.c);
    });
#pragma unroll 1
  for (int i = lane; i < k; i += 32)
    if (!ans.good || i >= n) {
      idx[i] = -1;
      val[i] = ans.good ? -INFINITY : NAN;
    }
}

template <typename T, int kMode>
__device__ bool distill_row(WarpDistill& x, uint4* v, uint64_t* bar, const Args& a, int64_t row, const Row<T>& z, int je, float ze) {
  constexpr int kVec = El<T>::kVec;
  const int lane = threadIdx.x & 31;
  const Distill& d = a.d;
  int idx[2];
  float lp[2], zv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = lane + 32 * h;
    idx[h] = e < d.k ? d.t_idx[row * d.k + e] : -1;
    lp[h] = e < d.k ? d.t_lp[row * d.k + e] : -INFINITY;
    zv[h] = idx[h] >= 0 && idx[h] < z.n ? up(z.row[idx[h]]) : 0.f;
  }
#pragma unroll 4
  for (int i = lane; i < Marks::kWords; i += 32) x.marks.w[i] = 0;
  __syncwarp();
  load_teacher(x.t, x.marks, d, idx, lp, zv, z.n, a.c);
  int listed = -1;
  if (__any_sync(kFull, je >= 0))
#pragma unroll 1
    for (int e = 0; e < d.k; ++e)
      if (je >= 0 && x.t.idx[e] == je) listed = e;
  // the listed entries' places among the vectors
  int at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    at[h] = x.t.idx[lane + 32 * h] - z.head;
    if (x.t.idx[lane + 32 * h] < 0 || at[h] >= z.nb * kVec) at[h] = -1;
  }
  if (z.nb > 0 && !wait_copy(bar, a.wait_ns)) return false;
  if constexpr (kMode == kGrad) {
    store_coef(x.k, d.stats + 4 * row, x.t, d, d.g[row], a.c);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)  // the sums are those of the unlisted entries
      if (at[h] >= 0) reinterpret_cast<T*>(v)[at[h]] = down<T>(-INFINITY);
    __syncwarp();
    const Student s(sum_row<T, false>(v, z.nb, lane_sums<false>(ze, je >= 0 && listed < 0, a.c.hi), a.c.hi), x.t, d, a.c);
    if (kMode == kStep) store_coef(x.k, s, x.t, d.g[row], a.c);
    store_loss(d, row, s, x.t, a.c);
  }
  if constexpr (kMode != kLoss) {
    __syncwarp();
    const Ref ref = x.k.ref;
    const float coef = x.k.coef;
    const bool zero = x.k.zero;
    T* dz = reinterpret_cast<T*>(d.dz) + row * d.ld_dz;
    T* out = dz + z.head;
    if (reinterpret_cast<uintptr_t>(out) % 16 == 0) {
#pragma unroll 4
      for (int i = lane; i < z.nb; i += 32)
        *reinterpret_cast<uint4*>(out + i * kVec) = grad_vec<T>(v[i], ref, coef, zero, a.c.hi);
    } else {
#pragma unroll 1
      for (int i = lane; i < z.nb; i += 32) store_unaligned<T>(out + i * kVec, grad_vec<T>(v[i], ref, coef, zero, a.c.hi));
    }
    __syncwarp();  // then the listed entries, over what the loop wrote in their places
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (at[h] >= 0) out[at[h]] = down<T>(zero ? 0.f : x.k.g[lane + 32 * h]);
    if (je >= 0) dz[je] = down<T>(zero ? 0.f : listed >= 0 ? x.k.g[listed] : x.k.at(ze, a.c.hi));
  }
  return true;
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kWarps * 32) short_kernel(const __grid_constant__ Args a, int row_bytes) {
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ uint64_t bars[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (row >= a.r.rows) return;
  uint8_t* mine = raw + warp * ((int)sizeof(WarpSmem<kMode>) + row_bytes);
  WarpSmem<kMode>& x = *reinterpret_cast<WarpSmem<kMode>*>(mine);
  uint4* v = reinterpret_cast<uint4*>(mine + sizeof(WarpSmem<kMode>));
  const Row<T> z(a.r.z, a.r.ld, row, a.r.vocab);
  uint64_t* bar = &bars[warp];
  if (lane == 0 && z.nb > 0) {
    tc::mbar_init(bar, 1);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc::mbar_expect_tx(bar, z.nb * 16);
    tc::bulk_load(v, z.row + z.head, z.nb * 16, bar);
  }
  __syncwarp();
  const int je = lane < kEdges ? z.edge(lane) : -1;
  const float ze = je >= 0 ? up(z.row[je]) : -INFINITY;
  bool ok;
  if constexpr (kMode == kLogprobs) {
    ok = z.nb == 0 || wait_copy(bar, a.wait_ns);
    if (ok) answer_row<T>(x, v, a, row, z, je, ze);
  } else {
    ok = distill_row<T, kMode>(x, v, bar, a, row, z, je, ze);
  }
  if (!ok) no_results<T, kMode>(a, row, lane, 32);
}

template <typename T, int kMode> cudaError_t run_short(const Args& a, cudaStream_t s) {
  const int row_bytes = std::max(16, a.r.vocab / El<T>::kVec * 16);
  const int smem = kWarps * ((int)sizeof(WarpSmem<kMode>) + row_bytes);
  constexpr int kMost = kWarps * ((int)sizeof(WarpSmem<kMode>) + kShortRow);
  if (!raise_smem_limit(reinterpret_cast<const void*>(&short_kernel<T, kMode>), kMost)) return cudaErrorInvalidValue;
  return launch_pdl(short_kernel<T, kMode>, dim3((unsigned)(((int64_t)a.r.rows + kWarps - 1) / kWarps)), dim3(kWarps * 32), smem,
                    s, a, row_bytes);
}

}  // namespace

cudaError_t short_rows(const Args& a, int mode, cudaStream_t s) {
  return by_type(a.r.dtype, [&](auto x) {
    using T = decltype(x);
    return mode == kLogprobs ? run_short<T, kLogprobs>(a, s)
           : mode == kLoss   ? run_short<T, kLoss>(a, s)
           : mode == kStep   ? run_short<T, kStep>(a, s)
                             : run_short<T, kGrad>(a, s);
  });
}

}  // namespace vocab
}  // namespace eg
