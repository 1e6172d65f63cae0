// Operators on vocabulary rows, long rows: log probabilities of given tokens with
// entropy and the best alternatives, and distillation from a teacher's top tokens
// (loss, gradient, both at once).
//
// All of them are bound by the bytes of the logits, so each reads a row once. One
// persistent kernel, two blocks an SM (for a loss: one of twice the size); a row
// belongs to a cluster of C blocks, each of which streams its part of the row through a
// ring of six chunks:
//   summing warps    sums of exponentials; the gradient's second look at the chunks,
//                    which stay in the ring until it is written
//   a copying warp   bulk copies into the ring, running ahead over rows
//   then, for log probabilities,
//   scanning warps   candidates for the best alternatives: a look at each chunk of their own
//   a selecting warp the best of a row's candidates, sorted
//   an answering one joins the sums and the lists over the blocks, writes the row's answers
//   or, for distillation,
//   teaching warps   the teacher, some rows ahead
//   a finishing one  joins the sums over the blocks, the gradient's coefficients
//   a writing one    the row's loss
// so that the copies never wait for the serial work of a row's end. Blocks of a cluster
// talk through distributed shared memory and barriers there. Nothing goes through
// global scratch: calls have no workspace and no atomics on global memory.
//
// A row is cut into units that depend on its length alone, and sums are joined unit by
// unit, so that a row's results depend neither on the number of rows nor on their blocks.
//
// Measured on one GB300 (128256 entries of bf16; passes replayed from a graph; copy
// bandwidth 6.78 TB/s):
//   loss, 1024 rows           45.7 us = 5.7 TB/s; the first row waits for its teacher, and
//                             the last round has 112 rows for 152 blocks
//   gradient, 1024 rows       89 us = 5.9 TB/s, bound by the memory
//   step, 2048 rows, k = 64   184 us = 5.7 TB/s read and written; clusters of 4 fill 144 of
//                             152 SMs (of 8, as float32 rows need, 120); then the summing
//                             warps' instructions (60% of the issue slots, ALU pipe 44%)
//   log probabilities, 2048 rows, k = 16: 127 us = 4.1 TB/s (k = 64: 222; without
//                             alternatives, 1024 rows, 49.5 us = 5.3): instructions, 68% of the
//                             issue slots on 30 warps; the scan's second look at each vector and
//                             the entropy's second sum are what it has beyond the loss
//   waits that say whether they were met, which a role leaves its rows on if not, cost a
//                             step 1% (183.7 to 185.8 us in turn), the rest less
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "tc_ptx.cuh"
#include "vocab_rows.cuh"

namespace eg {
namespace {

using namespace vocab;
using tc::mbar_arrive;
using tc::smem_u32;

constexpr int kScan = 4;          // scanning warps
constexpr int kSlots = 6;         // chunks in the ring
constexpr int kPer = 4;           // vectors of a chunk a summing thread takes, at most
constexpr int kMaxCluster = 8;    // blocks a row (the portable cluster size)
constexpr int kMaxUnits = 8;

// A step keeps two rows' parts in the ring: while the blocks join a row's sums, the next
// row is summed, and its gradient is written after that (joining takes 2,900 to 5,800 cycles,
// of some 5,900 from row to row, which two blocks an SM with a row each did not hide: 2048
// rows of 128256 bf16 entries took 209 to 255 us). So one block an SM, with the ring and the
// warps of two; the loss alone has the same shape (46 us for 1024 rows against 50).
template <int kMode> struct Shape {
  static constexpr bool kWide = kMode == kStep || kMode == kLoss;
  static constexpr int kBlocks = kWide ? 1 : 2;   // blocks an SM
  static constexpr int kNW = kWide ? 16 : 8;      // summing warps
  static constexpr int kNT = kNW * 32;
  static constexpr int kChunk = kPer * kNT;                // 16-byte vectors a chunk, at most
  static constexpr int kBuf = kMode == kLogprobs ? 2 : 4;  // rows between their teacher and their end
  // then the copying warp and: the scanning ones, the selecting and the answering one;
  // or two teaching ones; the finishing one and the one that writes the loss
  static constexpr int kThreads = kNT + 32 + (kMode == kLogprobs ? kScan + 2 : kMode == kGrad ? 2 : 4) * 32;
};

// ---- barriers --------------------------------------------------------------------------------------

// A wait ends after Args::wait_ns at the latest (2 s). The block then gives up: every later wait of it that is not
// over already fails at once, each role leaves its rows at a wait that failed, before it uses what it waited for, and
// the results of all the cluster's rows become NaN (give_up). The cluster's other blocks miss its parts and follow.
struct Limit {
  unsigned long long ns;
  int over;
};
template <bool kCluster> __device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  if (!kCluster) return tc::mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(tc::kSuspendNs) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool time_is_up(uint32_t tries, unsigned long long t0, const Limit* limit) {
  return limit->ns == 0 || (tries % 64 == 63 && tc::globaltimer() - t0 > limit->ns);
}
// One thread.
__device__ __noinline__ bool wait_one(uint64_t* bar, uint32_t parity, Limit* limit) {
  const unsigned long long t0 = tc::globaltimer();
  for (uint32_t i = 0; !try_wait<false>(bar, parity); ++i) {
    if (time_is_up(i, t0, limit)) *(volatile int*)&limit->over = 1;
    if (*(volatile int*)&limit->over) return false;
  }
  return true;
}
// A warp: the same answer for all its lanes.
template <bool kCluster> __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, Limit* limit) {
  const unsigned long long t0 = tc::globaltimer();
#pragma unroll 1
  for (uint32_t i = 0; !__all_sync(kFull, try_wait<kCluster>(bar, parity)); ++i) {
    const bool over = *(volatile int*)&limit->over || time_is_up(i, t0, limit);
    if (__any_sync(kFull, over)) {
      *(volatile int*)&limit->over = 1;
      return false;
    }
  }
  return true;
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Limit* limit) {
  return __all_sync(kFull, try_wait<kCluster>(bar, parity)) || wait_long<kCluster>(bar, parity, limit);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The cluster's rows: the first, and the distance to the next.
__device__ __forceinline__ void cluster_rows(uint32_t& row0, uint32_t& step) {
  asm volatile("mov.u32 %0, %%clusterid.x;\nmov.u32 %1, %%nclusterid.x;" : "=r"(row0), "=r"(step));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// A place of this block's shared memory in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Sums to that place, counted there by a barrier's expected bytes (no fence: an
// arrival that releases earlier stores would wait for them).
__device__ __forceinline__ void send(Sums* p, uint64_t* bar, uint32_t rank, const Sums& v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   remote(p, rank)),
               "f"(v.m), "f"(v.s), "f"(v.u), "f"(v.top), "r"(remote(bar, rank))
               : "memory");
}
__device__ __forceinline__ void st_remote(int* p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_remote(unsigned long long* p, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void arrive_remote(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank)) : "memory");
}

// ---- a block's part of a row -----------------------------------------------------------------------

// Units [u0, u1) of the row; a unit in chunks.
template <typename T> struct Part : Row<T> {
  int u0, u1, unit;
  __device__ Part(const Args& a, int64_t row, int rank) : Row<T>(a.r.z, a.r.ld, row, a.r.vocab) {
    u0 = min(a.units, rank * a.mine);
    u1 = min(a.units, u0 + a.mine);
    unit = a.unit;
  }
  __device__ int begin(int u) const { return min(this->nb, u * unit); }  // of unit u
  // f(first vector, vectors) for each chunk of unit u, until one is false
  template <int kChunk, typename F> __device__ __forceinline__ bool chunks(int u, F f) const {
    const int e = begin(u + 1);
#pragma unroll 1
    for (int v = begin(u); v < e; v += kChunk)
      if (!f(v, min(kChunk, e - v))) return false;
    return true;
  }
};

// ---- shared memory ---------------------------------------------------------------------------------

constexpr int kScanCluster = 4;   // blocks a row where there are alternatives

struct ScanSmem {
  unsigned long long cand[2][kScan][kCand];                    // 0: none
  unsigned long long list[kMaxAlternatives];                   // the block's best, sorted
  unsigned long long mail[2][kScanCluster][kMaxAlternatives];  // every block's
  int mail_n[2][kScanCluster];
  int list_n;
  Cut cut[2];  // of the block's entries
};

struct alignas(16) DistillRow {
  Teacher t;
  Coef k;
  // The block's part: its vectors, where their gradient goes, whether that is 16-byte aligned.
  int n_vec, aligned;
  void* out;
  // An entry's place in it, for the summing warp that has its vector: chunk * warps + warp (-1: in another block),
  // and the entry of the chunk.
  int owner[kMaxTeacher], at[kMaxTeacher];
  float edge_z[kEdges];
  int edge_entry[kEdges];  // the teacher's entry of an edge, -1: none
  Sums edges, joined;
};

template <int kMode> struct Smem {
  static constexpr int kBuf = Shape<kMode>::kBuf;
  uint4 ring[kSlots][Shape<kMode>::kChunk];
  Sums warp[kBuf][kMode == kLogprobs ? kScanCluster : 1][Shape<kMode>::kNW];
  Sums part[kBuf][kMaxUnits + 1];  // of the row's units and its edges
  std::conditional_t<kMode == kLogprobs, ScanSmem, DistillRow[4]> x;
  std::conditional_t<kMode == kLogprobs, char, Marks[2]> marks;  // of the teaching warps
  uint64_t full[kSlots], empty[kSlots];
  uint64_t ready[kBuf];         // the summing warps may begin the row
  uint64_t sums[kBuf];          // they have its sums
  uint64_t mail[kBuf];          // the blocks' sums (and lists) are here
  uint64_t ack[kBuf];           // the blocks have read this block's lists
  uint64_t joined[kBuf];        // the row's sums are joined, and its gradient's coefficients there
  uint64_t done[kBuf];          // the row is done with
  uint64_t scanned[2], taken[2];    // a row's candidates are there, are done with
  uint64_t listed, unlisted;        // the block's list is there, is done with
  Limit limit;
  uint32_t copied;  // chunks that the copying warp asked for
};
// Where row number `it` of a block keeps its data, and the parity of that place's barriers.
template <int kMode> __device__ __forceinline__ int buf_of(int it) { return it % Shape<kMode>::kBuf; }
template <int kMode> __device__ __forceinline__ int turn_of(int it) { return it / Shape<kMode>::kBuf & 1; }

// ---- the copying warp ------------------------------------------------------------------------------

template <typename T, int kMode>
__device__ void copy_rows(Smem<kMode>& sm, const Args& a, int rank, int64_t row0, int64_t step) {
  if ((threadIdx.x & 31) != 0) return;
  uint32_t g = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step) {
    const Part<T> z(a, row, rank);
#pragma unroll 1
    for (int u = z.u0; u < z.u1; ++u)
      if (!z.template chunks<Shape<kMode>::kChunk>(u, [&](int v, int n) {
            const uint32_t slot = g % kSlots, turn = g / kSlots;
            if (turn > 0 && !wait_one(&sm.empty[slot], (turn - 1) & 1, &sm.limit)) return false;
            tc::mbar_expect_tx(&sm.full[slot], n * 16);
            tc::bulk_load(sm.ring[slot], z.row + z.entry(v), n * 16, &sm.full[slot]);
            ++g;
            return true;
          })) {
        sm.copied = g;
        return;
      }
  }
  sm.copied = g;
}

// After the roles of a block that gave up (all of the cluster's have ended): what is under way to its shared memory
// has to land before it ends, and nobody may take what stands in the rows' results for such.
template <typename T, int kMode> __device__ __noinline__ void give_up(Smem<kMode>& sm, const Args& a) {
  if (threadIdx.x == 0) {
    // copies, by the chunks' barriers, 0.2 s each at most
    const uint32_t g = sm.copied;
#pragma unroll 1
    for (uint32_t o = g > kSlots ? g - kSlots : 0; o < g; ++o)
#pragma unroll 1
      for (int tries = 0; tries < 100000 && !try_wait<false>(&sm.full[o % kSlots], (o / kSlots) & 1); ++tries) {
      }
    // sums that other blocks sent, of which nothing here tells how many: they take microseconds, this a millisecond
#pragma unroll 1
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  uint32_t row0, step;
  cluster_rows(row0, step);
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step) no_results<T, kMode>(a, row, threadIdx.x, blockDim.x);
}

// ---- summing warps ---------------------------------------------------------------------------------

template <typename T, int kMode>
__device__ void sum_rows(Smem<kMode>& sm, const Args& a, int rank, int64_t row0, int64_t step) {
  using S = Shape<kMode>;
  constexpr int kVec = El<T>::kVec;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = a.c.hi;
  Limit* limit = &sm.limit;
  uint32_t g = 0;
  // a row's sums; the slots stay taken in a step
  auto sum = [&](int64_t row, int it) {
    const int b = buf_of<kMode>(it);
    if (!wait(&sm.ready[b], turn_of<kMode>(it), limit)) return false;
    Acc<T, kMode == kLogprobs, kPer, S::kNT> acc;
    acc.clear();
    if constexpr (kMode == kLogprobs) {
      const Part<T> z(a, row, rank);
#pragma unroll 1
      for (int u = z.u0; u < z.u1; ++u) {
        if (u > z.u0) acc.clear();
        if (!z.template chunks<S::kChunk>(u, [&](int, int n) {
              const uint32_t slot = g % kSlots;
              if (!wait(&sm.full[slot], (g / kSlots) & 1, limit)) return false;
              acc.add(sm.ring[slot], tid, n, c);
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.empty[slot]);
              ++g;
              return true;
            }))
          return false;
        const Sums w = acc.total(c);
        if (lane == 0) sm.warp[b][u - z.u0][warp] = w;
      }
    } else {
      const DistillRow& x = sm.x[b];
      const int owner[2] = {x.owner[lane], x.owner[lane + 32]}, at[2] = {x.at[lane], x.at[lane + 32]};
      int me = warp;  // of the chunk
#pragma unroll 1
      for (int left = x.n_vec; left > 0; left -= S::kChunk, me += S::kNW, ++g) {
        const uint32_t slot = g % kSlots;
        if (!wait(&sm.full[slot], (g / kSlots) & 1, limit)) return false;
        // The listed entries become -inf: the sums are those of the unlisted. (Taking them off the full sum
        // instead would leave nothing of an unlisted share below 2^-24.)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (owner[h] == me) {
            reinterpret_cast<T*>(sm.ring[slot])[at[h]] = down<T>(-INFINITY);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the slot's next copy
          }
        __syncwarp();
        acc.add(sm.ring[slot], tid, min(left, S::kChunk), c);
        if (kMode != kStep) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.empty[slot]);
        }
      }
      const Sums w = acc.total(c);
      if (lane == 0) sm.warp[b][0][warp] = w;
    }
    if (lane == 0) mbar_arrive(&sm.sums[b]);
    return true;
  };
  // a row's gradient; `slots` counts its chunks
  auto grad = [&](int it, uint32_t& slots) {
    if constexpr (kMode == kStep || kMode == kGrad) {
      const int b = buf_of<kMode>(it);
      if (!wait(kMode == kStep ? &sm.joined[b] : &sm.ready[b], turn_of<kMode>(it), limit)) return false;
      const DistillRow& x = sm.x[b];
      const int owner[2] = {x.owner[lane], x.owner[lane + 32]}, at[2] = {x.at[lane], x.at[lane + 32]};
      const Ref ref = x.k.ref;
      const float coef = x.k.coef;
      const bool zero = x.k.zero, aligned = x.aligned;
      T* out = reinterpret_cast<T*>(x.out);
      int me = warp;
#pragma unroll 1
      for (int left = x.n_vec; left > 0; left -= S::kChunk, me += S::kNW, ++slots, out += S::kChunk * kVec) {
        const uint32_t slot = slots % kSlots;
        if (kMode == kGrad && !wait(&sm.full[slot], (slots / kSlots) & 1, limit)) return false;
        const uint4* in = sm.ring[slot];
        if (aligned && left >= S::kChunk) {  // without a branch per vector
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            *reinterpret_cast<uint4*>(out + (i * S::kNT + tid) * kVec) = grad_vec<T>(in[i * S::kNT + tid], ref, coef, zero, c);
        } else if (aligned) {
#pragma unroll 1
          for (int v = tid; v < left; v += S::kNT)
            *reinterpret_cast<uint4*>(out + v * kVec) = grad_vec<T>(in[v], ref, coef, zero, c);
        } else {
#pragma unroll 1
          for (int v = tid; v < min(left, S::kChunk); v += S::kNT)
            store_unaligned<T>(out + v * kVec, grad_vec<T>(in[v], ref, coef, zero, c));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[slot]);
        // then the listed entries, over what this warp wrote in their places
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (owner[h] == me) out[at[h]] = down<T>(zero ? 0.f : x.k.g[lane + 32 * h]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.done[b]);
    }
    return true;
  };
  if constexpr (kMode == kStep) {
    uint32_t written = 0;
    int it = 0;
#pragma unroll 1
    for (int64_t row = row0; row < a.r.rows + step; row += step, ++it) {
      if (row < a.r.rows && !sum(row, it)) return;
      if (it > 0 && !grad(it - 1, written)) return;
    }
  } else {
    int it = 0;
#pragma unroll 1
    for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
      if (kMode == kGrad ? !grad(it, g) : !sum(row, it)) return;
    }
  }
}

// ---- scanning and selecting warps ------------------------------------------------------------------

// The chunks are dealt to the scanning warps, one at a time: what a look costs besides
// its 1,024 vectors (waits, the way to the candidates, the ring's slot) is paid once a
// chunk, and nothing but the cut is shared. Entries are compared with a cut that at
// least k entries reach: a warp's first chunk of the row gives one (from its lanes'
// maxima), and the candidates of all, looked at after 2, 4, 8, ... chunks, raise it, so
// that some hundred of a row's entries become candidates. A vector's maximum decides
// whether its entries are looked at.
template <typename T>
__device__ void scan_rows(Smem<kLogprobs>& sm, const Args& a, int rank, int wid, int64_t row0, int64_t step) {
  using S = Shape<kLogprobs>;
  constexpr int kAtOnce = 8, kRounds = S::kChunk / 32 / kAtOnce;  // vectors a lane: 8 in flight, 4 times
  static_assert(kAtOnce * kRounds <= 32, "a bit a vector");
  const int lane = threadIdx.x & 31, k = a.t.k;
  const uint32_t below = (1u << lane) - 1;
  Limit* limit = &sm.limit;
  ScanSmem& x = sm.x;
  uint32_t g = 0;
  int it = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
    const int b = it & 1, ph = (it >> 1) & 1;
    const Part<T> z(a, row, rank);
    unsigned long long* cand = x.cand[b][wid];
    Cut* cut = &x.cut[b];
    if (it >= 2 && !wait(&sm.taken[b], ph ^ 1, limit)) return;
    int seen = 0, n_cand = 0;
    bool first = true;
#pragma unroll 1
    for (int u = z.u0; u < z.u1; ++u)
      if (!z.template chunks<S::kChunk>(u, [&](int v0, int n) {
            const uint32_t slot = g % kSlots, turn = g / kSlots;
            ++seen;
            if (g++ % kScan != wid) return true;
            // The slot's turn before was another warp's. While its copy has not landed, the parity to wait for is that of
            // the turn before it, which has: so first the end of that turn (the one before was over when it was asked for).
            if (turn > 0 && !wait(&sm.empty[slot], (turn - 1) & 1, limit)) return false;
            if (!wait(&sm.full[slot], turn & 1, limit)) return false;
            const uint4* chunk = sm.ring[slot];
            if (first) {
              first = false;
              float most[kAtOnce];
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) most[i] = -INFINITY;
#pragma unroll 1
              for (int r = 0; r < kRounds; ++r)
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                  const int v = (r * kAtOnce + i) * 32 + lane;
                  const float t = vec_max<T>(chunk[min(v, n - 1)]);
                  if (v < n) most[i] = fmaxf(most[i], t);  // each entry once only
                }
              uint32_t o[kAtOnce];
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) o[i] = order_bits(most[i]);
              const uint32_t bits = kth_bits(o, k);
              if (lane == 0 && bits > order_bits(-INFINITY)) atomicMax(&cut->key, (unsigned long long)bits << 32);
              __syncwarp();
            }
            const float value = cut_value<T>(*(volatile unsigned long long*)&cut->key);
            uint32_t hits = 0;
#pragma unroll 1
            for (int r = 0; r < kRounds; ++r)
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                const int v = (r * kAtOnce + i) * 32 + lane;
                hits |= (uint32_t)(reaches<T>(chunk[min(v, n - 1)], value) & (v < n)) << (r * kAtOnce + i);
              }
            n_cand = scan_hits<T>(reinterpret_cast<const T*>(chunk), hits, 32, 0, z.entry(v0), cand, n_cand, cut, k);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[slot]);
            if ((seen & (seen - 1)) == 0) raise_cut<kScan * kCand>(&x.cand[b][0][0], cut, k);
            return true;
          }))
        return;
    if (wid == 0 && rank == 0) {  // the edges
      const int j = lane < kEdges ? z.edge(lane) : -1;
      const float v = j >= 0 ? up(z.row[j]) : -INFINITY;
      const uint32_t ons = __ballot_sync(kFull, v > -INFINITY);
      if (n_cand + __popc(ons) > kCand) n_cand = compact(cand, cut, k);
      if (v > -INFINITY) cand[n_cand + __popc(ons & below)] = order_key(v, j);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.scanned[b]);
  }
}

// The selecting warp: the best of a row's candidates, sorted.
__device__ void select_rows(Smem<kLogprobs>& sm, const Args& a, int64_t row0, int64_t step) {
  const int lane = threadIdx.x & 31, k = a.t.k;
  Limit* limit = &sm.limit;
  ScanSmem& x = sm.x;
  int it = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
    const int b = it & 1;
    unsigned long long* cand = &x.cand[b][0][0];
    if (!wait(&sm.scanned[b], (it >> 1) & 1, limit)) return;
    const int n = keep_best<kScan * kCand>(cand, *(volatile unsigned long long*)&x.cut[b].key, k);
    if (it >= 1 && !wait(&sm.unlisted, (it - 1) & 1, limit)) return;
    rank_best(cand, n, k, [&](int at, unsigned long long key) { x.list[at] = key; });
    if (lane == 0) x.list_n = min(n, k);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.listed);
#pragma unroll 1
    for (int i = lane; i < kScan * kCand; i += 32) cand[i] = 0;  // for the row after next
    if (lane == 0) x.cut[b].key = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.taken[b]);
  }
}

// ---- joining the blocks ----------------------------------------------------------------------------

// One warp: the sums of the block's units (and, from the cluster's first block, of the
// edges) to every block. Each group of kNW lanes joins a unit's warps.
template <bool kEntropy, int kMode>
__device__ __forceinline__ void mail_sums(Smem<kMode>& sm, const Args& a, int b, int u0, int u1, int rank, const Sums& edges) {
  constexpr int kNW = Shape<kMode>::kNW;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int s = 0; s < u1 - u0; s += 32 / kNW) {
    const int u = s + lane / kNW;
    Sums p = no_sums();
    if (u < u1 - u0) p = sm.warp[b][u][lane % kNW];
    p = join_lanes<kNW, kEntropy>(p, a.c.hi);
    if (u < u1 - u0 && lane % kNW < a.C) send(&sm.part[b][u0 + u], &sm.mail[b], lane % kNW, p);
  }
  if (rank == 0 && lane < a.C) send(&sm.part[b][kMaxUnits], &sm.mail[b], lane, edges);
  if (lane == 0) tc::mbar_expect_tx(&sm.mail[b], (a.units + 1) * (uint32_t)sizeof(Sums));  // what comes here
}
// The row's sums, from the parts that every block sent.
template <bool kEntropy, int kMode> __device__ __forceinline__ Sums row_sums(const Smem<kMode>& sm, const Args& a, int b) {
  const int lane = threadIdx.x & 31;
  Sums p = no_sums();
  if (lane <= kMaxUnits) p = sm.part[b][lane];
  p = join_lanes<16, kEntropy>(p, a.c.hi);
  // lanes 16..31 joined nothing
  p.m = __shfl_sync(kFull, p.m, 0);
  p.s = __shfl_sync(kFull, p.s, 0);
  p.u = __shfl_sync(kFull, p.u, 0);
  p.top = __shfl_sync(kFull, p.top, 0);
  return p;
}

// The answering warp of a call for log probabilities: the row's answers; of the alternatives, each block writes its own.
template <typename T>
__device__ void answer_rows(Smem<kLogprobs>& sm, const Args& a, int rank, int64_t row0, int64_t step) {
  const int lane = threadIdx.x & 31, C = a.C, k = a.t.k;
  Limit* limit = &sm.limit;
  ScanSmem& x = sm.x;
  int it = 0;
  if (lane < 2) mbar_arrive(&sm.ready[lane]);
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
    const int b = it & 1, ph = (it >> 1) & 1;
    const Part<T> z(a, row, rank);
    int tok = -1, je = -1;
    float zt = 0.f, ze = -INFINITY;
    if (rank == 0) {
      je = lane < kEdges ? z.edge(lane) : -1;
      if (je >= 0) ze = up(z.row[je]);
      if (a.t.logprob && lane == 0) {
        tok = a.t.tok[row];
        if (tok >= 0 && tok < z.n) zt = up(z.row[tok]);
      }
    }
    const Sums edges = lane_sums<true>(ze, je >= 0, a.c.hi);
    if (!wait(&sm.sums[b], ph, limit)) return;
    if (it >= 2 && !wait<true>(&sm.ack[b], ph ^ 1, limit)) return;
    if (k > 0) {
      if (!wait(&sm.listed, it & 1, limit)) return;
      const int n = x.list_n;
#pragma unroll 1
      for (int o = 0; o < C; ++o)
#pragma unroll 1
        for (int i = lane; i < n; i += 32) st_remote(&x.mail[b][rank][i], o, x.list[i]);
      if (lane < C) st_remote(&x.mail_n[b][rank], lane, n);
      __syncwarp();
      if (lane < C) arrive_remote(&sm.mail[b], lane);
    }
    mail_sums<true>(sm, a, b, z.u0, z.u1, rank, edges);
    if (lane == 0) {
      mbar_arrive(&sm.ready[b]);
      if (k > 0) mbar_arrive(&sm.unlisted);
    }
    if (!wait<true>(&sm.mail[b], ph, limit)) return;
    const Sums p = row_sums<true>(sm, a, b);
    const Answer ans(p, a.c);
    if (k > 0) {
      const int mine = lane < C ? x.mail_n[b][lane] : 0;
      int* idx = a.t.idx + row * k;
      float* val = a.t.val + row * k;
      int n[kScanCluster], total = 0;
#pragma unroll
      for (int o = 0; o < kScanCluster; ++o) {
        n[o] = __shfl_sync(kFull, mine, o);
        total += n[o];
      }
      const int own = __shfl_sync(kFull, mine, rank);
#pragma unroll 1
      for (int e = lane; ans.good && e < own; e += 32) {
        const unsigned long long key = x.mail[b][rank][e];
        // Before it are e of its own list and, of each other sorted list, the larger ones: bisections side by side.
        int at = e, lo[kScanCluster];
#pragma unroll
        for (int o = 0; o < kScanCluster; ++o) lo[o] = 0;
#pragma unroll 1
        for (int w = C == 1 ? 0 : k > 32 ? 64 : k > 16 ? 32 : k > 8 ? 16 : 8; w > 0; w /= 2) {
#pragma unroll
          for (int o = 0; o < kScanCluster; ++o)
            if (lo[o] + w <= n[o] && x.mail[b][o][lo[o] + w - 1] > key) lo[o] += w;
        }
#pragma unroll
        for (int o = 0; o < kScanCluster; ++o)
          if (o != rank) at += lo[o];
        if (at < k) {
          idx[at] = key_index(key);
          val[at] = ans.logprob(key_value(key), a.c);
        }
      }
      if (rank == 0)
#pragma unroll 1
        for (int i = lane; i < k; i += 32)
          if (!ans.good || i >= total) {
            idx[i] = -1;
            val[i] = ans.good ? -INFINITY : NAN;
          }
    }
    if (rank == 0 && lane == 0) store_answer(a.t, row, ans, p, tok, zt, z.n, a.c);
    __syncwarp();
    if (lane < C) arrive_remote(&sm.ack[b], lane);
  }
}

// ---- teaching warps --------------------------------------------------------------------------------

// The edges' gradients, by lanes 0..15 of a warp of the cluster's first block.
template <typename T>
__device__ __forceinline__ void store_edges(const DistillRow& x, const Args& a, const Row<T>& z, int64_t row) {
  const int lane = threadIdx.x & 31;
  const int j = lane < kEdges ? z.edge(lane) : -1;
  if (j < 0) return;
  const int e = x.edge_entry[lane];
  const float g = e >= 0 ? x.k.g[e] : x.k.at(x.edge_z[lane], a.c.hi);
  (reinterpret_cast<T*>(a.d.dz) + row * a.d.ld_dz)[j] = down<T>(x.k.zero ? 0.f : g);
}

// The teacher of every second row (`which`), some rows ahead; for the gradient alone its coefficients too.
template <typename T, int kMode>
__device__ void teach_rows(Smem<kMode>& sm, const Args& a, int rank, int which, int64_t row0, int64_t step) {
  const int lane = threadIdx.x & 31;
  Limit* limit = &sm.limit;
  int it = which, idx[2];
  float lp[2];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = lane + 32 * h;
      const bool in = row < a.r.rows && e < a.d.k;
      idx[h] = in ? a.d.t_idx[row * a.d.k + e] : -1;
      lp[h] = in ? a.d.t_lp[row * a.d.k + e] : -INFINITY;
    }
  };
  fetch(row0 + which * step);
#pragma unroll 1
  for (int64_t row = row0 + which * step; row < a.r.rows; row += 2 * step, it += 2) {
    const int b = buf_of<kMode>(it);
    const Part<T> z(a, row, rank);
    const int je = rank == 0 && lane < kEdges ? z.edge(lane) : -1;
    const float ze = je >= 0 ? up(z.row[je]) : -INFINITY;
    float zv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) zv[h] = idx[h] >= 0 && idx[h] < z.n ? up(z.row[idx[h]]) : 0.f;
    if (it >= Shape<kMode>::kBuf && !wait(&sm.done[b], turn_of<kMode>(it) ^ 1, limit)) return;
    DistillRow& x = sm.x[b];
    Teacher& t = x.t;
    load_teacher(t, sm.marks[which], a.d, idx, lp, zv, z.n, a.c);
    fetch(row + 2 * step);
    const int first = z.begin(z.u0), n_vec = z.begin(z.u1) - first;
    if (lane == 0) {
      T* out = reinterpret_cast<T*>(a.d.dz) + row * a.d.ld_dz + z.entry(first);
      x.n_vec = n_vec;
      x.out = out;
      x.aligned = reinterpret_cast<uintptr_t>(out) % 16 == 0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      using S = Shape<kMode>;
      const int i = lane + 32 * h;
      const int64_t at = (int64_t)t.idx[i] - z.entry(first);  // of the block's entries
      const bool in = t.idx[i] >= 0 && at >= 0 && at < (int64_t)n_vec * El<T>::kVec;
      const int v = (int)(at / El<T>::kVec);
      x.owner[i] = in ? v / S::kChunk * S::kNW + v % S::kNT / 32 : -1;
      x.at[i] = in ? (int)(at % ((int64_t)S::kChunk * El<T>::kVec)) : 0;
    }
    int listed = -1;
    if (__any_sync(kFull, je >= 0))
#pragma unroll 1
      for (int e = 0; e < a.d.k; ++e)
        if (je >= 0 && t.idx[e] == je) listed = e;
    if (lane < kEdges) {
      x.edge_z[lane] = ze;
      x.edge_entry[lane] = listed;
    }
    if constexpr (kMode == kGrad) {
      store_coef(x.k, a.d.stats + 4 * row, t, a.d, a.d.g[row], a.c);
      __syncwarp();
      if (rank == 0) store_edges<T>(x, a, z, row);
    } else {
      const Sums e = lane_sums<false>(ze, je >= 0 && listed < 0, a.c.hi);
      if (lane == 0) x.edges = e;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ready[b]);
  }
}

// ---- the finishing and the writing warp ------------------------------------------------------------

// The sums to every block, the row's sums, and for a step its coefficients.
template <typename T, int kMode>
__device__ void finish_rows(Smem<kMode>& sm, const Args& a, int rank, int64_t row0, int64_t step) {
  const int lane = threadIdx.x & 31;
  Limit* limit = &sm.limit;
  int it = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
    const int b = buf_of<kMode>(it), ph = turn_of<kMode>(it);
    const Part<T> z(a, row, rank);
    DistillRow& x = sm.x[b];
    const float gr = kMode == kStep ? a.d.g[row] : 0.f;
    if (!wait(&sm.sums[b], ph, limit)) return;
    // Another block sends a row's part only after it has this block's part of the row before, which this warp sends
    // when it has read all of the row before that: so a place is read before it is written again. No other warp
    // reads the places; the writing warp, which may be some rows behind, has the joined sums.
    mail_sums<false>(sm, a, b, z.u0, z.u1, rank, x.edges);
    if (!wait<true>(&sm.mail[b], ph, limit)) return;
    const Sums p = row_sums<false>(sm, a, b);
    if (lane == 0) x.joined = p;
    if constexpr (kMode == kStep) {
      store_coef(x.k, Student(p, x.t, a.d, a.c), x.t, gr, a.c);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.joined[b]);
    if (kMode == kStep && rank == 0) store_edges<T>(x, a, z, row);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.done[b]);
  }
}

// The row's loss and sums, by the cluster's first block.
template <int kMode>
__device__ void write_rows(Smem<kMode>& sm, const Args& a, int rank, int64_t row0, int64_t step) {
  const int lane = threadIdx.x & 31;
  Limit* limit = &sm.limit;
  int it = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.r.rows; row += step, ++it) {
    const int b = buf_of<kMode>(it);
    const DistillRow& x = sm.x[b];
    if (!wait(&sm.joined[b], turn_of<kMode>(it), limit)) return;
    if (rank == 0) store_loss(a.d, row, Student(x.joined, x.t, a.d, a.c), x.t, a.c);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.done[b]);
  }
}

// ---- the kernel ------------------------------------------------------------------------------------

template <typename T, int kMode>
__global__ void __launch_bounds__(Shape<kMode>::kThreads, Shape<kMode>::kBlocks) vocab_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem<kMode>& sm = *reinterpret_cast<Smem<kMode>*>(raw);
  const int rank = (int)cluster_rank(), warp = threadIdx.x >> 5;
  using S = Shape<kMode>;
  const bool scan = kMode == kLogprobs && a.t.k > 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], S::kNW + (scan ? 1 : 0));
    }
    for (int i = 0; i < S::kBuf; ++i) {
      tc::mbar_init(&sm.ready[i], 1);
      tc::mbar_init(&sm.sums[i], S::kNW);
      // the block's own warp, which knows how many bytes of sums come; and the blocks' lists
      tc::mbar_init(&sm.mail[i], 1 + (scan ? a.C : 0));
      tc::mbar_init(&sm.ack[i], a.C);
      tc::mbar_init(&sm.joined[i], 1);
      // the finishing and the writing warp where there is a loss, the summing ones where there is a gradient
      tc::mbar_init(&sm.done[i], (kMode == kGrad ? 0 : 2) + (kMode == kLoss ? 0 : S::kNW));
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.scanned[i], kScan);
      tc::mbar_init(&sm.taken[i], 1);
    }
    tc::mbar_init(&sm.listed, 1);
    tc::mbar_init(&sm.unlisted, 1);
    sm.limit = Limit{a.wait_ns, 0};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if constexpr (kMode != kLogprobs)
    for (int i = threadIdx.x; i < 2 * Marks::kWords; i += S::kThreads) sm.marks[i / Marks::kWords].w[i % Marks::kWords] = 0;
  if constexpr (kMode == kLogprobs) {
    for (int i = threadIdx.x; i < 2 * kScan * kCand; i += S::kThreads) (&sm.x.cand[0][0][0])[i] = 0;
    if (threadIdx.x < 2) sm.x.cut[threadIdx.x] = Cut{0, 0, 0};
  }
  if (threadIdx.x < S::kBuf * (kMaxUnits + 1))
    (&sm.part[0][0])[threadIdx.x] = no_sums();  // units that the row does not have
  __syncthreads();
  cluster_sync();
  pdl_wait();  // what the launch before this one wrote; nothing above touches it
  pdl_trigger();
  uint32_t row0, step;
  cluster_rows(row0, step);
  const int other = warp - S::kNW;
  if (other < 0) {
    sum_rows<T, kMode>(sm, a, rank, row0, step);
  } else if (other == 0) {
    copy_rows<T, kMode>(sm, a, rank, row0, step);
  } else if constexpr (kMode == kLogprobs) {
    if (other == kScan + 2) answer_rows<T>(sm, a, rank, row0, step);
    else if (scan && other <= kScan) scan_rows<T>(sm, a, rank, other - 1, row0, step);
    else if (scan) select_rows(sm, a, row0, step);
  } else {
    if (kMode == kGrad || other < 3) teach_rows<T, kMode>(sm, a, rank, other - 1, row0, step);
    else if (other == 3) finish_rows<T, kMode>(sm, a, rank, row0, step);
    else write_rows<kMode>(sm, a, rank, row0, step);
  }
  __syncwarp();
  cluster_sync();  // no block ends while another may write to it
  if (sm.limit.over) give_up<T, kMode>(sm, a);
}

// ---- launches --------------------------------------------------------------------------------------

// A kernel's launch for clusters of C blocks.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  Launch(int C, int64_t clusters, int threads, size_t smem, cudaStream_t s) {
    cfg.gridDim = dim3((unsigned)(clusters * C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
  }
};

// Clusters of C blocks that the current device holds at once (asked once per kernel, C and device).
template <typename T, int kMode> int max_clusters(int C, size_t smem) {
  static std::atomic<int> known[64][kMaxCluster + 1];  // 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>* slot = dev < 64 ? &known[dev][C] : nullptr;
  int n = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  Launch l(C, std::max(1, num_sms() / C), Shape<kMode>::kThreads, smem, nullptr);
  if (cudaOccupancyMaxActiveClusters(&n, vocab_kernel<T, kMode>, &l.cfg) != cudaSuccess) return 0;
  if (slot) slot->store(n, std::memory_order_relaxed);
  return n;
}

// Blocks a row. The order of a row's sums may depend on its length alone, so
//  - for log probabilities a row has up to 4 units, and up to 4 blocks: the count whose
//    rounds over the rows take least, a block's part of a row costing its bytes and
//    kRowBytes more for its ends, which are not overlapped in full (kListBytes where there
//    are alternatives): 1024 rows of 128256 bf16 entries take 132 us with one block a row and
//    151 with two at k = 64, without alternatives 54 and 49; 61 rows of float32 at k = 10
//    take 20.9, 15.3 and 14.0 us with 1, 2 and 4;
//  - for a loss a unit is a block's part, and their number follows from the length: the
//    least that keeps a part within kLossPart bytes, or, in a step, two parts in the ring (with
//    two chunks of room where the cluster allows it: 184 us for 2048 rows with four, 289 with
//    eight). Where kLossPart lies within 200 to 500 KB matters little with many rows (1024
//    rows of 250 KB: 45.7 us with one block, 44.7 with two; 600 of 400 KB: 41.5 and 42.6; 500
//    of 500 KB: 45.1, 43.7), while smaller parts cost more (four blocks 55.3, 47.7, 42.4; eight
//    108, 72, 57) and few rows of 250 KB would gain (30 rows: 9.7 us with one block, 7.8 with
//    two, 7.1 with four), which a count that follows from the length alone cannot have;
//  - the gradient alone has no sums: as for log probabilities (1024 rows of bf16 87, 89
//    and 90 us with 1, 2 and 4).
constexpr int64_t kRowBytes = 24 << 10, kListBytes = 96 << 10, kLossPart = 264 << 10;

template <typename T, int kMode> cudaError_t run(const Args& args, cudaStream_t s) {
  using S = Shape<kMode>;
  const void* kernel = reinterpret_cast<const void*>(&vocab_kernel<T, kMode>);
  constexpr size_t smem = sizeof(Smem<kMode>);
  static_assert(S::kBlocks * (smem + 1024) <= 233472, "shared memory of an SM");
  if (!raise_smem_limit(kernel, (int)smem)) return cudaErrorInvalidValue;
  const int nvec = std::max(1, args.r.vocab / El<T>::kVec);  // of the longest row
  auto div = [](int x, int y) { return (x + y - 1) / y; };
  Args a = args;
  int n_clusters = 0;
  int64_t best = 0;
  for (int C = 1; C <= (kMode == kLogprobs ? kScanCluster : kMaxCluster); C *= 2) {
    Args t = args;
    t.C = C;
    t.units = kMode == kLogprobs ? std::min(kScanCluster, div(nvec, S::kChunk)) : C;
    if (C > 1 && C >= 2 * t.units) break;
    t.mine = div(t.units, C);
    t.unit = div(nvec, t.units);
    // whole rounds of the summing warps, where that makes the parts no more than a 32nd uneven
    const int whole = div(t.unit, S::kNT) * S::kNT;
    if (whole - t.unit <= t.unit / 32) t.unit = whole;
    const int chunks = div(t.unit, S::kChunk);
    if (kMode == kLoss && C < kMaxCluster && (int64_t)t.unit * 16 > kLossPart) continue;
    if (kMode == kStep && chunks > (2 * C <= kMaxCluster ? kSlots / 2 - 1 : kSlots / 2)) continue;
    const int n = max_clusters<T, kMode>(C, smem);
    if (n <= 0) continue;
    const int64_t cost = (a.r.rows + n - 1) / n * ((int64_t)t.mine * t.unit * 16 + (kMode == kLogprobs && a.t.k > 0 ? kListBytes : kRowBytes));
    if (!n_clusters || cost < best) {
      a = t;
      n_clusters = n;
      best = cost;
    }
    if (kMode == kLoss || kMode == kStep) break;
  }
  if (!n_clusters) return cudaErrorInvalidValue;
  Launch l(a.C, std::min<int64_t>(a.r.rows, n_clusters), S::kThreads, smem, s);
  void* params[] = {&a};
  return cudaLaunchKernelExC(&l.cfg, kernel, params);
}

thread_local unsigned long long wait_ns = tc::kTimeoutNs;

Args args_of(const VocabRows& r) {
  Args a{};
  a.wait_ns = wait_ns;
  a.r = r;
  a.c = scale_of(r.temperature);
  return a;
}

// Rows of up to kShortRow bytes are a warp's (vocab_short.cu).
bool is_short(const VocabRows& r) { return (int64_t)r.vocab * (r.dtype == EAGLE_DTYPE_F32 ? 4 : 2) <= kShortRow; }

}  // namespace

void set_vocab_wait(int64_t ns) { wait_ns = ns < 0 ? tc::kTimeoutNs : (unsigned long long)ns; }

cudaError_t token_logprobs(const VocabRows& r, const TokenLogprobs& t, cudaStream_t s) {
  Args a = args_of(r);
  a.t = t;
  if (is_short(r)) return short_rows(a, kLogprobs, s);
  return by_type(r.dtype, [&](auto x) { return run<decltype(x), kLogprobs>(a, s); });
}

cudaError_t distill_loss(const VocabRows& r, const Distill& d, cudaStream_t s) {
  Args a = args_of(r);
  a.d = d;
  if (is_short(r)) return short_rows(a, kLoss, s);
  return by_type(r.dtype, [&](auto x) { return run<decltype(x), kLoss>(a, s); });
}

cudaError_t distill_grad(const VocabRows& r, const Distill& d, cudaStream_t s) {
  Args a = args_of(r);
  a.d = d;
  if (is_short(r)) return short_rows(a, kGrad, s);
  return by_type(r.dtype, [&](auto x) { return run<decltype(x), kGrad>(a, s); });
}

cudaError_t distill_loss_grad(const VocabRows& r, const Distill& d, cudaStream_t s) {
  Args a = args_of(r);
  a.d = d;
  if (is_short(r)) return short_rows(a, kStep, s);
  const int64_t size = r.dtype == EAGLE_DTYPE_F32 ? 4 : 2;
  // a longer row than a cluster holds twice: two passes
  static_assert(kMaxCluster * (kSlots / 2) * Shape<kStep>::kChunk * 16 == EAGLE_DISTILL_ONE_PASS_BYTES, "what eagle.h says");
  if (r.vocab * size > EAGLE_DISTILL_ONE_PASS_BYTES) {
    const cudaError_t err = distill_loss(r, d, s);
    return err != cudaSuccess ? err : distill_grad(r, d, s);
  }
  return by_type(r.dtype, [&](auto x) { return run<decltype(x), kStep>(a, s); });
}

}  // namespace eg
