// Cutting caches to a budget of rows by accumulated attention weight.
//
// A sequence with n > budget rows keeps its first `sink` rows, its last
// `recent` rows and, of the rows between, the budget - sink - recent heaviest
// (equal weights: the lower row first; a NaN weighs less than anything); the
// kept rows stay in order.  Two kernels:
//
//   k_evict_select  the kept rows of each sequence, in order: the K-th
//                   heaviest key by radix selection (weights mapped to
//                   integers of the same order; three digits of 11, 11 and 10
//                   bits, a shared-memory histogram each), then a compaction of
//                   the rows above it and the first of those equal.  Latency
//                   is its bound: 4 n bytes per sequence in a chain of
//                   dependent steps.  So a sequence gets a cluster of CTAs,
//                   one per 4096 rows up to eight, whose threads hold their
//                   keys in registers across the steps and add up the
//                   histograms over distributed shared memory (one CTA for
//                   60,001 rows: 98 us; eight: 22 us).
//   k_evict_move    the rows' bytes, scales and weights, each kept row read and
//                   written once.  16-bit rows of a batch are bound by HBM (16
//                   x 8192 rows of 3 KB to half: 66 us, 6.1 TB/s, 0.93 of a
//                   copy's rate; in place, in order, 4.6 TB/s).  A quantised
//                   cache's scales, like the weights, are moved by one CTA a
//                   sequence in dependent rounds (move_small), which bounds
//                   long sequences: whole calls, to half, into other memory /
//                   in place, us: 16 x 8192 rows int8 r 768 60 / 50, int4 r 1536
//                   81 / 83; one of 60,001 rows 155 / 204 and 252 / 343 (fp16 r
//                   1536: 62 / 91)
//
// In place the move has an order to keep: row j of the result is row
// src[j] >= j of the source, src increasing.  A CTA owns a column slice of a
// sequence and walks the rows in chunks, the whole chunk read before any of
// it is written: what chunk k writes, rows below its end, no later chunk
// reads, since src[j] >= j -- so the next chunk is already loading.  Into other
// memory there is no order, and a CTA copies whole rows.
#include "internal.cuh"

namespace qsvd {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 8;                              // consecutive rows per thread
constexpr int kSelChunk = kSelThreads * kSelKeys;        // rows of a CTA held in registers at a time
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster, with release / acquire of its memory accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at p (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Two consecutive words from an even one on.
__device__ __forceinline__ unsigned long long peer_pair(const uint32_t* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}

// Order-preserving integer of a weight; NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the CTA's 1024 threads; *total: the sum.  red: 32 words
// that the call before did not use (one barrier a call: every warp scans the
// warps' sums for itself).
__device__ __forceinline__ uint32_t cta_exclusive(uint32_t v, uint32_t* red, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  uint32_t y = red[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xffffffffu, y, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
  return (warp ? before : 0u) + x - v;
}

// grid B x CS in clusters of CS, block 1024.  CTA `rank` of a sequence's
// cluster sees to rows [rank, rank + 1) x span.
__global__ void __launch_bounds__(kSelThreads)
k_evict_select(const float* __restrict__ weights, const int32_t* lengths, int max_len, int budget, int sink,
               int recent, int32_t* __restrict__ src, int32_t* __restrict__ new_len, int32_t* dst_lengths,
               int32_t* kept, int32_t* __restrict__ status, int CS) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  __shared__ __align__(8) uint32_t hist[3][kBins];
  __shared__ uint32_t red[2][32];
  int turn = 0;   // of red's halves
  __shared__ uint32_t found[2];    // digit, count above it
  __shared__ uint32_t counts[2];   // this CTA's rows above the threshold (or kept anyway), and equal to it
  const int b = int(blockIdx.x) / CS, tid = threadIdx.x;
  const uint32_t rank = CS > 1 ? cluster_rank() : 0u;
  const int n = dev::clamp_len(lengths[b], max_len, tid == 0 && rank == 0 ? status : nullptr);
  const float* w = weights + size_t(b) * max_len;
  int32_t* sb = src + size_t(b) * budget;
  int32_t* kb = kept ? kept + size_t(b) * budget : nullptr;
  const int m = min(n, budget);
  for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[0][i] = 0;
  // every thread has read the length before dst_lengths, which may be the same array, is written
  if (CS > 1) cluster_sync(); else __syncthreads();
  if (tid == 0 && rank == 0) {
    new_len[b] = m;
    dst_lengths[b] = m;
  }
  const unsigned step = unsigned(CS) * kSelThreads, first = rank * kSelThreads + unsigned(tid);
  if (kb)
    for (unsigned j = unsigned(m) + first; j < unsigned(budget); j += step) kb[j] = -1;
  if (n <= budget) {   // uniform across the cluster
    for (unsigned j = first; j < unsigned(n); j += step) {
      sb[j] = int32_t(j);
      if (kb) kb[j] = int32_t(j);
    }
    return;
  }
  // this CTA's rows [r0, r1), the candidates [sink, n - recent) among them
  const unsigned span = (unsigned(n) + unsigned(CS) - 1) / unsigned(CS);
  const unsigned r0 = min(rank * span, unsigned(n)), r1 = min(r0 + span, unsigned(n));
  const unsigned lo = unsigned(sink), hi = unsigned(n - recent);
  const bool held = r1 - r0 <= unsigned(kSelChunk);   // one chunk: its keys stay in registers
  uint32_t key[kSelKeys];
  uint32_t cand = 0, fixed = 0;   // bit i: row c0 + 8 tid + i is a candidate; is kept whatever the weights
  auto load = [&](unsigned c0) {
    cand = fixed = 0;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      const unsigned t = c0 + unsigned(tid) * kSelKeys + i;
      const bool in = t < r1, mid = t >= lo && t < hi;
      cand |= uint32_t(in && mid) << i;
      fixed |= uint32_t(in && !mid) << i;
      key[i] = in && mid ? weight_key(__ldg(w + t)) : 0u;
    }
  };
  if (held) load(r0);
  // threshold: the K-th largest key of the candidates
  const bool some = budget > sink + recent;   // else the budget is all sink and recent
  uint32_t K = uint32_t(budget - sink - recent), prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3 && some; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1024u : 2048u;
    const int above = shift + (pass == 2 ? 10 : 11);   // bits decided before
    for (unsigned c0 = r0; c0 < r1; c0 += kSelChunk) {
      if (!held) load(c0);
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i)
        if ((cand >> i & 1u) && (pass == 0 || (key[i] >> above) == (prefix >> above)))
          atomicAdd(&hist[pass][(key[i] >> shift) & (digits - 1)], 1u);
    }
    if (CS > 1) cluster_sync(); else __syncthreads();
    // thread i sees to bins 2 (1023 - i) + 1 and 2 (1023 - i): counted from the top, over the cluster
    const int bin = 2 * (kSelThreads - 1 - tid);
    uint32_t top = 0, low = 0;
    if (CS > 1) {
      unsigned long long v[kMaxCluster];   // both bins of every CTA, the loads in flight together
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) v[c] = c < CS ? peer_pair(&hist[pass][bin], uint32_t(c)) : 0ull;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        top += uint32_t(v[c] >> 32);
        low += uint32_t(v[c]);
      }
    } else {
      top = hist[pass][bin + 1];
      low = hist[pass][bin];
    }
    uint32_t total;
    const uint32_t before = cta_exclusive(top + low, red[turn ^= 1], &total);
    if (before < K && K <= before + top + low) {   // one thread, the same in every CTA
      const bool upper = K <= before + top;
      found[0] = uint32_t(bin + (upper ? 1 : 0));
      found[1] = before + (upper ? 0u : top);
    }
    __syncthreads();
    prefix |= found[0] << shift;
    K -= found[1];   // still to take among the keys equal so far
  }
  // The K lowest rows equal to the threshold are taken.  Bits of the thread's
  // rows kept whatever the others are, and of those equal.
  auto sort_out = [&](uint32_t* above, uint32_t* equal) {
    *above = fixed;
    *equal = 0;
    if (!some) return;
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) {
      *above |= (cand & (uint32_t(key[i] > prefix) << i));
      *equal |= (cand & (uint32_t(key[i] == prefix) << i));
    }
  };
  unsigned out = 0, eq = 0;   // kept rows and equal rows before this CTA's
  if (CS > 1) {
    unsigned na = 0, ne = 0;
    for (unsigned c0 = r0; c0 < r1; c0 += kSelChunk) {
      if (!held) load(c0);
      uint32_t above, equal;
      sort_out(&above, &equal);
      na += __popc(above);
      ne += __popc(equal);
    }
    if (tid < 2) counts[tid] = 0;
    __syncthreads();
    na = __reduce_add_sync(0xffffffffu, na);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if ((tid & 31) == 0) {
      atomicAdd(&counts[0], na);
      atomicAdd(&counts[1], ne);
    }
    cluster_sync();
    for (uint32_t c = 0; c < rank; ++c) {
      const uint32_t e = peer_word(&counts[1], c);
      out += peer_word(&counts[0], c) + min(e, K - min(K, eq));
      eq += e;
    }
  }
  for (unsigned c0 = r0; c0 < r1; c0 += kSelChunk) {
    if (!held) load(c0);
    uint32_t above, equal;
    sort_out(&above, &equal);
    uint32_t all;   // 16 bits each: rows above, rows equal (a chunk has 8192)
    const uint32_t before = cta_exclusive((uint32_t(__popc(above)) << 16) + uint32_t(__popc(equal)), red[turn ^= 1], &all);
    const unsigned left = K - min(K, eq);   // equal rows still to take at the chunk's start
    unsigned a = before >> 16, e = before & 0xFFFFu;
    for (uint32_t rest = above | equal; rest; rest &= rest - 1) {
      const int i = __ffs(rest) - 1;
      const bool ab = above >> i & 1u;
      if (ab || e < left) {
        const unsigned at = out + a + min(e, left);
        const int32_t t = int32_t(c0 + unsigned(tid) * kSelKeys + i);
        sb[at] = t;
        if (kb) kb[at] = t;
      }
      a += ab;
      e += !ab;
    }
    out += (all >> 16) + min(all & 0xFFFFu, left);
    eq += all & 0xFFFFu;
  }
  if (CS > 1) cluster_sync();   // no CTA leaves while another may read its counts
}

constexpr int kMvThreads = 256;
constexpr int kMvUnroll = 8;   // loads in flight per thread

// The rows' group scales (ng 2-byte words each) and weights of sequence b, in
// ordered chunks; weights behind the new length become 0.  One CTA.
__device__ void move_small(const uint16_t* scales, uint16_t* dst_scales, int ng, const float* weights,
                           float* dst_weights, const int32_t* sb, int b, int m, int max_len, int dst_max_len) {
  constexpr int U = kMvUnroll;
  if (dst_scales) {
    const uint16_t* s0 = scales + size_t(b) * max_len * ng;
    uint16_t* d0 = dst_scales + size_t(b) * dst_max_len * ng;
    // thread = word g of rows j0 + its row: 256 / ng rows at a time (ng <= 256)
    const int rows = kMvThreads / ng, row = int(threadIdx.x) / ng, g = int(threadIdx.x) % ng;
    for (long long j0 = 0; j0 < m; j0 += rows * U) {
      uint16_t x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * rows + row;
        if (row < rows && j < m)
          asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(x[i]) : "l"(s0 + size_t(sb[j]) * ng + g) : "memory");
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * rows + row;
        if (row < rows && j < m) d0[size_t(j) * ng + g] = x[i];
      }
    }
  }
  if (dst_weights) {
    const float* s0 = weights + size_t(b) * max_len;
    float* d0 = dst_weights + size_t(b) * dst_max_len;
    for (long long j0 = 0; j0 < m; j0 += kMvThreads * U) {
      float x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * kMvThreads + threadIdx.x;
        if (j < m) asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x[i]) : "l"(s0 + sb[j]) : "memory");
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * kMvThreads + threadIdx.x;
        if (j < m) d0[j] = x[i];
      }
    }
    __syncthreads();   // in place: the last rows are read before they are zeroed
    for (long long j = m + int(threadIdx.x); j < dst_max_len; j += kMvThreads) d0[j] = 0.f;
  }
}

__device__ __forceinline__ uint4 ld_cg(const uint8_t* p) {
  uint4 x;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p) : "memory");
  return x;
}

struct MoveArgs {
  const uint8_t* rows;
  uint8_t* dst_rows;
  const uint16_t* scales;
  uint16_t* dst_scales;     // null: none
  const float* weights;
  float* dst_weights;       // null: none
  const int32_t *src, *new_len;
  int vecs, ng, max_len, dst_max_len, budget;
};

// Rows of 16-byte vectors.  grid (1 + walkers, B), block 256; the first CTA
// of a sequence moves its scales and weights.
//   in place: walker = column slice of 1 << ws vectors, chunks of (256 >> ws) x 8 rows in order
//   else:     walkers share the sequence's (row, vector) pairs in chunks of 2048, row after row
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMvThreads)
k_evict_move(const MoveArgs a, int ws) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  const int b = blockIdx.y, m = a.new_len[b];
  const int32_t* sb = a.src + size_t(b) * a.budget;
  if (blockIdx.x == 0) {
    move_small(a.scales, a.dst_scales, a.ng, a.weights, a.dst_weights, sb, b, m, a.max_len, a.dst_max_len);
    return;
  }
  const int walker = int(blockIdx.x) - 1;
  const size_t rb = size_t(a.vecs) * 16;
  const uint8_t* s0 = a.rows + size_t(b) * a.max_len * rb;
  uint8_t* d0 = a.dst_rows + size_t(b) * a.dst_max_len * rb;
  if (IN_PLACE) {
    const int v = (walker << ws) + (int(threadIdx.x) & ((1 << ws) - 1));
    const int rows = kMvThreads >> ws, row = int(threadIdx.x) >> ws, chunk = rows * kMvUnroll;
    const bool mine = v < a.vecs;
    s0 += size_t(v) * 16;
    d0 += size_t(v) * 16;
    // the first chunk with a row that moves: src[j] >= j, increasing, so a
    // chunk whose last row stays does so whole, and all before it
    const int chunks = int(((long long)m + chunk - 1) / chunk);
    int k0 = 0;
    for (int hi = chunks; k0 < hi;) {   // uniform
      const int mid = (k0 + hi) >> 1, last = int(min((long long)m, (long long)(mid + 1) * chunk)) - 1;
      if (sb[last] == last) k0 = mid + 1; else hi = mid;
    }
    // The next chunk's rows load while this one's are stored (what this one
    // stores no later chunk reads), their indices one chunk earlier still; the
    // barrier puts every thread's loads of a chunk before any of its stores.
    int at[kMvUnroll];
    auto index = [&](int k) {
#pragma unroll
      for (int i = 0; i < kMvUnroll; ++i) {
        const long long j = (long long)k * chunk + i * rows + row;
        at[i] = j < m ? __ldg(sb + j) : -1;
      }
    };
    auto load = [&](uint4 (&x)[kMvUnroll]) {
#pragma unroll
      for (int i = 0; i < kMvUnroll; ++i)
        if (mine && at[i] >= 0) x[i] = ld_cg(s0 + size_t(at[i]) * rb);
    };
    auto store = [&](int k, const uint4 (&x)[kMvUnroll]) {
#pragma unroll
      for (int i = 0; i < kMvUnroll; ++i) {
        const long long j = (long long)k * chunk + i * rows + row;
        if (mine && j < m) *reinterpret_cast<uint4*>(d0 + size_t(j) * rb) = x[i];
      }
    };
    uint4 x0[kMvUnroll], x1[kMvUnroll];
    index(k0);
    load(x0);
    index(k0 + 1);
    for (int k = k0; k < chunks; k += 2) {
      load(x1);        // chunk k + 1 (no row past the last chunk: its indices are -1)
      index(k + 2);
      __syncthreads();
      store(k, x0);
      if (k + 1 >= chunks) break;
      load(x0);
      index(k + 3);
      __syncthreads();
      store(k + 1, x1);
    }
  } else {
    const unsigned long long total = (unsigned long long)m * a.vecs;
    const unsigned long long stride = (unsigned long long)(gridDim.x - 1) * (kMvThreads * kMvUnroll);
    const unsigned vecs = unsigned(a.vecs);
    for (unsigned long long e0 = (unsigned long long)walker * (kMvThreads * kMvUnroll); e0 < total; e0 += stride) {
      const unsigned long long j0 = e0 / vecs;                 // row of the chunk's start: the only wide division
      const unsigned v0 = unsigned(e0 - j0 * vecs);
      uint4 x[kMvUnroll];
#pragma unroll
      for (int i = 0; i < kMvUnroll; ++i) {
        const unsigned e = v0 + i * kMvThreads + threadIdx.x, j = e / vecs;
        if (j0 + j < (unsigned long long)m) x[i] = ld_cg(s0 + size_t(sb[j0 + j]) * rb + size_t(e - j * vecs) * 16);
      }
#pragma unroll
      for (int i = 0; i < kMvUnroll; ++i) {
        const unsigned e = v0 + i * kMvThreads + threadIdx.x;
        if (j0 + e / vecs < (unsigned long long)m) *reinterpret_cast<uint4*>(d0 + size_t(j0) * rb + size_t(e) * 16) = x[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const qsvd_dims& d, const float* weights, const int32_t* lengths, int budget, int sink,
                         int recent, const void* cache, const void* scales, int dst_max_len, void* dst_cache,
                         void* dst_scales, float* dst_weights, int32_t* dst_lengths, int32_t* kept, int32_t* src,
                         int32_t* new_len, int32_t* status, cudaStream_t s) {
  // one CTA per 4096 rows of the longest sequence, a power of two up to eight
  int CS = 1;
  while (CS < kMaxCluster && (long long)CS * (kSelChunk / 2) < d.max_len) CS *= 2;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned(d.batch) * unsigned(CS));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(CS);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_select, weights, lengths, d.max_len, budget, sink, recent, src,
                                     new_len, dst_lengths, kept, status, CS);
  if (e != cudaSuccess) return e;
  note_launch();
  if ((e = check_launch()) != cudaSuccess) return e;
  const bool q = cache_is_int(d), in_place = cache == dst_cache;
  const MoveArgs a{static_cast<const uint8_t*>(cache), static_cast<uint8_t*>(dst_cache),
                   static_cast<const uint16_t*>(scales), static_cast<uint16_t*>(q ? dst_scales : nullptr), weights,
                   dst_weights, src, new_len, int(cache_row_bytes(d) / 16), q ? d.r / d.group : 1, d.max_len,
                   dst_max_len, budget};
  int ws = 0;
  long long walkers;
  if (in_place) {
    // slices of 512 bytes, narrower ones where those are too few for the SMs, down to a sector of 32
    const int sms = device_sms();
    for (ws = 5; ws > 1 && (long long)((a.vecs + (1 << ws) - 1) >> ws) * d.batch < sms; --ws) {}
    walkers = (a.vecs + (1 << ws) - 1) >> ws;
  } else {
    walkers = ((long long)budget * a.vecs + kMvThreads * kMvUnroll - 1) / (kMvThreads * kMvUnroll);
    if (walkers > (1 << 20)) walkers = 1 << 20;
  }
  e = launch_pdl(in_place ? k_evict_move<true> : k_evict_move<false>, dim3(unsigned(1 + walkers), unsigned(d.batch)),
                 dim3(kMvThreads), 0, s, a, ws);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

}  // namespace qsvd
