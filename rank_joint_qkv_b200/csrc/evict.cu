// Cutting caches to a budget of rows by accumulated attention weight.
//
// A sequence with n > budget rows keeps its first `sink` rows, its last
// `recent` rows and, of the rows between, the budget - sink - recent heaviest
// (equal weights: the lower row first; a NaN weighs less than anything); the
// kept rows stay in order.  Two steps:
//
//   k_evict_select  the kept rows of each sequence, in order: the K-th
//                   heaviest key by radix selection (weights mapped to
//                   integers of the same order, three digits of 11, 11 and 10
//                   bits, a shared-memory histogram each), then one pass that
//                   compacts the rows above it and the first of those equal
//   k_evict_move    the rows' bytes (and k_evict_small their scales and
//                   weights): bound by HBM, each kept row read and written once
//
// In place the move has an order to keep: row j of the result is row
// src[j] >= j of the source, src increasing.  A CTA owns a column slice of a
// sequence and walks the rows in chunks, the whole chunk read before any of
// it is written: what chunk k writes, rows below its end, no later chunk
// reads, since src[j] >= j.
#include "internal.cuh"

namespace qsvd {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// Order-preserving integer of a weight; NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the CTA's threads; *total: the sum.  red: 33 words.
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
  if (warp == 0) {
    uint32_t y = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    red[lane] = y;
  }
  __syncthreads();
  const uint32_t before = warp ? red[warp - 1] : 0u;
  *total = red[31];
  __syncthreads();   // red is reused by the next call
  return before + x - v;
}

// grid B, block 1024.
__global__ void __launch_bounds__(kSelThreads)
k_evict_select(const float* __restrict__ weights, const int32_t* lengths, int max_len, int budget, int sink,
               int recent, int32_t* __restrict__ src, int32_t* __restrict__ new_len, int32_t* dst_lengths,
               int32_t* kept, int32_t* __restrict__ status) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t red[33];
  __shared__ uint32_t found[2];   // digit, count above it
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = dev::clamp_len(lengths[b], max_len, tid == 0 ? status : nullptr);
  const float* w = weights + size_t(b) * max_len;
  int32_t* sb = src + size_t(b) * budget;
  int32_t* kb = kept ? kept + size_t(b) * budget : nullptr;
  const int m = min(n, budget);
  __syncthreads();   // every thread has read the length: dst_lengths may be the same array
  if (tid == 0) {
    new_len[b] = m;
    dst_lengths[b] = m;
  }
  if (kb)
    for (unsigned j = unsigned(m + tid); j < unsigned(budget); j += kSelThreads) kb[j] = -1;
  if (n <= budget) {
    for (unsigned j = unsigned(tid); j < unsigned(n); j += kSelThreads) {
      sb[j] = int32_t(j);
      if (kb) kb[j] = int32_t(j);
    }
    return;
  }
  // threshold: the K-th largest key of rows [sink, n - recent)
  const int lo = sink, hi = n - recent;
  uint32_t K = uint32_t(budget - sink - recent), prefix = 0;
  if (K > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1024u : 2048u;
      const int above = shift + (pass == 2 ? 10 : 11);   // bits decided before
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (unsigned t = unsigned(lo + tid); t < unsigned(hi); t += kSelThreads) {   // past 2^31 without wrapping
        const uint32_t k = weight_key(w[t]);
        if (pass == 0 || (k >> above) == (prefix >> above)) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1u);
      }
      __syncthreads();
      // thread i holds the bins 2 (1023 - i) + 1 and 2 (1023 - i): counted from the top
      const uint32_t top = hist[2 * (kSelThreads - 1 - tid) + 1], low = hist[2 * (kSelThreads - 1 - tid)];
      uint32_t total;
      const uint32_t before = cta_exclusive(top + low, red, &total);
      if (before < K && K <= before + top + low) {
        const bool first = K <= before + top;
        found[0] = uint32_t(2 * (kSelThreads - 1 - tid) + (first ? 1 : 0));
        found[1] = before + (first ? 0u : top);
      }
      __syncthreads();
      prefix |= found[0] << shift;
      K -= found[1];   // still to take among the keys equal so far
      __syncthreads();
    }
  }
  // K rows equal to the threshold are taken, the lowest first; none when the budget is all sink and recent
  const bool some = budget > sink + recent;
  uint32_t taken_eq = 0, out = 0;
  for (unsigned t0 = 0; t0 < unsigned(n); t0 += kSelThreads) {
    const unsigned t = t0 + unsigned(tid);
    const bool mid = t >= unsigned(lo) && t < unsigned(hi);
    const uint32_t k = mid ? weight_key(w[t]) : 0u;
    const bool eq = some && mid && k == prefix;
    uint32_t neq, nkeep;
    const uint32_t eq_before = cta_exclusive(eq ? 1u : 0u, red, &neq);
    const bool keep = t < unsigned(n) && (!mid || (some && (k > prefix || (eq && taken_eq + eq_before < K))));
    const uint32_t at = cta_exclusive(keep ? 1u : 0u, red, &nkeep);
    if (keep) {
      sb[out + at] = int32_t(t);
      if (kb) kb[out + at] = int32_t(t);
    }
    taken_eq += neq;
    out += nkeep;
  }
}

constexpr int kMvThreads = 256;
constexpr int kMvUnroll = 8;   // 16-byte loads in flight per thread

// Rows of 16-byte vectors.  A CTA owns the vectors [slice << ws, +1 << ws) of
// sequence b's rows and walks their chunks of (256 >> ws) x 8 rows from
// blockIdx.z on in steps of gridDim.z (1 in place: the order above).
// grid (slices, B, chunk walkers), block 256.
__global__ void __launch_bounds__(kMvThreads)
k_evict_move(const uint8_t* src_rows, uint8_t* dst_rows, const int32_t* __restrict__ src,
             const int32_t* __restrict__ new_len, int vecs, int ws, int max_len, int dst_max_len, int budget,
             int in_place) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  const int b = blockIdx.y, m = new_len[b];
  const int32_t* sb = src + size_t(b) * budget;
  const int v = (int(blockIdx.x) << ws) + (int(threadIdx.x) & ((1 << ws) - 1));
  const int rows = kMvThreads >> ws, row = int(threadIdx.x) >> ws;
  const size_t rb = size_t(vecs) * 16;
  const uint8_t* s0 = src_rows + size_t(b) * max_len * rb + size_t(v) * 16;
  uint8_t* d0 = dst_rows + size_t(b) * dst_max_len * rb + size_t(v) * 16;
  const int chunk = rows * kMvUnroll;
  const bool mine = v < vecs;
  for (long long j0 = (long long)blockIdx.z * chunk; j0 < m; j0 += (long long)gridDim.z * chunk) {
    const int last = int(min((long long)m, j0 + chunk)) - 1;
    if (in_place && sb[last] == last) continue;   // src[j] >= j, increasing: the whole chunk stays (uniform)
    uint4 x[kMvUnroll];
#pragma unroll
    for (int i = 0; i < kMvUnroll; ++i) {
      const long long j = j0 + i * rows + row;
      if (mine && j <= last) {
        const uint8_t* p = s0 + size_t(sb[j]) * rb;
        asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w) : "l"(p) : "memory");
      }
    }
    if (in_place) __syncthreads();
#pragma unroll
    for (int i = 0; i < kMvUnroll; ++i) {
      const long long j = j0 + i * rows + row;
      if (mine && j <= last) *reinterpret_cast<uint4*>(d0 + size_t(j) * rb) = x[i];
    }
  }
}

constexpr int kSmThreads = 512;

// The rows' group scales (ng 2-byte words each) and weights, in the same
// ordered chunks; weights behind the new length become 0.  grid B, block 512.
__global__ void __launch_bounds__(kSmThreads)
k_evict_small(const uint16_t* scales, uint16_t* dst_scales, int ng, const float* weights, float* dst_weights,
              const int32_t* __restrict__ src, const int32_t* __restrict__ new_len, int max_len, int dst_max_len,
              int budget) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  const int b = blockIdx.x, m = new_len[b];
  const int32_t* sb = src + size_t(b) * budget;
  constexpr int U = 8;
  if (dst_scales) {
    const uint16_t* s0 = scales + size_t(b) * max_len * ng;
    uint16_t* d0 = dst_scales + size_t(b) * dst_max_len * ng;
    const long long total = (long long)m * ng;
    for (long long e0 = 0; e0 < total; e0 += kSmThreads * U) {
      uint16_t x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long e = e0 + i * kSmThreads + threadIdx.x;
        if (e < total) {
          const int j = int(e / ng), g = int(e % ng);
          asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(x[i]) : "l"(s0 + size_t(sb[j]) * ng + g) : "memory");
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long e = e0 + i * kSmThreads + threadIdx.x;
        if (e < total) d0[e] = x[i];
      }
    }
  }
  if (dst_weights) {
    const float* s0 = weights + size_t(b) * max_len;
    float* d0 = dst_weights + size_t(b) * dst_max_len;
    for (long long j0 = 0; j0 < m; j0 += kSmThreads * U) {
      float x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * kSmThreads + threadIdx.x;
        if (j < m) asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x[i]) : "l"(s0 + sb[j]) : "memory");
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long j = j0 + i * kSmThreads + threadIdx.x;
        if (j < m) d0[j] = x[i];
      }
    }
    __syncthreads();   // in place: the last rows are read before they are zeroed
    for (long long j = m + int(threadIdx.x); j < dst_max_len; j += kSmThreads) d0[j] = 0.f;
  }
}

}  // namespace

cudaError_t launch_evict(const qsvd_dims& d, const float* weights, const int32_t* lengths, int budget, int sink,
                         int recent, const void* cache, const void* scales, int dst_max_len, void* dst_cache,
                         void* dst_scales, float* dst_weights, int32_t* dst_lengths, int32_t* kept, int32_t* src,
                         int32_t* new_len, int32_t* status, cudaStream_t s) {
  cudaError_t e = launch_pdl(k_evict_select, dim3(unsigned(d.batch)), dim3(kSelThreads), 0, s, weights, lengths,
                             d.max_len, budget, sink, recent, src, new_len, dst_lengths, kept, status);
  if (e != cudaSuccess) return e;
  note_launch();
  if ((e = check_launch()) != cudaSuccess) return e;
  const int vecs = int(cache_row_bytes(d) / 16);
  const int in_place = cache == dst_cache;
  int ws = 3;   // 128-byte slices; in place narrower ones where there are too few to fill the GPU
  while (in_place && ws > 1 && (long long)((vecs + (1 << ws) - 1) >> ws) * d.batch < 296) --ws;
  const int slices = (vecs + (1 << ws) - 1) >> ws;
  const int chunk = (kMvThreads >> ws) * kMvUnroll;
  long long walkers = in_place ? 1 : (budget + chunk - 1) / chunk;
  if (walkers > 65535) walkers = 65535;
  e = launch_pdl(k_evict_move, dim3(unsigned(slices), unsigned(d.batch), unsigned(walkers)), dim3(kMvThreads), 0, s,
                 static_cast<const uint8_t*>(cache), static_cast<uint8_t*>(dst_cache), src, new_len, vecs, ws,
                 d.max_len, dst_max_len, budget, in_place);
  if (e != cudaSuccess) return e;
  note_launch();
  if ((e = check_launch()) != cudaSuccess) return e;
  if (!dst_weights && !cache_is_int(d)) return cudaSuccess;
  e = launch_pdl(k_evict_small, dim3(unsigned(d.batch)), dim3(kSmThreads), 0, s, static_cast<const uint16_t*>(scales),
                 static_cast<uint16_t*>(cache_is_int(d) ? dst_scales : nullptr),
                 cache_is_int(d) ? d.r / d.group : 1, weights, dst_weights, src, new_len, d.max_len, dst_max_len,
                 budget);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

}  // namespace qsvd
