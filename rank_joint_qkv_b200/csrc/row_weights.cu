// Attention weight of each cache row, summed over the heads, from the scores
// the split phase kept and the merged softmax statistics:
//
//   w_t (+)= sum_h 2^(s_{h,t} - M_h) / L_h   (log2 domain; M and L from the merge)
//
// the quantity by which rows of a cache are kept or dropped.  It reads the
// scores once, 4 H bytes per row (16.8 MB at LLaVA-7B shapes, B 16, L 8192),
// just written by the split kernel and so mostly in L2: 7.8 us alone, most of
// it under the value up-projection, beside which it runs.  Forming the weights
// by a second pass over the latent instead would read 403 MB again, 62 us.
#include "internal.cuh"

namespace qsvd {
namespace {

constexpr int kRwThreads = 256;
constexpr int kRwHeads = 1024;   // heads' statistics held at a time

// grid (ceil(max_len / 256), B), block 256: thread = row; 1024 heads at a time.
// Runs beside the value up-projection (see launch_pdl): it reads what the
// merge and the split phase wrote, and the up-projection's CTAs have waited
// for the merge before this kernel starts.
__global__ void __launch_bounds__(kRwThreads)
k_row_weights(const int32_t* __restrict__ sched, const float2* __restrict__ ml, const float* __restrict__ scores,
              float* __restrict__ w, int add, int B, int H, int max_len) {
  __shared__ float2 stat[kRwHeads];
  const int b = blockIdx.y;
  const long long t = (long long)blockIdx.x * kRwThreads + threadIdx.x;
  const int n = sched[B + 1 + b];
  if (t - threadIdx.x < n) {   // uniform across the CTA
    float acc = 0.f;
    for (int h0 = 0; h0 < H; h0 += kRwHeads) {
      const int nh = min(kRwHeads, H - h0);
      if (h0) __syncthreads();   // every thread is done with the heads before
      for (int h = threadIdx.x; h < nh; h += kRwThreads) stat[h] = __ldcg(ml + size_t(b) * H + h0 + h);
      __syncthreads();
      if (t >= n) continue;
      const float* sc = scores + (size_t(b) * H + h0) * max_len + t;
      int h = 0;
      for (; h + 16 <= nh; h += 16) {   // sixteen loads in flight, added in head order
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __ldcg(sc + size_t(h + i) * max_len);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc = fmaf(exp2f(v[i] - stat[h + i].x), stat[h + i].y, acc);
      }
      for (; h < nh; ++h) acc = fmaf(exp2f(__ldcg(sc + size_t(h) * max_len) - stat[h].x), stat[h].y, acc);
    }
    if (t < n) {
      float* o = w + size_t(b) * max_len + t;
      *o = add ? *o + acc : acc;
    }
  }
  dev::pdl_wait();
  dev::pdl_trigger();
}

}  // namespace

cudaError_t launch_row_weights(const qsvd_dims& d, const int32_t* sched, const float2* ml, const float* scores,
                               float* w, int add, cudaStream_t s) {
  const dim3 grid(unsigned((d.max_len + kRwThreads - 1) / kRwThreads), unsigned(d.batch));
  const cudaError_t e = launch_pdl(k_row_weights, grid, dim3(kRwThreads), 0, s, sched,
                                   ml, scores, w, add, d.batch, d.H, d.max_len);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

}  // namespace qsvd
