// Decode attention of a whole batch over a prefix that its sequences share
// (absorbed query): the latent rows c_0 .. c_{P-1} are stored once, and all B
// sequences' H heads read them in one pass as B H query rows,
//
//   S = Qt C^T  (B H x P, K = r)     P = 2^(S - m)     Z = P C  (B H x r, K = P)
//
// 4 B H r P flops for P r values read: with tens of sequences both products
// are bound by the tensor cores, not by HBM as the per-sequence decode is.
// The accumulator of Z alone is r columns per 128 query rows, three times
// TMEM at r 1536, so the two products are two kernels with P between them
// (16-bit, 2 B H P bytes: 8 MB at B 16, H 32, P 8192, within L2) rather than
// one that keeps a tile's scores on chip:
//
//   k_prefix_gemm<scores>   128 query rows x 256 tokens per unit; the epilogue
//                           (thread = query row) takes the tile's maximum,
//                           writes 2^(s - ref) and keeps ref and the sum
//   k_prefix_norm           per row and token split: the reference of the
//                           split's tiles made one, m and l of the split (not
//                           needed where each split is one tile); 5 us of
//                           latency at B 16, H 32, P 8192
//   k_prefix_gemm<values>   128 query rows x 256 channels per unit over a
//                           split's tokens; float32 partials for the merge
//
// A tile's reference is its maximum rounded down to a multiple of 15 (log2
// units): P < 2^15 is within fp16, and a row's tiles mostly share it, so that
// k_prefix_norm rewrites few of them (a multiple of 8, the split kernels'
// bound, lies in the middle of 256 scores' usual maxima); where it does, the
// factor is a power of two and the only loss is a fp16 subnormal's.
//
// Precision as in the split kernels: the query as two 16-bit parts (three of
// bf16's where weights are asked for; the products accumulate in float32), P as
// two for bf16; a quantised prefix is
// expanded to the fp16 hi and lo parts of code x scale (18 bits: exact up to
// 65,504), each a pass of both products, and its query parts are scaled by a
// power of two per (sequence, head) (k_quant_query), so that the scores are as
// good as the integer ones of the sequences' own rows whatever the query's size.
// One fp16 part of P (each weight within 2^-11) under an unrounded sum is what
// outputs of fp16 and quantised rows mostly differ by from 32-bit ones; a second
// part would double the values' product (17 of 101 us at B 16, P 8192, 74 of
// 400 at B 64, P 16384).
//
// Measured at B 64, H 32, r 1536 over 16,384 fp16 rows (206 and 103 GFLOP with
// the query's two parts counted): scores 137 us, 1.50 PFLOP/s, values 74 us,
// 1.39 PFLOP/s -- 0.92 and 0.85 of what a library GEMM of bf16 reaches here, at
// a clock that the power cap holds near 1.5 GHz.  What is left beside them is
// the second product of the query's residual: one fp16 part alone (2^-11 at
// most per channel) would move attention weights by some 1e-4 of themselves.
//
// Roles (320 threads per CTA): warp 0 TMA producer, warp 1 TMEM and the MMA thread,
// warps 2-9 epilogue; two TMEM accumulators of 256 columns, so the epilogue
// of a unit runs under the next one's products.  Every wait is bounded.
#include <cuda.h>

#include <cstring>

#include "internal.cuh"
#include "prefix.cuh"
#include "wsvd.cuh"
#include "tc_common.cuh"

namespace qsvd {
namespace {

constexpr int kPxThreads = 320;
constexpr int kPxEpi = 256;                // epilogue threads: two warps per 32 TMEM lanes, half of the columns each
constexpr int kPxA = 128 * 128;            // A box: 128 rows x 64 K x 2 bytes
constexpr int kPxB = 256 * 128;            // B: 256 N x 64 K x 2 bytes
constexpr int kPxMaxSlots = 6;
constexpr int kPxStage = 32 * 128;         // epilogue staging per warp: 32 rows x 128 bytes
constexpr float kRefStep = 15.f;           // log2 units between references
constexpr int kPxSmem = 232448;            // opt-in dynamic shared memory per block on sm_100

// One ring slot per CTA, and slots in 192 KB.  A CTA of a pair holds its own
// 128 query rows and half of B.
template <int AP, bool PAIR>
__host__ __device__ constexpr int px_slot() { return AP * kPxA + (PAIR ? kPxB / 2 : kPxB); }
template <int AP, bool PAIR>
__host__ __device__ constexpr int px_slots() { return 192 * 1024 / px_slot<AP, PAIR>(); }

struct PxArgs {
  int B, H, r, plen, nb, MB, tiles, ppad, SP;
  void* p;        // [AP parts][MB 128][ppad] P (scores: written)
  float* mt;      // [tiles][MB 128] reference of a tile ...
  float* lt;      // [tiles][MB 128] ... and the sum of its P
  float* pm;      // [SP B][H] instead of both, where every tile is a token
  float* pl;      // split of its own (tiles == SP)
  float* pz;      // [SP B][H][r] (values: written)
  float gain;     // on the scores (see launch_prefix)
  const float* qinv;   // [B][H] and the inverse of the query's scale (null: not scaled)
  int32_t* counter;   // score units taken (single CTAs)
  int32_t* status;
};

// Tiles [t0, t1) of token split sp.
__device__ __forceinline__ int split_tile(int sp, int tiles, int SP) { return int((long long)sp * tiles / SP); }

// PAIR: two CTAs of a cluster work on 256 query rows, each with its own 128 in
// its shared memory and TMEM and half of the B tile (tcgen05 cta_group::2;
// the first CTA issues): per 64 K of two A parts a CTA alone reads 64 KB from
// L2, one of a pair 48 KB (one A part: 48 KB, and 32 KB).
//
// The scores of single CTAs are dealt out as CTAs become free (a counter): they
// run beside the own rows' split kernel, whose CTAs hold their SMs for longer
// than a unit takes, and a fixed share would wait behind them.
//
// AP: 16-bit parts of A in pass 0 (a second pass, for the lo part of an
// expanded prefix, takes A's first part only).  CP: passes (parts of C).
// PS: parts of P that the scores' epilogue writes.
template <bool BF16, int AP, int CP, int PS, bool VALUES, bool PAIR>
__global__ void __launch_bounds__(kPxThreads, 1)
k_prefix_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b0,
              const __grid_constant__ CUtensorMap tm_b1, const PxArgs g) {
  if (VALUES) {
    dev::pdl_wait();   // see launch_pdl
    dev::pdl_trigger();
  }
  // (the scores run beside the own rows' split kernel before them in the
  // stream: its CTAs have waited for the query's parts, and nothing of its own
  // is read here; this kernel's wait is at its end)
  constexpr int kSlot = px_slot<AP, PAIR>(), ns = px_slots<AP, PAIR>();
  constexpr int W = PAIR ? 2 : 1;            // CTAs, and row blocks, per unit
  constexpr bool DYN = !VALUES && !PAIR;     // units by the counter
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* stage0 = base + size_t(ns) * kSlot;              // [8 warps][32 rows][128 bytes]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage0 + 8 * kPxStage);
  uint64_t* full = bars;                    // [kPxMaxSlots]
  uint64_t* empty = bars + kPxMaxSlots;     // [kPxMaxSlots]
  uint64_t* afull = bars + 2 * kPxMaxSlots; // [2] accumulator complete
  uint64_t* aempty = afull + 2;             // [2] accumulator read by the epilogue
  uint64_t* drain = aempty + 2;
  uint64_t* uq_full = drain + 1;            // [4] DYN: a unit published by the producer ...
  uint64_t* uq_empty = uq_full + 4;         // [4] ... and read by the MMA thread and the epilogue
  volatile int* uq = reinterpret_cast<volatile int*>(uq_empty + 4);   // [4]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(uq_empty + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NB = VALUES ? (g.r + 255) / 256 : g.tiles;       // column blocks of the product
  const int MU = (g.MB + W - 1) / W;                          // row blocks per column block, in units
  const int units = MU * NB * (VALUES ? g.SP : 1);
  const int walker = int(blockIdx.x) / W, walkers = int(gridDim.x) / W;
  const uint32_t rank = PAIR ? pair_rank() : 0u;
  // units of this CTA (at most, when they are dealt out)
  const int mine = DYN ? units : units > walker ? (units - 1 - walker) / walkers + 1 : 0;
  // unit u: row block(s) u % MU, so that the blocks in flight share their B
  // tiles in L2.  mb: this CTA's; the last pair's second may lie past MB (zeros)
  auto unit = [&](int u, int* mb, int* n, int* sp, int* k0, int* k1) {
    *mb = (u % MU) * W + int(rank);
    *n = (u / MU) % NB;
    *sp = (u / MU) / NB;
    if (VALUES) {   // 64-token blocks of the split's tiles
      *k0 = 4 * split_tile(*sp, g.tiles, g.SP);
      *k1 = min(4 * split_tile(*sp + 1, g.tiles, g.SP), (g.plen + 63) / 64);
    } else {
      *k0 = 0;
      *k1 = g.r / 64;
    }
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < ns; ++i) {
      mbar_init(saddr(&full[i]), 1);
      mbar_init(saddr(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(saddr(&afull[i]), 1);
      mbar_init(saddr(&aempty[i]), W);
    }
    mbar_init(saddr(drain), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(saddr(&uq_full[i]), 1);
      mbar_init(saddr(&uq_empty[i]), 2);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(tmem_holder))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(tmem_holder))
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
  }
  __syncthreads();
  if (PAIR) pair_sync();   // both CTAs' barriers and TMEM stand before either is used by the other
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t ring0 = saddr(base);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Ring rg(ns);
    long long k = 0;
    bool ok = true;
    for (int j = 0; j < mine && ok; ++j) {
      int u = walker + j * walkers;
      if (DYN) {
        if (j >= 4 && !__all_sync(0xffffffffu, mbar_wait(saddr(&uq_empty[j & 3]), uint32_t((j - 4) >> 2) & 1u))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          u = atomicAdd(g.counter, 1);
          uq[j & 3] = u;
          mbar_arrive(saddr(&uq_full[j & 3]));
        }
        u = __shfl_sync(0xffffffffu, u, 0);
        if (u >= units) break;
      }
      int mb, n, sp, k0, k1;
      unit(u, &mb, &n, &sp, &k0, &k1);
      for (int pass = 0; pass < CP && ok; ++pass) {
        const int parts = pass == 0 ? AP : 1;
        const uint32_t abytes = uint32_t(VALUES ? kPxA : g.nb * g.H * 128);
        for (int ki = k0; ki < k1; ++ki) {
          if (!__all_sync(0xffffffffu, mbar_wait(saddr(&empty[rg.slot]), rg.phase ^ 1u))) { ok = false; break; }
          const uint32_t dst = ring0 + uint32_t(rg.slot) * kSlot;
          const uint32_t fb = saddr(&full[rg.slot]);
          const int ln = int(k % 10) * 3;   // rotating issuing lanes, one per operation
          const CUtensorMap* tb = pass == 0 ? &tm_b0 : &tm_b1;
          const int part = lane - ln;
          if constexpr (PAIR) {
            // both CTAs' bytes are counted on the first's barrier, which its
            // MMA thread waits for
            if (rank == 0 && lane == 0) mbar_expect_tx(fb, 2u * parts * abytes + uint32_t(kPxB));
            __syncwarp();
            const uint32_t lb = pair_leader(fb);
            if (lane >= ln && lane < ln + parts) {
              if (VALUES) tma_load_3d(dst + part * kPxA, &tm_a, 64 * ki, mb * 128, part, lb, PairLoad());
              else tma_load_4d(dst + part * kPxA, &tm_a, 64 * ki, 0, part, mb * g.nb, lb, PairLoad());
            }
            if (lane == ln + 2) {
              if (VALUES) tma_load_3d(dst + AP * kPxA, tb, 0, 64 * ki, 4 * n + 2 * int(rank), lb, PairLoad());
              else tma_load_2d(dst + AP * kPxA, tb, 64 * ki, kPxTile * n + 128 * int(rank), lb, PairLoad());
            }
          } else {
            if (lane == 0) mbar_expect_tx(fb, parts * abytes + uint32_t(kPxB));
            __syncwarp();
            if (lane >= ln && lane < ln + parts) {
              if (VALUES) tma_load_3d(dst + part * kPxA, &tm_a, 64 * ki, mb * 128, part, fb);
              else tma_load_4d(dst + part * kPxA, &tm_a, 64 * ki, 0, part, mb * g.nb, fb);
            }
            if (lane == ln + 2) {
              if (VALUES) tma_load_3d(dst + AP * kPxA, tb, 0, 64 * ki, 4 * n, fb);
              else tma_load_2d(dst + AP * kPxA, tb, 64 * ki, kPxTile * n, fb);
            }
          }
          __syncwarp();
          rg.advance();
          ++k;
        }
      }
      if (__any_sync(0xffffffffu, *abort_flag)) ok = false;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(g.status, QSVD_STATUS_TIMEOUT);
      // copies in flight land before the CTA leaves (of a pair: on the first
      // CTA's barriers, and the second waits for it at the end)
      if (rank == 0)
        for (long long kk = (k > ns ? k - ns : 0); kk < k; ++kk)
          mbar_wait(saddr(&full[int(kk % ns)]), uint32_t(kk / ns) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = idesc_f16(128 * W, 256, BF16, false, VALUES);   // values: C is the MN-major operand
      const uint64_t da0 = sdesc(ring0, 16, 1024);                          // K-major
      const uint64_t db0 = sdesc(ring0 + AP * kPxA, VALUES ? 64 * 128 : 16, 1024);
      constexpr int kBStep = VALUES ? 16 * 128 : 32;                        // 16 tokens, or 16 channels
      Ring rg(ns);
      bool ok = true;
      for (int j = 0; j < mine && ok; ++j) {
        int u = walker + j * walkers;
        if (DYN) {
          if (!mbar_wait(saddr(&uq_full[j & 3]), uint32_t(j >> 2) & 1u)) { ok = false; break; }
          u = uq[j & 3];
          mbar_arrive(saddr(&uq_empty[j & 3]));
          if (u >= units) break;
        }
        int mb, n, sp, k0, k1;
        unit(u, &mb, &n, &sp, &k0, &k1);
        const int ab = j & 1;
        if (j >= 2 && !mbar_wait(saddr(&aempty[ab]), uint32_t((j - 2) >> 1) & 1u)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(ab * 256);
        uint32_t acc = 0;
        for (int pass = 0; pass < CP && ok; ++pass) {
          const int parts = pass == 0 ? AP : 1;
          for (int ki = k0; ki < k1; ++ki) {
            if (!mbar_wait(saddr(&full[rg.slot]), rg.phase)) { ok = false; break; }
            tc_fence_after();
            const uint64_t off = uint64_t((rg.slot * kSlot) >> 4);
            for (int part = 0; part < parts; ++part) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {   // K = 16 per MMA
                const uint64_t a = da0 + off + uint64_t((part * kPxA + kk * 32) >> 4);
                const uint64_t b = db0 + off + uint64_t((kk * kBStep) >> 4);
                if (PAIR) tc_mma_pair(d, a, b, id, acc);
                else tc_mma(d, a, b, id, acc);
                acc = 1;
              }
            }
            if (PAIR) tc_commit_pair(saddr(&empty[rg.slot]));
            else tc_commit(saddr(&empty[rg.slot]));
            rg.advance();
          }
        }
        if (!ok) break;
        if (PAIR) tc_commit_pair(saddr(&afull[ab]));
        else tc_commit(saddr(&afull[ab]));
        if (*abort_flag) ok = false;
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(g.status, QSVD_STATUS_TIMEOUT);
      }
      if (PAIR) tc_commit_pair(saddr(drain));
      else tc_commit(saddr(drain));
      mbar_wait(saddr(drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int t = 32 * q + lane;   // query row of the block == TMEM lane
    const int c_lo = 128 * half;   // this warp's columns [c_lo, c_lo + 128)
    const uint32_t lane_off = uint32_t(32 * q) << 16;
    const size_t rows = size_t(g.MB) * 128;
    // A lane holds a row's values; stored as they are, 16 bytes a lane, a store
    // instruction would touch 32 rows.  So the warp turns 32 rows x 128 bytes
    // around in shared memory (16-byte chunks, swizzled by row) and stores
    // four whole lines an instruction.
    const uint32_t st0 = saddr(stage0) + uint32_t(warp - 2) * kPxStage;
    const uint32_t mate0 = saddr(stage0) + uint32_t((warp - 2) ^ 4) * kPxStage;   // the same rows, the other columns
    auto put = [&](int c, uint4 v) {   // chunk c of this lane's row
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(st0 + lane * 128 + ((c ^ (lane & 7)) << 4)),
                   "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    };
    // the warp's 32 rows from row0 on; the rows' second halves `skip` bytes further
    auto flush = [&](uint8_t* row0, size_t skip, size_t pitch, int live_rows) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = 4 * i + (lane >> 3), c = lane & 7;
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(st0 + rr * 128 + ((c ^ (rr & 7)) << 4)) : "memory");
        if (32 * q + rr < live_rows)
          *reinterpret_cast<uint4*>(row0 + size_t(rr) * pitch + c * 16 + (c >= 4 ? skip : 0)) = v;
      }
      __syncwarp();
    };
    // this row's value in the other warp, through the two staging buffers (not in use)
    auto exchange = [&](float mine) {
      float other;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(st0 + lane * 4), "f"(mine) : "memory");
      bar_sync(1, kPxEpi);
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(mate0 + lane * 4) : "memory");
      bar_sync(1, kPxEpi);
      return other;
    };
    for (int j = 0; j < mine; ++j) {
      int u = walker + j * walkers;
      bool ok = true;
      if (DYN) {
        ok = mbar_wait(saddr(&uq_full[j & 3]), uint32_t(j >> 2) & 1u);
        u = ok ? uq[j & 3] : 0;
      }
      if (DYN && bar_or(!ok || u >= units, 1, kPxEpi)) {   // no unit is left (or the producer gave up)
        if (!ok && t == 0 && half == 0) { *abort_flag = 1; atomicOr(g.status, QSVD_STATUS_TIMEOUT); }
        break;
      }
      if (DYN && t == 0 && half == 0) mbar_arrive(saddr(&uq_empty[j & 3]));
      int mb, n, sp, k0, k1;
      unit(u, &mb, &n, &sp, &k0, &k1);
      const int ab = j & 1;
      const int fail = bar_or(!mbar_wait(saddr(&afull[ab]), uint32_t(j >> 1) & 1u), 1, kPxEpi);
      if (fail) {
        if (t == 0 && half == 0) { *abort_flag = 1; atomicOr(g.status, QSVD_STATUS_TIMEOUT); }
        break;
      }
      tc_fence_after();
      const int live_rows = min(g.nb, g.B - mb * g.nb) * g.H;   // rows of the block that are queries (none past MB)
      const uint32_t ta = tmem + lane_off + uint32_t(ab * 256);
      if (VALUES) {
        // rows mb nb H + t of the split's [B H][r]
        uint8_t* z = reinterpret_cast<uint8_t*>(g.pz + ((size_t(sp) * g.B + size_t(mb) * g.nb) * g.H + 32 * q) * g.r +
                                                size_t(n) * 256);
        const int nc = min(c_lo + 128, g.r - n * 256);   // a multiple of 64
#pragma unroll 1
        for (int c = c_lo; c < nc; c += 32) {
          float v[32];
          tmem_ld16(ta + uint32_t(c), v);
          tmem_ld16(ta + uint32_t(c + 16), v + 16);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            put(e, make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]),
                              __float_as_uint(v[4 * e + 3])));
          flush(z + c * 4, 0, size_t(g.r) * 4, live_rows);
        }
      } else {
        const int nv = min(kPxTile, g.plen - n * kPxTile);   // tokens of the tile, >= 1
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = c_lo; c < c_lo + 128; c += 32) {
          float v[32];
          tmem_ld16(ta + uint32_t(c), v);
          tmem_ld16(ta + uint32_t(c + 16), v + 16);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = c + e < nv ? fmaxf(mx, v[e]) : mx;
        }
        mx = fmaxf(mx, exchange(mx));
        const float gain = g.qinv && t < live_rows ? g.gain * __ldcg(g.qinv + size_t(mb) * g.nb * g.H + t) : g.gain;
        const float ref = kRefStep * floorf(mx * gain / kRefStep);
        float sum = 0.f;
        uint8_t* prow = reinterpret_cast<uint8_t*>(static_cast<T16*>(g.p) + (size_t(mb) * 128 + 32 * q) * g.ppad + size_t(n) * kPxTile);
        constexpr int kStep = PS == 2 ? 32 : 64;   // tokens staged at a time: hi parts, and lo parts beside them
#pragma unroll 1
        for (int c = c_lo; c < c_lo + 128; c += kStep) {
#pragma unroll
          for (int e32 = 0; e32 < kStep / 32; ++e32) {
            float v[32];
            tmem_ld16(ta + uint32_t(c + 32 * e32), v);
            tmem_ld16(ta + uint32_t(c + 32 * e32 + 16), v + 16);
            tmem_wait_ld();
#pragma unroll
            for (int e8 = 0; e8 < 4; ++e8) {
              uint4 hi, lo;
              T16* hv = reinterpret_cast<T16*>(&hi);
              T16* lv = reinterpret_cast<T16*>(&lo);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float p = c + 32 * e32 + 8 * e8 + e < nv ? exp2f(fmaf(v[8 * e8 + e], gain, -ref)) : 0.f;
                sum += p;
                hv[e] = dev::from_f<T16>(p);
                if (PS == 2) lv[e] = dev::from_f<T16>(p - dev::to_f(hv[e]));
              }
              put(4 * e32 + e8, hi);
              if (PS == 2) put(4 + e8, lo);
            }
          }
          // chunks 4-7: the next 32 tokens, or (PS == 2) the lo parts
          flush(prow + c * 2, PS == 2 ? rows * g.ppad * 2 - 64 : 0, size_t(g.ppad) * 2, live_rows);
        }
        sum += exchange(sum);   // the same two terms in both warps
        if (half == 0 && t < live_rows) {
          const bool own = g.tiles == g.SP;
          const size_t at = own ? (size_t(n) * g.B + size_t(mb) * g.nb) * g.H + t : size_t(n) * rows + size_t(mb) * 128 + t;
          (own ? g.pm : g.mt)[at] = ref;
          (own ? g.pl : g.lt)[at] = sum;
        }
      }
      tc_fence_before();
      bar_sync(1, kPxEpi);
      if (t == 0 && half == 0) {
        if (PAIR) pair_arrive(pair_leader(saddr(&aempty[ab])));
        else mbar_arrive(saddr(&aempty[ab]));
      }
      if (bar_or(*abort_flag, 1, kPxEpi)) break;
    }
  }
  if (!VALUES) {
    dev::pdl_wait();
    dev::pdl_trigger();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) pair_sync();   // no CTA of a pair leaves while the other's copies, MMAs or arrivals still reach it
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Per (query row, token split): m = the largest reference of the split's
// tiles, l = their sums brought to it, and P of the tiles with a lower one
// scaled to it.  A CTA has 32 rows, lane = row (whole lines of statistics); the
// split's tiles are shared out over its eight warps, a row's P to rescale taken
// by the whole warp.  Bound by the latency of its loads.
// grid (MB 4, SP), block 256.
template <typename T16, int PS>
__global__ void __launch_bounds__(256)
k_prefix_norm(T16* __restrict__ p, const float* __restrict__ mt, const float* __restrict__ lt, float* __restrict__ pm,
              float* __restrict__ pl, int B, int H, int nb, int MB, int tiles, int ppad, int SP) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  __shared__ float red[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mb = int(blockIdx.x) >> 2, i0 = 32 * (int(blockIdx.x) & 3), sp = blockIdx.y;
  const int live = min(nb, B - mb * nb) * H;   // rows of the block that are queries
  if (i0 >= live) return;   // uniform across the CTA
  const size_t rows = size_t(MB) * 128, row0 = size_t(mb) * 128 + i0;
  const bool mine = i0 + lane < live;
  const float* mr = mt + row0 + (mine ? lane : 0);
  const float* lr = lt + row0 + (mine ? lane : 0);
  const int t0 = split_tile(sp, tiles, SP) + warp, t1 = split_tile(sp + 1, tiles, SP);
  float m = -INFINITY;
#pragma unroll 4
  for (int t = t0; t < t1; t += 8) m = fmaxf(m, __ldcg(mr + size_t(t) * rows));
  red[0][warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, red[0][w][lane]);
  float l = 0.f;
#pragma unroll 4
  for (int t = t0; t < t1; t += 8) {
    const float f = exp2f(__ldcg(mr + size_t(t) * rows) - m);   // a power of two
    l = fmaf(f, __ldcg(lr + size_t(t) * rows), l);
    unsigned lower = __ballot_sync(0xffffffffu, mine && f != 1.f);
    while (lower) {
      const int i = __ffs(lower) - 1;
      lower &= lower - 1;
      const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
      for (int part = 0; part < PS; ++part) {
        uint4* v = reinterpret_cast<uint4*>(p + (part * rows + row0 + i) * ppad + size_t(t) * kPxTile) + lane;
        uint4 x = __ldcg(v);
        T16* e = reinterpret_cast<T16*>(&x);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = dev::from_f<T16>(dev::to_f(e[k]) * fi);
        *v = x;
      }
    }
  }
  red[1][warp][lane] = l;
  __syncthreads();
  if (warp == 0 && mine) {
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += red[1][w][lane];
    const size_t at = (size_t(sp) * B + size_t(mb) * nb) * H + i0 + lane;
    pm[at] = m;
    pl[at] = l;
  }
}

// Rotary mode: what the scores' epilogue does, from scores in memory
// [B][H][ppad].  Warp = (row, tile of 256 tokens), lane = 8 tokens.
// Bound by the scores read and P written, 6 B H P bytes (fp16), from L2.
// grid ceil(B H tiles / 8), block 256.
template <typename T16, int PS>
__global__ void __launch_bounds__(256)
k_prefix_probs(const float* __restrict__ scores, T16* __restrict__ p, float* __restrict__ mt, float* __restrict__ lt,
               int B, int H, int nb, int MB, int plen, int tiles, int ppad, bool own) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= (long long)B * H * tiles) return;
  const int tile = int(u % tiles), bh = int(u / tiles), b = bh / H, h = bh % H;
  const size_t rows = size_t(MB) * 128, row = size_t(b / nb) * 128 + (b % nb) * H + h;
  const int t0 = tile * kPxTile + 8 * lane;   // padded to ppad: loads stay inside the row
  float v[8];
  const float4* src = reinterpret_cast<const float4*>(scores + size_t(bh) * ppad + t0);
  *reinterpret_cast<float4*>(v) = __ldcg(src);
  *reinterpret_cast<float4*>(v + 4) = __ldcg(src + 1);
  float mx = -INFINITY;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = t0 + e < plen ? fmaxf(mx, v[e]) : mx;
  const float ref = kRefStep * floorf(dev::warp_max(mx) / kRefStep);
  float sum = 0.f;
  uint4 hi, lo;
  T16* hv = reinterpret_cast<T16*>(&hi);
  T16* lv = reinterpret_cast<T16*>(&lo);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = t0 + e < plen ? exp2f(v[e] - ref) : 0.f;
    sum += x;
    hv[e] = dev::from_f<T16>(x);
    if (PS == 2) lv[e] = dev::from_f<T16>(x - dev::to_f(hv[e]));
  }
  *reinterpret_cast<uint4*>(p + row * ppad + t0) = hi;
  if (PS == 2) *reinterpret_cast<uint4*>(p + (rows + row) * ppad + t0) = lo;
  sum = dev::warp_sum(sum);
  if (lane == 0) {
    const size_t at = own ? (size_t(tile) * B + b) * H + h : size_t(tile) * rows + row;
    mt[at] = ref;
    lt[at] = sum;
  }
}

// Quantised prefix -> fp16 hi and lo parts of code x scale, [2][P][r].
// Thread = one 16-byte vector of codes.
template <qsvd_dtype CT>
__global__ void __launch_bounds__(256)
k_prefix_expand(const uint8_t* __restrict__ codes, const __half* __restrict__ scales, __half* __restrict__ out,
                int plen, int r, int group) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  constexpr int N = dev::CacheVec<CT>::N;
  const int vpr = r / N;
  const size_t total = size_t(plen) * vpr, part = size_t(plen) * r;
  for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += size_t(gridDim.x) * 256) {
    const size_t t = i / vpr;
    const int j0 = int(i % vpr) * N;
    const float s = __half2float(scales[t * (r / group) + j0 / group]);
    float v[N];
    dev::CacheVec<CT>::load(codes + t * (size_t(r) * (CT == QSVD_I4 ? 1 : 2) / 2), j0, s, v);
    __half* o = out + t * r + j0;
#pragma unroll
    for (int e0 = 0; e0 < N; e0 += 8) {
      uint4 hi, lo;
      __half* hv = reinterpret_cast<__half*>(&hi);
      __half* lv = reinterpret_cast<__half*>(&lo);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hv[e] = __float2half_rn(v[e0 + e]);
        lv[e] = __float2half_rn(v[e0 + e] - __half2float(hv[e]));
      }
      *reinterpret_cast<uint4*>(o + e0) = hi;
      *reinterpret_cast<uint4*>(o + part + e0) = lo;
    }
  }
}

// Schedules that need no lengths: the prefix as B sequences of plen rows
// (CUDA cores), as one sequence (behind it: rotary scores), and one tile per
// sequence for the combine of merged slots.
__global__ void __launch_bounds__(256)
k_prefix_schedule(int32_t* __restrict__ sched, int32_t* __restrict__ csched, WsHeader* __restrict__ hdr, int B,
                  int plen) {
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  const int nt = (plen + kTile - 1) / kTile;
  for (int i = threadIdx.x; i <= B; i += 256) {
    sched[i] = i * nt;
    csched[i] = i;
    if (i < B) {
      sched[B + 1 + i] = plen;
      csched[B + 1 + i] = 1;
    }
  }
  if (threadIdx.x == 0) {
    sched[2 * B + 1] = 0;
    sched[2 * B + 2] = nt;
    sched[2 * B + 3] = plen;
    hdr->status = 0;
    hdr->G = B;
    hdr->tile = kTile;
    hdr->kernel = 0;
  }
}

// The merge of combine.cu with the prefix's partials beside the own splits'.
// grid (ceil(r / 512), H, B), block 128.
struct MergeIn {
  const float *pm, *pl, *pz;   // own: slot c + b of split c
  const int32_t* sched;
  const float *xm, *xl, *xz;   // prefix: slot sp B + b (n = SP), or slot c + b of schedule xsched, G xg
  const int32_t* xsched;
  int n, xg;
  int most;                    // entries at most
};

__global__ void __launch_bounds__(128)
k_merge_shared(const WsHeader* __restrict__ hdr, const MergeIn in, float* __restrict__ zout, float* __restrict__ cm,
               float* __restrict__ cl, float2* __restrict__ ml, int B, int H, int r, const uint8_t* __restrict__ pf,
               unsigned long long pf_bytes) {
  // the following GEMV's weights towards L2 (constant; a hint)
  if (pf_bytes && threadIdx.x == 32) dev::l2_prefetch_share(pf, pf_bytes);
  dev::pdl_wait();   // see launch_pdl
  dev::pdl_trigger();
  // the partials that count, own splits first: where their z starts and their weight
  extern __shared__ uint64_t merge_smem[];   // most entries: own splits G + the prefix's
  const float** from = reinterpret_cast<const float**>(merge_smem);
  float* wt = reinterpret_cast<float*>(merge_smem + in.most);
  __shared__ int count;
  const int ch = blockIdx.x * 512 + 4 * threadIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const int T = in.sched[B], t0 = in.sched[b], t1 = in.sched[b + 1], G = hdr->G;
    const int XT = in.xsched ? in.xsched[B] : 0, x0 = in.xsched ? in.xsched[b] : 0, x1 = in.xsched ? in.xsched[b + 1] : 0;
    int c0 = 0, n0 = 0, c1 = 0, n1 = in.n;   // first split and splits of the own rows, of the prefix
    if (t1 > t0) {
      c0 = int(dev::split_of_tile(t0, G, T));
      n0 = int(dev::split_of_tile(t1 - 1, G, T)) - c0 + 1;
    }
    if (in.xsched) {
      c1 = int(dev::split_of_tile(x0, in.xg, XT));
      n1 = int(dev::split_of_tile(x1 - 1, in.xg, XT)) - c1 + 1;
    }
    // entry e of the two lists: its slot, or -1 for an empty split
    auto slot_of = [&](int e) -> long long {
      if (e < n0) return dev::split_begin(c0 + e, G, T) == dev::split_begin(c0 + e + 1, G, T) ? -1 : (long long)(c0 + e) + b;
      e -= n0;
      if (!in.xsched) return (long long)e * B + b;
      return dev::split_begin(c1 + e, in.xg, XT) == dev::split_begin(c1 + e + 1, in.xg, XT) ? -1 : (long long)(c1 + e) + b;
    };
    const int n = n0 + n1;
    // m and l of the first 32 entries in registers, loaded together; further ones (long runs of splits) again below
    float m0 = -INFINITY, l0 = 0.f;
    const long long s0 = lane < n ? slot_of(lane) : -1;
    if (s0 >= 0) {
      const size_t at = size_t(s0) * H + h;
      m0 = __ldcg((lane < n0 ? in.pm : in.xm) + at);
      l0 = __ldcg((lane < n0 ? in.pl : in.xl) + at);
    }
    float M = m0;
    for (int e = lane + 32; e < n; e += 32) {
      const long long s = slot_of(e);
      if (s >= 0) M = fmaxf(M, __ldcg((e < n0 ? in.pm : in.xm) + size_t(s) * H + h));
    }
    M = dev::warp_max(M);
    const float w0 = s0 >= 0 ? exp2f(m0 - M) : 0.f;
    float L = w0 * l0;
    for (int e = lane + 32; e < n; e += 32) {
      const long long s = slot_of(e);
      if (s >= 0)
        L += exp2f(__ldcg((e < n0 ? in.pm : in.xm) + size_t(s) * H + h) - M) *
             __ldcg((e < n0 ? in.pl : in.xl) + size_t(s) * H + h);
    }
    L = dev::warp_sum(L);
    const float invL = L > 0.f ? 1.f / L : 0.f;
    int kept = 0;   // compacted in order: entries of weight 0 are left out
    for (int e0 = 0; e0 < n; e0 += 32) {
      const int e = e0 + lane;
      const long long s = e0 == 0 ? s0 : e < n ? slot_of(e) : -1;
      float w = 0.f;
      if (s >= 0) w = (e0 == 0 ? w0 : exp2f(__ldcg((e < n0 ? in.pm : in.xm) + size_t(s) * H + h) - M)) * invL;
      const unsigned on = __ballot_sync(0xffffffffu, w != 0.f);
      if (w != 0.f) {
        const int at = kept + __popc(on & ((1u << lane) - 1u));
        from[at] = (e < n0 ? in.pz : in.xz) + (size_t(s) * H + h) * r;
        wt[at] = w;
      }
      kept += __popc(on);
    }
    if (lane == 0) {
      count = kept;
      if (blockIdx.x == 0) {
        ml[size_t(b) * H + h] = make_float2(M, invL);
        if (cm) {   // one slot per sequence (2 b), merged already
          cm[size_t(2 * b) * H + h] = 0.f;
          cl[size_t(2 * b) * H + h] = 1.f;
        }
      }
    }
  }
  __syncthreads();
  if (ch >= r) return;
  const int n = count;
  float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e0 = 0; e0 < n; e0 += 8) {   // eight partials' loads in flight, added in order
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = e0 + i < n ? __ldcg(reinterpret_cast<const float4*>(from[e0 + i] + ch)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = e0 + i < n ? wt[e0 + i] : 0.f;
      z.x = fmaf(w, v[i].x, z.x); z.y = fmaf(w, v[i].y, z.y);
      z.z = fmaf(w, v[i].z, z.z); z.w = fmaf(w, v[i].w, z.w);
    }
  }
  *reinterpret_cast<float4*>(zout + (size_t(cm ? 2 * b : b) * H + h) * r + ch) = z;
}

// ------------------------------------------------------------------ host

bool encode(CUtensorMap* tm, bool bf16, int rank, const void* p, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  TensorMapEncode enc = tensor_map_encoder();
  const cuuint32_t es[4] = {1, 1, 1, 1};
  memset(tm, 0, sizeof(*tm));
  return enc && enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, cuuint32_t(rank),
                    const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, int AP, int CP, int PS, bool VALUES, bool PAIR>
cudaError_t gemm_p(const CUtensorMap& ta, const CUtensorMap& tb0, const CUtensorMap& tb1, const PxArgs& g, int sms,
                   cudaStream_t s) {
  constexpr int W = PAIR ? 2 : 1;
  const long long units = (long long)((g.MB + W - 1) / W) * (VALUES ? (long long)((g.r + 255) / 256) * g.SP : g.tiles);
  if (units > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const int walkers = units < sms / W ? int(units) : sms / W;
  constexpr size_t smem = 1024 + size_t(px_slots<AP, PAIR>()) * px_slot<AP, PAIR>() + 8 * kPxStage +
                          (2 * kPxMaxSlots + 5 + 10) * 8 + 16;
  static_assert(px_slots<AP, PAIR>() <= kPxMaxSlots && smem <= kPxSmem, "ring fits");
  auto kern = k_prefix_gemm<BF16, AP, CP, PS, VALUES, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(unsigned(walkers * W));
  cfg.blockDim = dim3(kPxThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, ta, tb0, tb1, g);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

template <bool BF16, int AP, int CP, int PS, bool VALUES>
cudaError_t gemm_t(const CUtensorMap& ta, const CUtensorMap& tb0, const CUtensorMap& tb1, const PxArgs& g, bool pair,
                   int sms, cudaStream_t s) {
  return pair ? gemm_p<BF16, AP, CP, PS, VALUES, true>(ta, tb0, tb1, g, sms, s)
                  : gemm_p<BF16, AP, CP, PS, VALUES, false>(ta, tb0, tb1, g, sms, s);
}

// C parts: CP copies of [plen][r] 16-bit rows at `c`, one after another.
// given: the scores are in memory already (rotary mode).
template <bool BF16, int CP>
cudaError_t fast_t(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* c, const void* qt16, int qparts,
                   float gain, int sms, int32_t* counter, int32_t* status, cudaStream_t s, const float* given = nullptr) {
  constexpr int PS = BF16 ? 2 : 1;
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const cuuint64_t r = cuuint64_t(d.r), P = cuuint64_t(L.plen), rows = cuuint64_t(L.MB) * 128, ppad = cuuint64_t(L.ppad);
  CUtensorMap tq, tp, tbs[2], tbv[2];
  if (!given) {
    // query parts [B][qparts][H][r] as {channel, head, part, sequence}: one box is a block's rows of one part
    const cuuint64_t dims[4] = {r, cuuint64_t(d.H), cuuint64_t(qparts), cuuint64_t(d.batch)};
    const cuuint64_t strides[3] = {r * 2, cuuint64_t(d.H) * r * 2, cuuint64_t(qparts) * cuuint64_t(d.H) * r * 2};
    const cuuint32_t box[4] = {64, cuuint32_t(d.H), 1, cuuint32_t(L.nb)};
    if (!encode(&tq, BF16, 4, qt16, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    // P [PS][MB 128][ppad] as {token, row, part}
    const cuuint64_t dims[3] = {ppad, rows, cuuint64_t(PS)};
    const cuuint64_t strides[2] = {ppad * 2, rows * ppad * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    if (!encode(&tp, BF16, 3, ws + L.p, dims, strides, box)) return cudaErrorInvalidValue;
  }
  for (int part = 0; part < 2; ++part) {
    const uint8_t* cp = static_cast<const uint8_t*>(c) + (part < CP ? size_t(part) * L.plen * d.r * 2 : 0);
    const cuuint64_t sd[2] = {r, P}, ss[1] = {r * 2};   // scores: 256 tokens x 64 channels, K-major; rows past P zeros
    const cuuint32_t sb[2] = {64, cuuint32_t(L.pair ? kPxTile / 2 : kPxTile)};   // (a pair's CTA loads half)
    const cuuint64_t vd[3] = {64, P, r / 64}, vs[2] = {r * 2, 128};   // values: 64 tokens x 256 channels, MN-major
    const cuuint32_t vb[3] = {64, 64, cuuint32_t(L.pair ? 2 : 4)};
    if (!encode(&tbs[part], BF16, 2, cp, sd, ss, sb) || !encode(&tbv[part], BF16, 3, cp, vd, vs, vb))
      return cudaErrorInvalidValue;
  }
  PxArgs g{d.batch, d.H, d.r, L.plen, L.nb, L.MB, L.tiles, L.ppad, L.SP, ws + L.p,
           reinterpret_cast<float*>(ws + L.mt), reinterpret_cast<float*>(ws + L.lt), reinterpret_cast<float*>(ws + L.pm),
           reinterpret_cast<float*>(ws + L.pl), reinterpret_cast<float*>(ws + L.pz),
           gain, cache_is_int(d) ? reinterpret_cast<const float*>(ws + L.qinv) : nullptr, counter, status};
  cudaError_t e;
  if (given) {
    const bool own = L.tiles == L.SP;   // as in the scores' epilogue
    const long long warps = (long long)d.batch * d.H * L.tiles;
    e = launch_pdl(k_prefix_probs<T16, PS>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0, s, given,
                   reinterpret_cast<T16*>(ws + L.p), own ? g.pm : g.mt, own ? g.pl : g.lt, d.batch, d.H, L.nb, L.MB,
                   L.plen, L.tiles, L.ppad, own);
    if (e == cudaSuccess) { note_launch(); e = check_launch(); }
  } else {
    bool done = false;
    if constexpr (BF16)   // (only bf16 comes in three parts)
      if ((done = qparts == 3)) e = gemm_t<BF16, 3, CP, PS, false>(tq, tbs[0], tbs[1], g, L.pair, sms, s);
    if (!done) e = gemm_t<BF16, 2, CP, PS, false>(tq, tbs[0], tbs[1], g, L.pair, sms, s);
  }
  if (e != cudaSuccess) return e;
  if (L.tiles != L.SP) {
    e = launch_pdl(k_prefix_norm<T16, PS>, dim3(unsigned(4 * L.MB), unsigned(L.SP)), dim3(256), 0, s,
                   reinterpret_cast<T16*>(ws + L.p), g.mt, g.lt, g.pm, g.pl, d.batch, d.H, L.nb, L.MB, L.tiles, L.ppad,
                   L.SP);
    if (e != cudaSuccess) return e;
    note_launch();
    if ((e = check_launch()) != cudaSuccess) return e;
  }
  return gemm_t<BF16, PS, CP, PS, true>(tp, tbv[0], tbv[1], g, L.pair, sms, s);
}

}  // namespace

PrefixLayout prefix_layout(const qsvd_dims& d, int plen, int sms, size_t base) {
  PrefixLayout L{};
  const bool q = cache_is_int(d);
  L.plen = plen;
  L.fast = d.kernel != QSVD_KERNEL_SIMT && d.H <= 128 &&
           (d.rope ? rope_tc_supported(d) : d.cache_dtype != QSVD_F32 && d.r % 64 == 0);
  const size_t B = size_t(d.batch), H = size_t(d.H), r = size_t(d.r), P = size_t(plen);
  size_t o = base;
  L.ml = o; o = align256(o + B * H * 8);
  L.sched = o; o = align256(o + (2 * B + 4) * 4);
  L.csched = o; o = align256(o + (2 * B + 1) * 4);
  L.hdr = o; o = align256(o + sizeof(WsHeader));
  if (!combine_uses_gemv(d)) {   // merged slots for the CUDA-core combine
    L.cm = o; o = align256(o + 2 * B * H * 4);
    L.cl = o; o = align256(o + 2 * B * H * 4);
    L.cz = o; o = align256(o + 2 * B * H * r * 4);
  }
  if (plen == 0) { L.total = o; return L; }
  if (d.rope) { L.tab = o; o = align256(o + (P + size_t(d.max_len)) * d.d_h * 4); }
  if (L.fast) {
    L.tiles = (plen + kPxTile - 1) / kPxTile;
    L.nb = 128 / d.H;
    if (L.nb > d.batch) L.nb = d.batch;
    L.MB = (d.batch + L.nb - 1) / L.nb;
    L.ppad = L.tiles * kPxTile;
    // token splits of the value product: the fewest that come within 3% of
    // the best fill of the GPU's waves (a split costs B H r float32 partials,
    // written and merged)
    // pairs once the scores take more than two waves of single CTAs (H 32, r 1536,
    // fp16, step without / with pairs, us): B 16, P 12,000 (188 tiles) 101.5 /
    // 110.8; B 32, P 8192 (256) 146 / 150; B 64, P 4096 (256) 196 / 198, P 6144
    // (384) 220.5 / 217.7, P 8192 (512) 247 / 241, P 16,384 (1024) 407 / 391; int8,
    // r 768, B 64: P 8192 197 / 191, P 16,384 287 / 267
    L.pair = L.MB > 1 && (long long)L.MB * L.tiles > 2LL * sms;
    const int W = L.pair ? 2 : 1;   // CTAs per unit
    const long long units = (long long)((L.MB + W - 1) / W) * ((d.r + 255) / 256), walkers = sms / W > 0 ? sms / W : 1;
    double best = 1e30;
    for (int pass = 0; pass < 2; ++pass)
      for (int sp = 1; sp <= 16 && sp <= L.tiles; ++sp) {
        const double cost = double((units * sp + walkers - 1) / walkers) / sp;
        if (pass == 0 && cost < best) best = cost;
        if (pass == 1 && cost <= best * 1.03) { L.SP = sp; break; }
      }
    L.slots = L.SP * d.batch;
    if (q) { L.qt16 = o; o = align256(o + 2 * B * H * r * 2); }   // beside the int8 parts
    if (q) { L.qinv = o; o = align256(o + B * H * 4); }
    if (q) { L.cparts = o; o = align256(o + 2 * P * r * 2); }
    const size_t rows = size_t(L.MB) * 128;
    L.p = o; o = align256(o + (d.cache_dtype == QSVD_BF16 ? 2 : 1) * rows * L.ppad * 2);
    L.mt = o; o = align256(o + size_t(L.tiles) * rows * 4);
    L.lt = o; o = align256(o + size_t(L.tiles) * rows * 4);
    if (d.rope) { L.scores = o; o = align256(o + B * H * L.ppad * 4); }
    if (d.rope) { L.qpack = o; o = align256(o + B * H * kRopePackWords * 4); }
  } else {
    const long long t = (long long)d.batch * ((plen + kTile - 1) / kTile);
    const int hb = split_simt_grid_heads(d);
    long long G = hb > 0 ? (2LL * sms + hb - 1) / hb : sms;
    if (G > t) G = t;
    if (G > kMaxSplits) G = kMaxSplits;
    L.G = int(G < 1 ? 1 : G);
    L.slots = L.G + d.batch;
  }
  L.pm = o; o = align256(o + size_t(L.slots) * H * 4);
  L.pl = o; o = align256(o + size_t(L.slots) * H * 4);
  L.pz = o; o = align256(o + size_t(L.slots) * H * r * 4);
  L.total = o;
  return L;
}

cudaError_t launch_prefix(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                          const void* scales, const void* qt16, int qparts, const float* qt32, float gain, int sms,
                          int32_t* counter, int32_t* status,
                          cudaStream_t s) {
  if (!L.fast) {
    // the CUDA-core split kernel with the same rows for every sequence: no
    // stride between sequences
    qsvd_dims v = d;
    v.max_len = 0;
    return launch_split_simt_absorbed(v, qt32, prefix, scales, reinterpret_cast<const int32_t*>(ws + L.sched), L.G,
                                      reinterpret_cast<float*>(ws + L.pm), reinterpret_cast<float*>(ws + L.pl),
                                      reinterpret_cast<float*>(ws + L.pz), s);
  }
  if (d.cache_dtype == QSVD_BF16) return fast_t<true, 1>(d, L, ws, prefix, qt16, qparts, gain, sms, counter, status, s);
  if (d.cache_dtype == QSVD_F16) return fast_t<false, 1>(d, L, ws, prefix, qt16, qparts, gain, sms, counter, status, s);
  return fast_t<false, 2>(d, L, ws, ws + L.cparts, qt16, qparts, gain, sms, counter, status, s);
}

cudaError_t launch_prefix_table(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, cudaStream_t s) {
  return launch_rope_table(reinterpret_cast<float*>(ws + L.tab), L.plen + d.max_len, d.d_h, d.rope_base, s, true);
}

cudaError_t launch_prefix_rope(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                               const void* scales, const void* wuk, const void* wukT, const float* qrot,
                               float simt_gain, int sms, int32_t* status, cudaStream_t s) {
  const float* tab = reinterpret_cast<const float*>(ws + L.tab);
  const int32_t* sched = reinterpret_cast<const int32_t*>(ws + L.sched);
  if (!L.fast) {
    qsvd_dims v = d;   // as in launch_prefix
    v.max_len = 0;
    return launch_split_simt_rope(v, qrot, wuk, tab, prefix, scales, sched, L.G, reinterpret_cast<float*>(ws + L.pm),
                                  reinterpret_cast<float*>(ws + L.pl), reinterpret_cast<float*>(ws + L.pz), s, nullptr,
                                  simt_gain);
  }
  float* scores = reinterpret_cast<float*>(ws + L.scores);
  const cudaError_t e = launch_rope_scores_shared(d, prefix, L.plen, wukT, reinterpret_cast<const uint32_t*>(ws + L.qpack), tab, sched + 2 * d.batch + 1, sms, scores,
                                                  L.ppad, status, s);
  if (e != cudaSuccess) return e;
  return d.cache_dtype == QSVD_BF16 ? fast_t<true, 1>(d, L, ws, prefix, nullptr, 2, 1.f, sms, nullptr, status, s, scores)
                                    : fast_t<false, 1>(d, L, ws, prefix, nullptr, 2, 1.f, sms, nullptr, status, s, scores);
}

cudaError_t launch_prefix_expand(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                                 const void* scales, cudaStream_t s) {
  if (!L.fast || !cache_is_int(d)) return cudaSuccess;
  const size_t vecs = size_t(L.plen) * cache_row_bytes(d) / 16;
  const unsigned grid = unsigned(vecs / 256 + 1 < 1184 ? vecs / 256 + 1 : 1184);   // eight CTAs an SM
  const cudaError_t e = launch_pdl(d.cache_dtype == QSVD_I8 ? k_prefix_expand<QSVD_I8> : k_prefix_expand<QSVD_I4>, dim3(grid),
                             dim3(256), 0, s, static_cast<const uint8_t*>(prefix), static_cast<const __half*>(scales),
                             reinterpret_cast<__half*>(ws + L.cparts), L.plen, d.r, d.group);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

cudaError_t launch_prefix_schedule(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, cudaStream_t s) {
  cudaError_t e = launch_pdl(k_prefix_schedule, dim3(1), dim3(256), 0, s, reinterpret_cast<int32_t*>(ws + L.sched),
                             reinterpret_cast<int32_t*>(ws + L.csched), reinterpret_cast<WsHeader*>(ws + L.hdr), d.batch,
                             L.plen);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

cudaError_t launch_merge_shared(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const WsHeader* hdr, int G,
                                const int32_t* sched, const float* pm, const float* pl, const float* pz, float* zm,
                                bool slots, const void* next_weights, size_t next_bytes, cudaStream_t s) {
  const float* xm = reinterpret_cast<const float*>(ws + L.pm);
  const bool listed = L.plen > 0 && !L.fast;
  const int most = G + (L.plen > 0 ? (L.fast ? L.SP : L.G) : 0);
  const MergeIn in{pm, pl, pz, sched, xm, reinterpret_cast<const float*>(ws + L.pl),
                   reinterpret_cast<const float*>(ws + L.pz),
                   listed ? reinterpret_cast<const int32_t*>(ws + L.sched) : nullptr, L.plen > 0 ? L.SP : 0, L.G, most};
  cudaError_t e = launch_pdl(k_merge_shared, dim3(unsigned((d.r + 511) / 512), unsigned(d.H), unsigned(d.batch)),
                             dim3(128), size_t(most) * 12, s, hdr, in, slots ? reinterpret_cast<float*>(ws + L.cz) : zm,
                             slots ? reinterpret_cast<float*>(ws + L.cm) : nullptr,
                             slots ? reinterpret_cast<float*>(ws + L.cl) : nullptr, reinterpret_cast<float2*>(ws + L.ml),
                             d.batch, d.H, d.r, static_cast<const uint8_t*>(next_weights),
                             (unsigned long long)next_bytes);
  if (e != cudaSuccess) return e;
  note_launch();
  return check_launch();
}

}  // namespace qsvd
