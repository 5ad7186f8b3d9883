// Workspace and launchers of the shared-prefix decode (prefix.cu), used by
// the C-ABI layer.
#pragma once

#include "internal.cuh"

namespace qsvd {

constexpr int kPxTile = 256;   // tokens per score tile

// Sections behind the decode's own workspace.
struct PrefixLayout {
  bool pair;        // fast: CTA pairs
  bool fast;        // tensor cores; else the CUDA-core split kernels on B views of the prefix
  int plen, tiles;  // prefix rows, score tiles
  int nb, MB;       // sequences per block of 128 query rows, blocks
  int ppad;         // tokens per row of P (tiles x 256)
  int SP;           // token splits of the value product
  int G;            // CUDA cores: split CTAs
  int slots;        // partials (fast: SP x B; CUDA cores: G + B)
  size_t qt16, qinv, cparts, p, mt, lt, pm, pl, pz, ml, sched, hdr, cm, cl, cz, csched, tab, scores, qpack, total;
};
PrefixLayout prefix_layout(const qsvd_dims& d, int plen, int sms, size_t base);

// The prefix's partials (m, l, z per slot) from the absorbed query: qt16 its
// 16-bit parts [B][qparts][H][r] (fast; of a quantised prefix scaled per
// (sequence, head), the scales' inverses at L.qinv), qt32 [B][H][r] (CUDA cores).  gain: on
// the tensor cores' scores, for what their accumulation truncates.  counter:
// one word, zero.
// launch_prefix_expand goes before the own rows' split kernel and
// launch_prefix directly behind it: the scores wait for nothing of it.
cudaError_t launch_prefix_expand(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                                 const void* scales, cudaStream_t s);
cudaError_t launch_prefix(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                          const void* scales, const void* qt16, int qparts, const float* qt32, float gain, int sms,
                          int32_t* counter, int32_t* status,
                          cudaStream_t s);
// Rotary mode: the table of all positions, prefix then own rows (tab, built
// per call: the packed one ends at max_len), and the partials from the rotated
// query qrot [B][H][d_h].  simt_gain: on the scores of the CUDA cores, which
// truncate nothing (the tensor cores' come about as the own rows' do).
cudaError_t launch_prefix_table(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, cudaStream_t s);
cudaError_t launch_prefix_rope(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const void* prefix,
                               const void* scales, const void* wuk, const void* wukT, const float* qrot,
                               float simt_gain, int sms, int32_t* status, cudaStream_t s);
cudaError_t launch_prefix_schedule(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, cudaStream_t s);
// Merge of the own splits' and the prefix's partials: zm [B][H][r], or (slots
// != 0) one slot per sequence for launch_combine; ml {M, 1 / L} [B][H].
cudaError_t launch_merge_shared(const qsvd_dims& d, const PrefixLayout& L, uint8_t* ws, const WsHeader* hdr, int G,
                                const int32_t* sched, const float* pm, const float* pl, const float* pz, float* zm,
                                bool slots, const void* next_weights, size_t next_bytes, cudaStream_t s);

}  // namespace qsvd
