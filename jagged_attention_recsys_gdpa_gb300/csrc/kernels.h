// Host-side launchers of the attention kernels.
#pragma once
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace jattn {

struct AttnArgs;
struct CacheView;
struct DecodeArgs;
struct DevStatus;
struct NormArgs;
struct NormJoinArgs;
struct RotaryArgs;
template <int PAIRS>
struct RotaryTablesArgs;
struct PageArgs;

// Forward: schedule rows are blocks of fwd_rows_per_item() query rows. `split`
// selects the column-split arrangement of the activation warps (for items that
// mostly hold one query tile) over the ping-pong one; `block` selects the
// kernels compiled for block masks (fwd_block.cu) and `hilo` those that pass P
// as bf16 hi + lo parts (pointwise activations without the 1/Lkv normaliser,
// fwd_hilo.cu, fwd_block_hilo.cu).
cudaError_t launch_fwd(int D, int act, bool split, bool block, bool hilo, const CUtensorMap& q, const CUtensorMap& k,
                       const CUtensorMap& v, const AttnArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_fwd_block(int D, int act, bool split, const CUtensorMap& q, const CUtensorMap& k,
                             const CUtensorMap& v, const AttnArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_fwd_hilo(int D, int act, bool split, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const AttnArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_fwd_block_hilo(int D, int act, bool split, const CUtensorMap& q, const CUtensorMap& k,
                                  const CUtensorMap& v, const AttnArgs& a, int grid, cudaStream_t stream);
int fwd_rows_per_item();

// MXFP8 forward (softmax, D = 128): maps of the E4M3 codes (uint8 [rows, H*128],
// boxes of 128 rows x 128 bytes); a.sf_* / a.bs_* carry the block scales.
cudaError_t launch_fwd_mx(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a,
                          int grid, cudaStream_t stream);

// MXFP8 backward (softmax, D = 128). launch_mx_di: D_i = <dO~_i, O_i> per
// query row and head into di (row blocks from block_start, at most
// max_blocks of them). dq: over 128-row query tiles (maps of 128-row boxes);
// dkdv: over 128-row key tiles, queries in steps of 96 (the Q and dO maps
// have 96-row boxes). a.f0 = LSE, a.f1 = D; a.sf_* / a.bs_* the block scales.
cudaError_t launch_mx_di(const int64_t* q_off, int B, int H, int64_t max_blocks, const uint8_t* dout,
                         const uint8_t* dout_scales, const int* block_start, const void* o, float* di,
                         cudaStream_t stream);
cudaError_t launch_bwd_dq_mx(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                             const CUtensorMap& dout, const AttnArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_bwd_dkdv_mx(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const CUtensorMap& dout, const AttnArgs& a, int grid, cudaStream_t stream);

// dK, dV over key tiles (transposed schedule, 128-row key tiles); a.out0 /
// a.out1 receive dK / dV.
cudaError_t launch_bwd_dkdv(int D, int act, bool hilo, const CUtensorMap& q, const CUtensorMap& k,
                            const CUtensorMap& v, const CUtensorMap& dout, const AttnArgs& a, int grid,
                            cudaStream_t stream);
cudaError_t launch_bwd_dkdv_hilo(int D, int act, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                 const CUtensorMap& dout, const AttnArgs& a, int grid, cudaStream_t stream);
// dQ over query tiles (128-row query tiles). For softmax it also computes
// Di = rowsum(dO * O) from the dO tiles and O (the map `o` in the one-ring
// layout, the rows at a.in0 in the two-ring one) into a.f1, so it runs before
// the dK/dV pass, which reads Di. `split`: K and V tiles in two rings (used at
// D = 128, for items of many key tiles).
cudaError_t launch_bwd_dq(int D, int act, bool hilo, bool split, const CUtensorMap& q, const CUtensorMap& k,
                          const CUtensorMap& v, const CUtensorMap& dout, const CUtensorMap& o, const AttnArgs& a,
                          int grid, cudaStream_t stream);
cudaError_t launch_bwd_dq_hilo(int D, int act, bool split, const CUtensorMap& q, const CUtensorMap& k,
                               const CUtensorMap& v, const CUtensorMap& dout, const CUtensorMap& o, const AttnArgs& a,
                               int grid, cudaStream_t stream);

// Short-query / short-key attention (pma.cu): pointwise activations, no
// mask, D = 128, keys on the MMA's M dimension and at most 64 queries per
// product. The forward takes items of at most 64 query rows from the 64-row
// query-tile schedule; its Q map has 64-row boxes (a.out0 = O). The fused
// backward (Q and dO maps with 64-row boxes; a.out0 = dQ, a.out1 = dV, a.out2
// = dK) has a pooling mode (items from the 64-row query-tile schedule, every
// sequence with 1 <= Lq <= 64 or no keys) and a cross mode (`cross`: items
// from the 128-row key-tile schedule with 64-column query ranges, every
// sequence with Lkv <= 128 and keys whenever it has queries). It runs only
// when launch_pma_gate found the batch within its mode's limits; the gate
// then empties the general dQ and dK/dV schedules.
cudaError_t launch_pma_fwd(int act, bool hilo, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const AttnArgs& a, int grid, cudaStream_t stream);
// Short-key forward (pma.cu): cross-attention whose every sequence has at
// most 128 keys (the gate's cross mode), items from the 128-row key-tile
// schedule with 128-row query ranges; Q map with 128-row boxes, a.out0 = O.
cudaError_t launch_skv_fwd(int act, bool hilo, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const AttnArgs& a, const int* gate, int grid, cudaStream_t stream);
// Short-key backward (pma.cu): the same shapes and schedule as
// launch_skv_fwd (128-row query ranges), Q / dO maps with 128-row boxes;
// a.out0 = dQ, a.out1 = dV, a.out2 = dK.
cudaError_t launch_skv_bwd(int act, bool hilo, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                           const CUtensorMap& dout, const AttnArgs& a, const int* gate, int grid,
                           cudaStream_t stream);
cudaError_t launch_pma_gate(const int64_t* q_off, const int64_t* kv_off, int64_t B, bool cross, int* gate,
                            int* n_tiles_q, int* n_tiles_kv, cudaStream_t stream);
cudaError_t launch_pma_bwd(int act, bool hilo, bool cross, const CUtensorMap& q, const CUtensorMap& k,
                           const CUtensorMap& v, const CUtensorMap& dout, const AttnArgs& a, const int* gate,
                           int grid, cudaStream_t stream);
int pma_rows_per_item();

// Rotary embedding of a jagged tensor x ([total, H, D] bf16, rows described
// by own_off; other_off describes the other side for the alignment):
// y = R(pos) x, or R(pos)^T x with `inverse`. keys: x holds key rows.
cudaError_t launch_rope(const int64_t* own_off, const int64_t* other_off, int B, int keys, int inverse, int H,
                        int D, int64_t total, const void* x, void* y, const float* cos_t, const float* sin_t,
                        int rows, DevStatus* status, cudaStream_t stream);
// MXFP8 (E4M3 + one E8M0 scale per 32 x 32 block) quantization of a jagged
// bf16 tensor; block_start / n_blocks come from sched_prefix_launch(32).
cudaError_t launch_mx_quant(const int64_t* off, int B, int H, int D, int64_t max_blocks, const void* x, void* codes,
                            uint8_t* scales, const int* block_start, const int* n_blocks, cudaStream_t stream);
// Row-major [rows, half] cos / sin tables to pair-major [half, rows] copies.
cudaError_t launch_rope_transpose(const float* cos_t, const float* sin_t, int rows, int half, float* cos_pm,
                                  float* sin_pm, cudaStream_t stream);

// Paged cache (cache.cu): jagged bf16 rows into and out of the pages.
cudaError_t launch_cache_append(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                                const int64_t* start, const void* k, const void* v, int D, const float* cos_t,
                                const float* sin_t, int rope_rows, DevStatus* status, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheView& c, bool mx, int64_t B, int64_t total, const int64_t* off,
                              const int64_t* start, void* k, void* v, int D, DevStatus* status, cudaStream_t stream);
// Attention over the paged cache (decode.cu): scratch of decode_scratch_bytes;
// k and v map the pages as {line, page_size, lines of a row, H, n_pages}, lines
// of 128 bytes (codes at D = 64: 64), with boxes of decode_box's rows and lines.
size_t decode_scratch_bytes(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H);
void decode_box(int D, bool mx, int64_t B, int64_t total_q, int64_t max_kv, int G, int H, int page_size, int* rows,
                int* lines);
cudaError_t launch_decode(int D, bool mx, DecodeArgs a, const CUtensorMap& k, const CUtensorMap& v, void* scratch,
                          cudaStream_t stream);

// Layer norm (norm.cu, norm_bwd.cu) of JATTN_F32 / BF16 / F16 rows, which are read in vectors of 16 bytes (everything is
// aligned to them), in vectors that start before the rows (all tensors alike, see norm.cuh) or value by value. The
// backward writes norm_bwd_parts partial rows, which launch_norm_join adds.
enum class NormPath { kVectors, kShifted, kValues };
cudaError_t launch_norm(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream);
int norm_bwd_parts(int type, NormPath path, int64_t rows, int N, int sms);
cudaError_t launch_norm_bwd(int type, NormPath path, const NormArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_norm_join(int weight_type, const NormJoinArgs& a, cudaStream_t stream);

// Rotary positions of rows (rotary.cu), read in vectors of 16 bytes, two values at a time or one by one, and their tables
// (`vectors`: in 16 bytes).
enum class RotaryPath { kVectors, kPairs, kValues };
cudaError_t launch_rotary(int type, RotaryPath path, bool half_layout, const RotaryArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_rotary_tables(const RotaryTablesArgs<512>& a, bool vectors, int sms, cudaStream_t stream);

// Page pool (pages.cu); total: an assign's rows, -1 for a release.
size_t page_scratch_bytes(int64_t B, int64_t total, int64_t max_pages);
cudaError_t launch_page_assign(const PageArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_page_release(const PageArgs& a, int sms, cudaStream_t stream);

}  // namespace jattn
