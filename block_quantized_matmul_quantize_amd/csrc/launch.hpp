// Host-side launch functions implemented by the kernel translation units.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm.h"

namespace qmm {

// Plan overrides (qmm_set_override), read once at the start of a call so that every decision of
// that call (workspace layout, regime, kernels) sees the same values; 0 = automatic throughout.
struct Ovr {
    int path = 0;        // 1 matrix-vector, 2 tiled
    int streamk = 0;     // 1 off, 2 on
    int tile_j = 0;      // 32, 64, 128
    int mv_steps = 0;    // register-streamed matrix-vector kernel: 256-value steps per wave (1, 2, 4)
    int mv_kernel = 0;   // 1 register-streamed, 2 LDS-staged, 3 dot4
    int fuse_cols = 0;   // most columns the LDS-staged kernel quantizes itself (1..8)
};

hipError_t launch_quantize_q8_1(const float *x, int64_t n_rows, int64_t k, uint8_t *y, hipStream_t s);

// Tiled-kernel activation layout (tiled_act.hpp): for each 256-value step kb and activation row r,
// the 8 blocks' codes (256 bytes), fp32 d (32 bytes) and s parts (32 bytes), each kind in a table
// of its own indexed by kb * n_rows + r.
inline size_t q8_1_tiled_bytes(int64_t n_rows, int64_t k) { return (size_t)((k / 32 + 7) / 8) * n_rows * 320; }
// fp32 rows -> tiled layout (and, if canon is not null, the canonical q8_1 blocks as well); the
// same launch sets the nzero words at zero to 0 (the tiled kernel's stream-K counters)
hipError_t launch_quantize_q8_1_tiled(const float *x, int64_t n_rows, int64_t k, uint8_t *tiled, uint8_t *canon,
                                      hipStream_t s, int32_t *zero = nullptr, int64_t nzero = 0);
// canonical q8_1 blocks -> tiled layout (zero / nzero as above)
hipError_t launch_relayout_q8_1_tiled(const uint8_t *xq, int64_t n_rows, int64_t k, uint8_t *tiled, hipStream_t s,
                                      int32_t *zero = nullptr, int64_t nzero = 0);
hipError_t launch_fill_u32(uint32_t *p, int64_t n, uint32_t v, hipStream_t s);

// Column map for the matrix-vector and tiled kernels.  Dense: column j reads activation row j
// and writes output row j.  Expert mode: columns are the expert's (token, slot) pairs taken from
// the device-side sorted list.
struct ColMap {
    // expert mode only (all null / zero for dense)
    const int32_t *sorted;     // [pairs] pair index (t*top_k + slot), grouped by expert
    const int32_t *bounds;     // [n_exp + 1] segment starts in `sorted`
    const int32_t *tile_start; // [n_exp + 1] prefix of tiled-kernel column tiles per expert
    const int32_t *small;      // [n_exp] experts handled by the matrix-vector kernel, then -1
    int32_t top_k;
    int32_t x_per_tok;
    int32_t n_exp;
    int64_t w_expert_stride;   // bytes between expert matrices
    int64_t act_rows;          // activation rows (n_tok * x_per_tok): row count of the tiled layout
    int64_t pairs;             // (token, slot) pairs of the call
};

// Matrix-vector kernel: n <= 8 columns (dense) or the small experts (expert mode, grid.y = n_exp).
hipError_t launch_mmvq(int type, const uint8_t *w, int64_t rows, int64_t k, const uint8_t *xq, int64_t n,
                       float *y, int32_t *dbg, const ColMap *cm, int64_t n_exp, const Ovr &o, hipStream_t s);

// Gate/up fusion, matrix-vector: y = silu(W_gate x) * (W_up x) for n <= 8 dense q8_1 columns (cm
// null) or the small experts (cm set, grid.y = n_exp); the LDS-staged kernel where both matrices
// meet its rules, else the register-streamed one.
int mmvq_glu_f32_choice(int type, const void *wg, const void *wu, int64_t rows, int64_t k, const float *x, int64_t n,
                        const Ovr &o);
hipError_t launch_mmvq_glu(int type, const uint8_t *wg, const uint8_t *wu, int64_t rows, int64_t k, const uint8_t *xq,
                           int64_t n, float *y, const ColMap *cm, int64_t n_exp, const Ovr &o, hipStream_t s);

// The same on the dot4 kernel for 1..3 dense fp32 columns (quantized inside); Q4_K and Q8_0 under
// mmvq_dot4_supported's alignment rules for both matrices.
hipError_t launch_mmvq_dot4_glu_f32(int type, const uint8_t *wg, const uint8_t *wu, int64_t rows, int64_t k,
                                    const float *x, int64_t n, float *y, hipStream_t s);

// And on the LDS-staged kernel (mmvq_stream_supported's rules for both matrices): dense fp32
// (x_fp32, quantized inside) or q8_1 columns, or the small experts (cm set, q8_1).
hipError_t launch_mmvq_stream_glu(int type, const uint8_t *wg, const uint8_t *wu, int64_t rows, int64_t k,
                                  const void *x, bool x_fp32, int64_t n, float *y, const ColMap *cm, int64_t n_exp,
                                  hipStream_t s);

// fp32-input matrix-vector product with the q8_1 quantization done inside the dot4 or the
// LDS-staged kernel (no separate quantize launch): dense calls either kernel would take.
// Kernel launch_mmvq takes for q8_1 input: 3 dot4, 2 LDS-staged MFMA, 1 register-streamed, 0 none
// (a forced kernel that cannot serve the call); host logic only.
int mmvq_kernel_choice(int type, const void *w, int64_t rows, int64_t k, const void *xq, int64_t n, const ColMap *cm,
                       const Ovr &o);
// Kernel launch_mmvq_fused takes for fp32 input: 3 dot4, 2 LDS-staged MFMA, 0 not fused.
int mmvq_fused_choice(int type, const void *w, int64_t rows, int64_t k, const float *x, int64_t n, const Ovr &o);
// Launches the kernel mmvq_fused_choice names (`choice`, non-zero).
hipError_t launch_mmvq_fused(int choice, int type, const uint8_t *w, int64_t rows, int64_t k, const float *x, int64_t n,
                             float *y, hipStream_t s);
hipError_t launch_mmvq_dot4_f32(int type, const uint8_t *w, int64_t rows, int64_t k, const float *x, int64_t n,
                                float *y, hipStream_t s);
hipError_t launch_mmvq_stream_f32(int type, const uint8_t *w, int64_t rows, int64_t k, const float *x, int64_t n,
                                  float *y, hipStream_t s);

// LDS-streamed matrix-vector kernel (mmvq_stream.hip): 16-byte aligned weights, activations and
// rows, K a multiple of 256.
bool mmvq_stream_supported(int type, const void *w, int64_t k, const void *xq, const ColMap *cm);
hipError_t launch_mmvq_stream(int type, const uint8_t *w, int64_t rows, int64_t k, const uint8_t *xq, int64_t n,
                              float *y, int32_t *dbg, const ColMap *cm, int64_t n_exp, hipStream_t s);
// dot4 matrix-vector kernel (mmvq_dot4.hip) for 1..mmvq_dot4_max_cols() dense columns: Q4_K and
// Q8_0, K a multiple of 256.
int device_cus();   // compute units of the current device, looked up once per device (api.cpp)
int mmvq_dot4_max_cols();
bool mmvq_dot4_supported(int type, const void *w, int64_t k, const void *xq, const ColMap *cm);
hipError_t launch_mmvq_dot4(int type, const uint8_t *w, int64_t rows, int64_t k, const uint8_t *xq, int64_t n,
                            float *y, int32_t *dbg, const ColMap *cm, int64_t n_exp, int max_cols, hipStream_t s);

// Tiled int8-MFMA kernel plan.
struct MmqLaunch {
    int tile_j;          // 32, 64 or 128
    int64_t ntiles;      // row tiles x column tiles (dense)
    int64_t n_ct;        // column tiles
    int64_t k_iters;     // K steps of 256 values
    int64_t units;       // workgroups (== ntiles unless stream-K)
    bool stream_k;
    float *partials;     // [units][2][128*tile_j] when stream_k
    int32_t *counters;   // [ntiles] split-tile arrival counters when stream_k, zero at launch
    bool packed = false; // w in the panel layout (repack.hip), k % 256 == 0
};
hipError_t launch_mmq(int type, const uint8_t *w, int64_t rows, int64_t k, const uint8_t *xq, int64_t n,
                      float *y, int32_t *dbg, const MmqLaunch &plan, hipStream_t s);
// Gate/up fusion: y[n][rows] = silu(W_gate x) * (W_up x), tiles of 64 outputs, no stream-K.
hipError_t launch_mmq_glu(int type, const uint8_t *wg, const uint8_t *wu, int64_t rows, int64_t k, const uint8_t *xq,
                          int64_t n, float *y, int tile_j, hipStream_t s);
// Expert mode: grid over (row tiles, max column tiles); experts with > 8 columns.  w_up not null:
// gate/up fusion, w the gate matrices.
hipError_t launch_mmq_id(int type, const uint8_t *w, const uint8_t *w_up, int64_t rows, int64_t k,
                         const uint8_t *xq, float *y, const ColMap &cm, int tile_j, int64_t max_col_tiles,
                         hipStream_t s);

// Expert grouping: counts, bounds, stable sorted pair list, column-tile prefix, small-expert list.
hipError_t launch_moe_group(const int32_t *ids, int64_t pairs, int32_t n_exp, int32_t tile_j,
                            int32_t small_max, int32_t *sorted, int32_t *bounds, int32_t *tile_start,
                            int32_t *small, int32_t *invalid, hipStream_t s);
// Grouping + activation quantization (tiled and canonical layouts) in one launch, for n_exp up to
// the per-wave grouping's limit (moe_prologue_fused); cus: compute units of the device.
bool moe_prologue_fused(int32_t n_exp);
hipError_t launch_moe_prologue(const int32_t *ids, int64_t pairs, int32_t n_exp, int32_t tile_j, int32_t small_max,
                               int32_t *sorted, int32_t *bounds, int32_t *tile_start, int32_t *small, int32_t *invalid,
                               const float *x, int64_t n_rows, int64_t k, uint8_t *tiled, uint8_t *canon,
                               int32_t cus, hipStream_t s);

// Panel layout (repack.hip): bytes of the layout for a [rows][k] matrix (-1: type or shape not
// supported), and the one-time repack of the original blocks w into wp (16-byte aligned).
int64_t panel_bytes(int type, int64_t rows, int64_t k);
hipError_t launch_repack_panels(int type, const uint8_t *w, int64_t rows, int64_t k, uint8_t *wp, hipStream_t s);
// Dense products reading panel-layout weights: n <= 8 fp32 columns (the LDS-staged kernel, which
// quantizes x itself; x 16-byte aligned), and the tiled kernel (plan.packed set).
hipError_t launch_mmvq_stream_panel_f32(int type, const uint8_t *wp, int64_t rows, int64_t k, const float *x, int64_t n,
                                        float *y, hipStream_t s);

// fp16-activation mode (f16act.hip)
hipError_t launch_f16act_encode(const float *x, int64_t n, int64_t k, uint16_t *y16, int32_t *e, float *bsum,
                                hipStream_t s);
hipError_t launch_mmvq_f16act(int type, const uint8_t *w, int64_t rows, int64_t k, const uint16_t *y16,
                              const int32_t *e, const float *bsum, int64_t n, float *out, hipStream_t s);

// Row operators (sort_ids.hip, combine.hip, embed.hip, lora.hip).  Types are the GGUF ids of include/qmm.h;
// arguments are checked in api_rows.cpp.
// Stable sort of n ids: order / pos (may be null) / bounds (may be null) as qmm_sort_ids.  with_keys: the
// sorted keys (ids outside [0, n_keys) as n_keys) stay in ws, at sort_ids_keys.
size_t sort_ids_bytes(int64_t n, int64_t n_keys, bool with_keys);
const int32_t *sort_ids_keys(const void *ws, int64_t n, int64_t n_keys);
hipError_t launch_sort_ids(const int32_t *ids, int64_t n, int64_t n_keys, int32_t *order, int32_t *pos,
                           int32_t *bounds, bool with_keys, uint8_t *ws, hipStream_t s);
hipError_t launch_gather_sorted(int type, const void *x, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                                const int32_t *n_valid, void *y, hipStream_t s);
// pos: places, null for (token, slot) order, or with n_ids > 0 the ids of pairs in that order.
hipError_t launch_combine(int type, const void *h, int64_t n_tok, int64_t top_k, int64_t k, const int32_t *pos,
                          int64_t n_ids, const float *w, const void *base, void *y, hipStream_t s);
hipError_t launch_combine_backward(int type, const void *dy, const void *h, int64_t n_tok, int64_t top_k, int64_t k,
                                   const int32_t *pos, int64_t n_ids, const float *w, const int32_t *n_valid,
                                   void *dh, float *dw, hipStream_t s);
hipError_t launch_embed(int type, const void *table, int64_t vocab, int64_t k, const int32_t *ids, int64_t n,
                        float scale, int y_type, void *y, hipStream_t s);
size_t embed_backward_bytes(int64_t n, int64_t k, int64_t vocab);
hipError_t launch_embed_backward(int dy_type, const void *dy, int64_t n, int64_t k, const int32_t *ids, int64_t vocab,
                                 float scale, int g_type, void *grad, uint8_t *ws, hipStream_t s);
// What the adapters' forward and backward calls have in common.
struct LoraCall {
    int x_type, w_type;
    const void *x;      // [n][k]
    int64_t n, k;
    const void *a;      // [n_adapters][rank][k]
    const void *b;      // [n_adapters][rows][rank]
    int64_t rows, rank, n_adapters;
    const int32_t *ids; // [n]
    const float *scale; // [n_adapters] or null (1)
};
// Padded rank of the partial and dh rows; slices of K that a product of k values a row is split into.
int lora_padded_rank(int64_t rank);
int lora_narrow_slices(int64_t n, int64_t k);
// Whether the launch below can also sort the rows (order not null) for this many rows and adapters.
bool lora_narrow_sorts(int64_t n, int64_t n_adapters);
// part [slices][n][padded rank] = v [n][k] times the row's matrix: m [rank][k] (by_row) or [k][rank] of each adapter.
hipError_t launch_lora_narrow(int x_type, int w_type, bool by_row, const void *v, int64_t n, int64_t k, const void *m,
                              int64_t rank, int64_t n_adapters, const int32_t *ids, float *part, int32_t *order,
                              int32_t *pos, int32_t *bounds, hipStream_t s);
// Between the two halves: sums of the slices, and what the gradients of A and B need.
struct LoraFinish {
    const float *part;      // or null: only kept
    int parts;
    int64_t n, rank, n_adapters;
    const int32_t *ids;
    const float *scale;
    float *sum;             // or null: [n][padded rank] (may be part: its first slice)
    float *h;               // or null: [n][rank], zeros for a row without an adapter
    // where not null, the bf16 parts [place / 32][3][padded rank][place % 32] of kept [n][rank] and of the scaled
    // sum, rows at their places pos of the order sorted by adapter
    const float *kept;
    uint16_t *parts_h, *parts_dh;
    const int32_t *pos;
};
hipError_t launch_lora_finish(const LoraFinish &c, hipStream_t s);
// out [n][cols] = base + scale * (sum of part's slices) times m, [rank][cols] (by_row) or [cols][rank].
hipError_t launch_lora_wide(int x_type, int w_type, bool by_row, const float *part, int parts, int64_t n, int64_t cols,
                            const void *m, int64_t rank, int64_t n_adapters, const int32_t *ids, const float *scale,
                            const void *base, void *out, hipStream_t s);
size_t lora_outer_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters);
// da [n_adapters][rank][k] from x and dh's parts, db [n_adapters][rows][rank] from dy and h's (either may be null).
hipError_t launch_lora_outer(int x_type, const void *x, const uint16_t *parts_dh, int64_t k, float *da, const void *dy,
                             const uint16_t *parts_h, int64_t rows, const float *scale, float *db, int64_t n,
                             int64_t rank, int64_t n_adapters, const int32_t *order, const int32_t *bounds, float *part,
                             hipStream_t s);
size_t lora_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters);
hipError_t launch_lora(const LoraCall &c, const void *base, void *y, float *h_out, uint8_t *ws, hipStream_t s);
size_t lora_backward_bytes(int64_t n, int64_t k, int64_t rows, int64_t rank, int64_t n_adapters);
hipError_t launch_lora_backward(const LoraCall &c, const void *dy, const float *h, const void *dx_base, void *dx,
                                float *da, float *db, uint8_t *ws, hipStream_t s);

// Dense fp32-input product with a workspace sized exactly to its plan (api.cpp), for the
// allocation-free entry point (noalloc.hip).  o: one reading of the overrides for the whole call.
Ovr load_overrides();
// Sets the calling thread's qmm_last_error message and returns st.
qmm_status report(qmm_status st, const char *msg);
// qmm_matmul's argument checks; *need = the workspace bytes the call's plan uses (0 for n == 0).
qmm_status matmul_exact_check(int type, const void *w, int64_t rows, int64_t k, const float *x, int64_t n,
                              const float *y, const Ovr &o, size_t *need);
// The product itself, with ws holding at least matmul_exact_check's bytes.
qmm_status matmul_exact_run(int type, const void *w, int64_t rows, int64_t k, const float *x, int64_t n, float *y,
                            uint8_t *ws, const Ovr &o, hipStream_t s);

}  // namespace qmm
