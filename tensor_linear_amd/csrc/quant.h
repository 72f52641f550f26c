// Launch interface of the 8-bit integer Linear: the quantizer, the int8 shard
// GEMMs and the fold of their int32 partials.  Internal, as kernels.h.
#pragma once

#include "kernels.h"

namespace tpl {

// Output of an int8 GEMM besides OUT_F32 / OUT_BF16: the int32 sums as they
// are (a row layer's partials; no scales, bias or activation).
constexpr int OUT_I32 = 2;

// The scales of an int8 product.  Token m of shard i: x_scale[m * x_ld + i *
// x_shard]; W row n of shard i: w_scale[i * w_shard + n].
struct QuantArgs {
    const float *x_scale; int64_t x_ld; int64_t x_shard;
    const float *w_scale; int64_t w_shard;
};

// Any shape, stride or alignment; every output type, bias and the gated unit.
// GemmArgs counts elements (bytes of A and B); ex as for the bf16 kernels
// (x_rows is not taken).
hipError_t launch_quant_generic(const GemmArgs &g, int out_type, const GemmExtra &ex,
                                const QuantArgs &q, hipStream_t s);

// Workgroups for T tiles, and their split over the 8 XCDs in contiguous ranges of
// tiles.  Fewer tiles than CUs are split too (up to 7 workgroups then have none):
// neighbouring tiles share rows of X or W, and each XCD has an L2 of its own.  Same
// box, us with weights from HBM / warm, split vs tile b to workgroup b: 8192 -> 10240,
// 700 tokens 63.5 / 58.3 vs 68.2 / 60.9; 4096 -> 6144, 500 tokens 18.9 / 19.0 vs 21.0 /
// 21.1; 4096 -> 4096, 256 tokens 13.3 / 13.0 vs 14.3 / 13.9; 4096 -> 28672, 100 tokens
// 34.0 / 22.1 vs 34.2 / 22.1.
inline int quant_grid(int64_t T, int cus, int &xcd_split, int &per_xcd) {
    xcd_split = cus % 8 == 0;
    const int grid = T >= cus ? cus : xcd_split ? (int)((T + 7) / 8 * 8) : (int)T;
    per_xcd = grid / 8;
    return grid;
}

// Whether the DMA-fed int8 kernels can load g's operands with tiles of `rows`
// rows: K, leading dims and shard offsets multiples of 16, 16-byte aligned.
bool quant_dma_supported(const GemmArgs &g, const GemmExtra &ex, int rows);
// 256 x 256 tiles; as launch_quant_generic otherwise.
hipError_t launch_quant_tile(const GemmArgs &g, int out_type, const GemmExtra &ex,
                             const QuantArgs &q, hipStream_t s);

// 256 x 128, 128 x 128 or 128 x 64 tiles, by their number.
hipError_t launch_quant_narrow(const GemmArgs &g, int out_type, const GemmExtra &ex,
                               const QuantArgs &q, hipStream_t s);

// 256 x 128 tiles with the fold of the P shards in registers, a scale for each
// token and shard (q.x_shard = 1); r places the output as in
// launch_gemm_rowfold.
bool quant_rowfold_supported(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &q);
hipError_t launch_quant_rowfold(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &q,
                                int out_type, hipStream_t s);

// Up to 32 tokens (48 of the gated unit), streaming W; fold != NULL: the P shard products folded with a
// scale for each token and shard into fold->Y (C unused).
bool quant_skinny_supported(const GemmArgs &g, const GemmExtra &ex);
hipError_t launch_quant_skinny(const GemmArgs &g, int out_type, const FoldArgs *fold,
                               const GemmExtra &ex, const QuantArgs &q, hipStream_t s);

// Rows of X to int8: scale[m * lds + j] for column group j of G.
struct QuantizeArgs {
    const void *X; int64_t ldx;
    int8_t *Q; int64_t ldq;
    float *scale; int64_t lds;
    int64_t M, Kg; int32_t G;
};
hipError_t launch_quantize_rows(const QuantizeArgs &a, int in_type, hipStream_t s);

// Fold of P int32 partials (r.partials, as int32) into the scaled output:
// per_shard: S = fma chain of float(p_i) * x_scale[m * x_ld + i], ascending;
// else S = float(sum of the p_i) * x_scale[m * x_ld].  Y = fma(S, w_scale[n],
// bias[n] or 0), placed as launch_shard_fold places it.
hipError_t launch_quant_fold(const ReduceArgs &r, const QuantArgs &q, bool per_shard, int out_type,
                             hipStream_t s);

}  // namespace tpl
