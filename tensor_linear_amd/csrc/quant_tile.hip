// Launch of the 256 x 256 tile kernel (gemm_tile_impl.h) on int8 operands: the
// pipeline of the bf16 form with twice the K a step, bound by the matrix cores at
// the clock that the chip's power limit leaves them (4096 tokens of 4096 -> 2 x 14336
// 356-366 us, 2.63-2.70 POP/s, of 5 at the full clock).
#include "gemm_tile_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <int OUT, int EPI>
void launch_t(const GemmArgs &g, const TileSched &ts, int vec, const GemmExtra &ex, const QuantArgs &q,
              int grid, hipStream_t s) {
    if (g.K % 128)
        gemm_tile_kernel<OUT, EPI, false, OpI8, true><<<dim3(grid), dim3(TT), 0, s>>>(g, ts, vec, ex, q);
    else
        gemm_tile_kernel<OUT, EPI, false, OpI8, false><<<dim3(grid), dim3(TT), 0, s>>>(g, ts, vec, ex, q);
}

}  // namespace

bool quant_dma_supported(const GemmArgs &g, const GemmExtra &ex, int rows) {
    // 16-byte chunks of K, and 32-bit per-lane offsets inside a tile's rows
    // (for the gated unit up to its up rows).
    const int64_t wspan = rows + (ex.act == ACT_SWIGLU ? ex.up_off : 0);
    return ex.x_rows == 0 && g.K > 0 && g.K % 16 == 0 && g.lda % 16 == 0 && g.ldb % 16 == 0 &&
           g.a_shard % 16 == 0 && g.b_shard % 16 == 0 && aligned16(g.A) && aligned16(g.B) &&
           (int64_t)rows * g.lda < (1ll << 31) && wspan * g.ldb < (1ll << 31);
}

hipError_t launch_quant_tile(const GemmArgs &g, int out_type, const GemmExtra &ex,
                             const QuantArgs &q, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const bool swiglu = ex.act == ACT_SWIGLU;
    const int tbn = swiglu ? TB / 2 : TB;
    const int64_t tm = (g.M + TB - 1) / TB, tn = (g.N + tbn - 1) / tbn;
    const int64_t T = tm * tn * g.P;
    if (tm > 0x7FFFFFFFll || tn > 0x7FFFFFFFll || tm * tn > 0x7FFFFFFFll || T > 0x7FFFFFFFll)
        return hipErrorInvalidConfiguration;
    TileSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    // Groups of 8 tile rows (same box, 8 shards, us with 4 / 8 / 16: 4096 tokens of 4096
    // -> 28672 386 / 382 / 392, gated 370 / 369 / 373; 2048 tokens of 8192 -> 2 x 28672
    // gated 728 / 704 / 701); 4 for int32 partials, as the bf16 form's fp32 ones.
    ts.group_m = out_type == OUT_I32 ? 4 : 8;
    ts.T = (int)T;
    const int cus = device_cu_count();
    const int grid = quant_grid(T, cus, ts.xcd_split, ts.per_xcd);
    const int vw = out_type == OUT_BF16 ? 8 : 4;
    const int vec = g.ldc % vw == 0 && g.c_shard % vw == 0 && aligned16(g.C);
    if (out_type == OUT_I32) launch_t<OUT_I32, EPI_NONE>(g, ts, vec, ex, q, grid, s);
    else if (out_type == OUT_BF16 && swiglu) launch_t<OUT_BF16, EPI_SWIGLU>(g, ts, vec, ex, q, grid, s);
    else if (out_type == OUT_BF16) launch_t<OUT_BF16, EPI_NONE>(g, ts, vec, ex, q, grid, s);
    else if (swiglu) launch_t<OUT_F32, EPI_SWIGLU>(g, ts, vec, ex, q, grid, s);
    else launch_t<OUT_F32, EPI_NONE>(g, ts, vec, ex, q, grid, s);
    return hipGetLastError();
}

}  // namespace tpl
