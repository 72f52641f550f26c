// Launch of the 256 x 256 bf16 tile kernel (gemm_tile_impl.h): which shapes it
// takes, its schedule, and the variant for each output and epilogue.
#include "gemm_tile_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool gemm_tile_supported(const GemmArgs &g, const GemmExtra *ex) {
    // 32-bit per-lane offsets: one tile's rows must span < 2 GiB (for the
    // gated unit, up to the up rows of the tile).
    const int64_t wspan = TB + (ex && ex->act == ACT_SWIGLU ? ex->up_off : 0);
    const bool small_rows = (int64_t)TB * g.lda * 2 < (1ll << 31) &&
                            wspan * g.ldb * 2 < (1ll << 31);
    bool ok = g.K > 0 && g.K % 64 == 0 && g.lda % 8 == 0 && g.ldb % 8 == 0 &&
              g.a_shard % 8 == 0 && g.b_shard % 8 == 0 && aligned16(g.B) && small_rows;
    if (!ex) return ok && aligned16(g.A);
    // Bias: 16-byte loads of 8 values per lane.
    if (ex->bias && (((uintptr_t)ex->bias % 16) != 0 || ex->bias_shard % 8 != 0)) return false;
    if (ex->act == ACT_SWIGLU && ex->up_off % 8 != 0) return false;
    if (ex->x_rows > 0) {
        if (ex->x_rows % TB != 0) return false;
        const int64_t ns = (g.M + ex->x_rows - 1) / ex->x_rows;
        for (int64_t j = 0; j < ns; ++j)
            if (!aligned16(ex->x_slice[j])) return false;
        return ok;
    }
    return ok && aligned16(g.A);
}

namespace {

template <int OUT, int EPI, bool XG>
hipError_t launch_tile_t(const GemmArgs &g, const TileSched &ts, int vec, const GemmExtra &ex,
                         int grid, hipStream_t s) {
    gemm_tile_kernel<OUT, EPI, XG><<<dim3(grid), dim3(TT), 0, s>>>(g, ts, vec, ex, QuantArgs{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_tile(const GemmArgs &g, int out_type, const GemmExtra *exp, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    GemmExtra ex{};
    if (exp) ex = *exp;
    const bool swiglu = ex.act == ACT_SWIGLU;
    const int tbn = swiglu ? TB / 2 : TB;
    const int64_t tm = (g.M + TB - 1) / TB, tn = (g.N + tbn - 1) / tbn;
    const int64_t T = tm * tn * g.P;
    if (T > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    TileSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    // Groups of 8 tile rows for the bf16 column products, 4 for the fp32
    // row partials (measured on one box: fc2 +1.2-1.4%, Llama-70B O row
    // +1.7-2.2% with 4; column products equal or better with 8).
    ts.group_m = out_type == OUT_BF16 ? 8 : 4;
    ts.T = (int)T;
    const int cus = device_cu_count();
    int grid = (int)(T < cus ? T : cus);
    ts.xcd_split = (grid == cus && cus % 8 == 0 && T >= cus) ? 1 : 0;
    ts.per_xcd = grid / 8;
    // 16-byte stores of 8 bf16 or 4 fp32 values: row starts and shard offsets
    // must keep that alignment.
    const int vw = out_type == OUT_BF16 ? 8 : 4;
    const int vec = (g.ldc % vw == 0) && (g.c_shard % vw == 0) && (((uintptr_t)g.C) % 16 == 0);
    const bool xg = ex.x_rows > 0;
    if (out_type != OUT_BF16) {
        // fp32 output (row partials): no epilogue options.
        if (xg || swiglu || ex.bias) return hipErrorInvalidValue;
        return launch_tile_t<OUT_F32, EPI_NONE, false>(g, ts, vec, ex, grid, s);
    }
    const int epi = swiglu ? EPI_SWIGLU : ex.bias ? EPI_BIAS : EPI_NONE;
    if (xg) {
        if (epi == EPI_SWIGLU) return launch_tile_t<OUT_BF16, EPI_SWIGLU, true>(g, ts, vec, ex, grid, s);
        if (epi == EPI_BIAS) return launch_tile_t<OUT_BF16, EPI_BIAS, true>(g, ts, vec, ex, grid, s);
        return launch_tile_t<OUT_BF16, EPI_NONE, true>(g, ts, vec, ex, grid, s);
    }
    if (epi == EPI_SWIGLU) return launch_tile_t<OUT_BF16, EPI_SWIGLU, false>(g, ts, vec, ex, grid, s);
    if (epi == EPI_BIAS) return launch_tile_t<OUT_BF16, EPI_BIAS, false>(g, ts, vec, ex, grid, s);
    return launch_tile_t<OUT_BF16, EPI_NONE, false>(g, ts, vec, ex, grid, s);
}

}  // namespace tpl
