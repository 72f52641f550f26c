// Launch of the row GEMM with the fold in registers (gemm_rowfold_impl.h) on
// int8 operands with a scale for each token and shard: 4096 tokens of 14336 -> 4096
// 219 us (2.19 POP/s; int32 partials and their fold 332).  Against the tile kernel's
// 2.7 POP/s it moves 1.5 times the operand bytes a product (the running sums take
// half of the registers) and, after each shard, converts and scales 128 sums a lane
// (2.5% of the time).
#include "gemm_rowfold_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <bool SCAT, int OUT, bool TAIL>
void launch_t(bool eight, int grid, const GemmArgs &g, const FoldSched &ts, const ReduceArgs &r,
              int vec, const QuantArgs &q, hipStream_t s) {
    if (eight) gemm_rowfold8_kernel<SCAT, OpI8, OUT, TAIL><<<dim3(grid), dim3(FT8), 0, s>>>(g, ts, r, vec, q);
    else gemm_rowfold_kernel<SCAT, OpI8, OUT, TAIL><<<dim3(grid), dim3(FT), 0, s>>>(g, ts, r, vec, q);
}

template <int OUT>
void launch_out(bool scat, bool eight, int grid, const GemmArgs &g, const FoldSched &ts,
                const ReduceArgs &r, int vec, const QuantArgs &q, hipStream_t s) {
    const bool tail = g.K % 128 != 0;
    if (scat && tail) launch_t<true, OUT, true>(eight, grid, g, ts, r, vec, q, s);
    else if (scat) launch_t<true, OUT, false>(eight, grid, g, ts, r, vec, q, s);
    else if (tail) launch_t<false, OUT, true>(eight, grid, g, ts, r, vec, q, s);
    else launch_t<false, OUT, false>(eight, grid, g, ts, r, vec, q, s);
}

}  // namespace

bool quant_rowfold_supported(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &q) {
    GemmExtra none{};
    // the scales' 32-bit offsets inside a tile, and tiles inside one token slice
    return quant_dma_supported(g, none, FM) && q.x_ld <= (1ll << 20) &&
           (r.slice_rows >= g.M || r.slice_rows % FM == 0);
}

hipError_t launch_quant_rowfold(const GemmArgs &g, const ReduceArgs &r, const QuantArgs &q,
                                int out_type, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const int64_t tm = (g.M + FM - 1) / FM, tn = (g.N + FN - 1) / FN;
    const int64_t T = tm * tn;
    if (tm > 0x7FFFFFFFll || tn > 0x7FFFFFFFll || T > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    FoldSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    ts.T = (int)T;
    const int cus = device_cu_count();
    const int grid = quant_grid(T, cus, ts.xcd_split, ts.per_xcd);
    const int vw = out_type == OUT_BF16 ? 8 : 4;
    bool vec = r.ldy % vw == 0;
    const bool scat = r.use_slices || r.slice_rows < g.M;
    if (scat && r.use_slices) {
        for (int64_t j = 0; j * r.slice_rows < g.M; ++j) vec = vec && aligned16(r.y_slice[j]);
    } else {
        vec = vec && aligned16(r.Y) && (!scat || r.slice_stride % vw == 0);
    }
    const bool eight = T < cus;   // two waves a SIMD, as the bf16 form chooses
    if (out_type == OUT_BF16) launch_out<OUT_BF16>(scat, eight, grid, g, ts, r, vec, q, s);
    else launch_out<OUT_F32>(scat, eight, grid, g, ts, r, vec, q, s);
    return hipGetLastError();
}

}  // namespace tpl
