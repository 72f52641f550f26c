// Launch of the bf16 row GEMM with the fold in registers (gemm_rowfold_impl.h):
// which shapes it takes and the form for a number of tiles.
#include "gemm_rowfold_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool gemm_rowfold_supported(const GemmArgs &g, const ReduceArgs &ro) {
    const bool small_rows = (int64_t)FM * g.lda * 2 < (1ll << 31) &&
                            (int64_t)FN * g.ldb * 2 < (1ll << 31);
    if (!(g.K > 0 && g.K % FBK == 0 && g.lda % 8 == 0 && g.ldb % 8 == 0 && g.a_shard % 8 == 0 &&
          g.b_shard % 8 == 0 && aligned16(g.A) && aligned16(g.B) && small_rows))
        return false;
    // A reduce-scatter tile must not span two token slices.
    if (ro.slice_rows < g.M && ro.slice_rows % FM != 0) return false;
    return true;
}

hipError_t launch_gemm_rowfold(const GemmArgs &g, const ReduceArgs &ro, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const int64_t tm = (g.M + FM - 1) / FM, tn = (g.N + FN - 1) / FN;
    const int64_t T = tm * tn;
    if (T > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    FoldSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    ts.T = (int)T;
    const int cus = device_cu_count();
    const int grid = (int)(T < cus ? T : cus);
    ts.xcd_split = (grid == cus && cus % 8 == 0 && T >= cus) ? 1 : 0;
    ts.per_xcd = grid / 8;
    bool vec = ro.ldy % 8 == 0;
    // Slice addressing whenever the output is split into slices or given as
    // slice allocations (with one slice, P = 1, slice 0 is the whole output
    // and ro.Y is not set).
    const bool scat = ro.use_slices || ro.slice_rows < g.M;
    if (scat && ro.use_slices) {
        for (int64_t j = 0; j * ro.slice_rows < g.M; ++j) vec = vec && aligned16(ro.y_slice[j]);
    } else {
        vec = vec && aligned16(ro.Y) && (!scat || ro.slice_stride % 8 == 0);
    }
    // Fewer tiles than CUs: the chip is not at its power limit, and the
    // second wave per SIMD, issuing MFMAs while the other waits on its reads
    // and loads, shows as wall time (measured on one box, cold / warm: M x N
    // = 520 x 4136, K/P = 512, 99 tiles, 63.1 / 48.8 vs 69.4 / 57.4 us; 300 x
    // 1000, K/P = 1024, 16 tiles, 107.4 / 82.5 vs 111.7 / 90.5 us).  From 256
    // tiles on the four-wave form holds its own (2048 x 4096, K/P = 2048:
    // 260.3 / 220.8 vs 262.6 / 220.2 us; larger shapes 2-3% behind).
    if (T < cus) {
        if (scat)
            gemm_rowfold8_kernel<true><<<dim3(grid), dim3(FT8), 0, s>>>(g, ts, ro, vec ? 1 : 0, QuantArgs{});
        else
            gemm_rowfold8_kernel<false><<<dim3(grid), dim3(FT8), 0, s>>>(g, ts, ro, vec ? 1 : 0, QuantArgs{});
    } else if (scat) {
        gemm_rowfold_kernel<true><<<dim3(grid), dim3(FT), 0, s>>>(g, ts, ro, vec ? 1 : 0, QuantArgs{});
    } else {
        gemm_rowfold_kernel<false><<<dim3(grid), dim3(FT), 0, s>>>(g, ts, ro, vec ? 1 : 0, QuantArgs{});
    }
    return hipGetLastError();
}

}  // namespace tpl
