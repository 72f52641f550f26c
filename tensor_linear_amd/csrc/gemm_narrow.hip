// Launch of the narrow bf16 tiles (gemm_narrow_impl.h): the tile shape for a
// problem and the variant for each output and epilogue.
#include "gemm_narrow_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

hipError_t launch_gemm_narrow(const GemmArgs &g, int out_type, const GemmExtra *exp,
                              hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    GemmExtra ex{};
    if (exp) ex = *exp;
    const bool sw = ex.act == ACT_SWIGLU;
    if ((ex.act != ACT_NONE && !sw) || ex.x_rows > 0 || (out_type != OUT_BF16 && (ex.bias || sw)))
        return hipErrorInvalidValue;
    // 128-row tiles when they fit in one pass over the CUs, else 256-row.
    // Same-box A/B, 8 shards, us after a read-only 1 GiB cache flush / warm,
    // 128-row vs 256-row tiles: M = 128, 4096 -> 28672: 61.6 / 41.0 vs
    // 65.5 / 56.9; M = 65, 8192 -> 10240: 74.2 / 54.6 vs 91.7 / 88.3;
    // M = 256, 8192 -> 10240: 83.9 / 62.0 vs 110.7 / 88.6; M = 200,
    // 4096 -> 14336: 49.0 / 41.6 vs 57.6 / 49.4.  Bitwise equal.
    const int cus = device_cu_count();
    const int64_t tn128 = sw ? (g.N + 63) / 64 : (g.N + 127) / 128;   // tiles of 128 W rows
    const int FM = ((g.M + 127) / 128) * tn128 * g.P <= cus ? 128 : 256;
    const int64_t tm = (g.M + FM - 1) / FM;
    // 64-column tiles where 128 x 128 ones would fill at most half of the
    // CUs.  Same box, 8 shards, us after a read-only 1 GiB flush / warm, 64-
    // vs 128-column tiles: M = 65, 8192 -> 10240 65.6 / 48.4 vs 74.5 / 55.6;
    // M = 128 70.1 / 51.6 vs 81.5 / 55.8; M = 128, 4096 -> 4096 36.9 / 27.3
    // vs 43.3 / 30.9; row partials M = 128, 8192 -> 2048 15.0 / 12.2 vs
    // 17.7 / 14.4.  Bitwise equal.
    const int TN = (!sw && FM == 128 && 2 * tm * tn128 * g.P <= cus) ? 64 : 128;
    const int64_t tn = sw ? tn128 : (g.N + TN - 1) / TN;
    const int64_t T = tm * tn * g.P;
    if (T > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    NarrowSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    ts.T = (int)T;
    const int grid = (int)(T < cus ? T : cus);
    ts.xcd_split = (grid == cus && cus % 8 == 0 && T >= cus) ? 1 : 0;
    ts.per_xcd = grid / 8;
    const int vw = out_type == OUT_BF16 ? 8 : 4;
    const int vec = g.ldc % vw == 0 && g.c_shard % vw == 0 && aligned16(g.C);
    const __bf16 *bias = (const __bf16 *)ex.bias;
    const int64_t uo = ex.up_off;
    if (sw) {
        if (FM == 128)
            gemm_narrow_kernel<OUT_BF16, 128, 128, true><<<dim3(grid), dim3(256), 0, s>>>(g, ts, bias, ex.bias_shard, vec, uo, QuantArgs{});
        else
            gemm_narrow_kernel<OUT_BF16, 256, 128, true><<<dim3(grid), dim3(512), 0, s>>>(g, ts, bias, ex.bias_shard, vec, uo, QuantArgs{});
    } else if (TN == 64) {
        if (out_type == OUT_BF16)
            gemm_narrow_kernel<OUT_BF16, 128, 64><<<dim3(grid), dim3(256), 0, s>>>(g, ts, bias, ex.bias_shard, vec, 0, QuantArgs{});
        else
            gemm_narrow_kernel<OUT_F32, 128, 64><<<dim3(grid), dim3(256), 0, s>>>(g, ts, nullptr, 0, vec, 0, QuantArgs{});
    } else if (FM == 128) {
        if (out_type == OUT_BF16)
            gemm_narrow_kernel<OUT_BF16, 128, 128><<<dim3(grid), dim3(256), 0, s>>>(g, ts, bias, ex.bias_shard, vec, 0, QuantArgs{});
        else
            gemm_narrow_kernel<OUT_F32, 128, 128><<<dim3(grid), dim3(256), 0, s>>>(g, ts, nullptr, 0, vec, 0, QuantArgs{});
    } else if (out_type == OUT_BF16) {
        gemm_narrow_kernel<OUT_BF16, 256, 128><<<dim3(grid), dim3(512), 0, s>>>(g, ts, bias, ex.bias_shard, vec, 0, QuantArgs{});
    } else {
        gemm_narrow_kernel<OUT_F32, 256, 128><<<dim3(grid), dim3(512), 0, s>>>(g, ts, nullptr, 0, vec, 0, QuantArgs{});
    }
    return hipGetLastError();
}

}  // namespace tpl
