// Launch of the narrow tiles (gemm_narrow_impl.h) on int8 operands: launches whose
// 256 x 256 tiles would leave CUs idle.  Bound by the loads' latency and rate: one
// workgroup a CU keeps two steps of 24-48 KB in flight (8192 -> 10240 at 48 tokens
// 28.1 us with the weights from HBM, 3.0 TB/s, 20.5 warm; 4096 -> 28672 at 100 tokens
// 34.0, 3.5 TB/s).
#include "gemm_narrow_impl.h"

namespace tpl {
namespace {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <int OUT, int FM, int TN, bool SW>
void launch_t(const GemmArgs &g, const NarrowSched &ts, int vec, const GemmExtra &ex, const QuantArgs &q,
              int grid, hipStream_t s) {
    if (g.K % 128)
        gemm_narrow_kernel<OUT, FM, TN, SW, OpI8, true><<<dim3(grid), dim3(FM * 2), 0, s>>>(g, ts, ex.bias, ex.bias_shard, vec, ex.up_off, q);
    else
        gemm_narrow_kernel<OUT, FM, TN, SW, OpI8, false><<<dim3(grid), dim3(FM * 2), 0, s>>>(g, ts, ex.bias, ex.bias_shard, vec, ex.up_off, q);
}

// Two groups of waves for the halves of K.
template <int OUT>
void launch_halves(const GemmArgs &g, const NarrowSched &ts, int vec, const GemmExtra &ex, const QuantArgs &q,
                   int grid, hipStream_t s) {
    if (g.K % 128)
        gemm_narrow_kernel<OUT, 128, 64, false, OpI8, true, 2><<<dim3(grid), dim3(512), 0, s>>>(g, ts, ex.bias, ex.bias_shard, vec, 0, q);
    else
        gemm_narrow_kernel<OUT, 128, 64, false, OpI8, false, 2><<<dim3(grid), dim3(512), 0, s>>>(g, ts, ex.bias, ex.bias_shard, vec, 0, q);
}

template <int FM, int TN>
void launch_out(int out_type, bool sw, const GemmArgs &g, const NarrowSched &ts, int vec, const GemmExtra &ex,
                const QuantArgs &q, int grid, hipStream_t s) {
    if constexpr (TN == 128) {
        if (sw) {
            if (out_type == OUT_BF16) launch_t<OUT_BF16, FM, 128, true>(g, ts, vec, ex, q, grid, s);
            else launch_t<OUT_F32, FM, 128, true>(g, ts, vec, ex, q, grid, s);
            return;
        }
    }
    if (out_type == OUT_I32) launch_t<OUT_I32, FM, TN, false>(g, ts, vec, ex, q, grid, s);
    else if (out_type == OUT_BF16) launch_t<OUT_BF16, FM, TN, false>(g, ts, vec, ex, q, grid, s);
    else launch_t<OUT_F32, FM, TN, false>(g, ts, vec, ex, q, grid, s);
}

}  // namespace

hipError_t launch_quant_narrow(const GemmArgs &g, int out_type, const GemmExtra &ex,
                               const QuantArgs &q, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    const bool sw = ex.act == ACT_SWIGLU;
    // The tile shape by the bf16 form's rule, which measured both sides of each: the
    // pipeline, its loads and its instructions are the same.
    const int cus = device_cu_count();
    const int64_t tn128 = sw ? (g.N + 63) / 64 : (g.N + 127) / 128;   // tiles of 128 W rows
    const int FM = ((g.M + 127) / 128) * tn128 * g.P <= cus ? 128 : 256;
    const int64_t tm = (g.M + FM - 1) / FM;
    const int TN = (!sw && FM == 128 && 2 * tm * tn128 * g.P <= cus) ? 64 : 128;
    const int64_t tn = sw ? tn128 : (g.N + TN - 1) / TN;
    const int64_t T = tm * tn * g.P;
    if (tm > 0x7FFFFFFFll || tn > 0x7FFFFFFFll || tm * tn > 0x7FFFFFFFll || T > 0x7FFFFFFFll)
        return hipErrorInvalidConfiguration;
    NarrowSched ts;
    ts.tiles_m = (int)tm;
    ts.tiles_n = (int)tn;
    ts.T = (int)T;
    const int grid = quant_grid(T, cus, ts.xcd_split, ts.per_xcd);
    const int vw = out_type == OUT_BF16 ? 8 : 4;
    const int vec = g.ldc % vw == 0 && g.c_shard % vw == 0 && aligned16(g.C);
    // The halves of K side by side where one pass of 64-column tiles is all there is
    // and K is long enough to pay for the join.  Same box, 8 shards, us with weights
    // from HBM / warm, halves vs one group: 8192 -> 10240, 64 tokens 30.1 / 21.2 vs
    // 35.6 / 25.9; 4096 -> 4096, 256 tokens 14.3 / 13.8 vs 16.1 / 15.9; 2048 -> 10240, 64
    // tokens 9.1 / 8.8 vs 10.0 / 9.4; 1024 -> 4096, 128 tokens 7.5 / 7.0 vs 7.4 / 6.6.
    if (TN == 64 && T <= cus && g.K >= 2048) {
        if (out_type == OUT_I32) launch_halves<OUT_I32>(g, ts, vec, ex, q, grid, s);
        else if (out_type == OUT_BF16) launch_halves<OUT_BF16>(g, ts, vec, ex, q, grid, s);
        else launch_halves<OUT_F32>(g, ts, vec, ex, q, grid, s);
    } else if (FM == 256) launch_out<256, 128>(out_type, sw, g, ts, vec, ex, q, grid, s);
    else if (TN == 128) launch_out<128, 128>(out_type, sw, g, ts, vec, ex, q, grid, s);
    else launch_out<128, 64>(out_type, sw, g, ts, vec, ex, q, grid, s);
    return hipGetLastError();
}

}  // namespace tpl
