// Launch of the skinny bf16 kernel (gemm_skinny_impl.h): which shapes it takes
// and the blocking for a number of tokens.
#include "gemm_skinny_impl.h"

namespace tpl {
namespace {

template <int NB, int MB, int KB, int NST, bool SWIGLU = false>
hipError_t launch_mb(const GemmArgs &g, int out_type, const FoldArgs *fold, const GemmExtra &ex,
                     hipStream_t s) {
    constexpr int ON = SWIGLU ? 16 : 16 * NB;
    const int64_t tn = (g.N + ON - 1) / ON;
    const int64_t blocks = fold ? tn : tn * g.P;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    dim3 grid((unsigned)blocks), block(SK_THREADS);
    FoldArgs f = fold ? *fold : FoldArgs{nullptr, 0, 0};
    if (SWIGLU) {
        if (fold) return hipErrorInvalidValue;
        if (out_type == OUT_BF16) gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, false, SWIGLU><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
        else gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, false, SWIGLU><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
    } else if (fold) {
        if (out_type == OUT_BF16) gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, true, false><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
        else gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, true, false><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
    } else {
        if (out_type == OUT_BF16) gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, false, false><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
        else gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, false, false><<<grid, block, 0, s>>>(g, f, ex, QuantArgs{});
    }
    return hipGetLastError();
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool gemm_skinny_supported(const GemmArgs &g, const GemmExtra *ex) {
    if (ex && ex->x_rows > 0) return false;
    return g.M >= 1 && g.M <= SKINNY_MAX_M && g.K > 0 && g.K % 8 == 0 && g.lda % 8 == 0 &&
           g.ldb % 8 == 0 && g.a_shard % 8 == 0 && g.b_shard % 8 == 0 &&
           aligned16(g.A) && aligned16(g.B);
}

hipError_t launch_gemm_skinny(const GemmArgs &g, int out_type, const FoldArgs *fold,
                              const GemmExtra *exp, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    GemmExtra ex{};
    if (exp) ex = *exp;
    if (ex.x_rows > 0) return hipErrorInvalidValue;
    // LDS per workgroup: NST * (16*NB + 16*MB) * KB * 2 bytes, plus the
    // cross-wave sums (4 * NB * MB KB).  Small stages let several workgroups share a CU, which
    // keeps more loads in flight when the grid is large (one workgroup per
    // 16 output columns and shard: three 16 KB stages, two in flight).  The
    // fused fold has a P times smaller grid: one workgroup per CU with 32
    // output columns and four 24 KB stages, three in flight (16 columns and
    // four 16 KB stages where 32 would leave CUs without one).  Measured with
    // M = 16, K = 8192, N = 28672 over 8 shards: column 82-83 us with 3 or 4
    // stages of 256 columns against 88-89 with 2; fused fold of 8 shards of
    // K = 3584, N = 8192: 82-83 us with 32 columns and 3-6 stages, 86-87 with
    // 16 columns and two 512-column stages; a later same-box sweep gave 86.6
    // us for this choice against 85.9 (32 columns, 3 stages), 89.6-90.8 (16
    // columns: 3 or 4 stages of 256, 2 of 512), 97.6 (32 columns, 2 stages of
    // 512) and 147.7 (64 columns: half the CUs idle); three later same-box
    // runs of 2-6 stages of 256 put 4 stages 2-7% ahead of 5 (6 stages 5% and
    // 2 stages 25% behind).  The gated unit streams 32 W rows (16 gate, 16
    // up) per workgroup with the column form's stages.
    if (ex.act == ACT_SWIGLU) {
        if (fold) return hipErrorInvalidValue;
        if (g.M <= 16) return launch_mb<2, 1, 256, 3, true>(g, out_type, fold, ex, s);   // 72 KB
        if (g.M <= 32) return launch_mb<2, 2, 256, 2, true>(g, out_type, fold, ex, s);   // 64 KB
        return launch_mb<2, 4, 256, 2, true>(g, out_type, fold, ex, s);                  // 96 KB
    }
    if (g.M <= 16) {
        // Fused fold: 32 output columns per workgroup where that still gives
        // every CU one, else 16.  Same box, 8 shards, us after a read-only
        // 1 GiB flush, 16 vs 32 columns: 4096 -> 4096 13.8 vs 16.3-16.8,
        // 8192 -> 4096 21.2-21.6 vs 26.0-26.1, 14336 -> 4096 31.8-32.2 vs
        // 38.6-39.4; bitwise equal.
        if (fold && g.N >= 32 * (int64_t)device_cu_count())
            return launch_mb<2, 1, 256, 4>(g, out_type, fold, ex, s);         // 96 KB
        if (fold) return launch_mb<1, 1, 256, 4>(g, out_type, fold, ex, s);   // 64 KB
        return launch_mb<1, 1, 256, 3>(g, out_type, fold, ex, s);             // 48 KB
    }
    // Above 16 tokens every workgroup re-reads its X rows from L2 with each
    // stage, so more W rows per workgroup share them (and no more 16-row X
    // blocks than M needs).  Same-box sweep, 8 shards, us for M = 24 / 32 /
    // 48 / 64, against 16 W rows per workgroup and 2 or 4 X blocks: column
    // 4096 -> 28672: 39.9 / 39.1 / 55.9 / 72.2 vs 53.1 / 51.9 / 108.1 / 116.0;
    // 8192 -> 10240: 33.8 / 35.2 / 43.0 / 67.8 vs 45.3 / 45.8 / 84.0 / 86.5;
    // 8192 -> 28672: 88.4 / 88.4 / 103.2 / 145.6 vs 124.4 / 125.5 / 216.2 /
    // 217.2; fused fold of 28672 -> 8192: 93.0 / 94.1 / 171.6 / 171.5 vs 119.8 /
    // 123.5 / 228.7 / 230.5.  All bitwise equal (each output's K blocks and
    // their order do not depend on the workgroup's shape).
    if (g.M <= 32) {
        if (fold) return launch_mb<4, 2, 256, 2>(g, out_type, fold, ex, s);   // 128 KB
        return launch_mb<2, 2, 256, 2>(g, out_type, fold, ex, s);             // 80 KB
    }
    if (fold) return launch_mb<2, 4, 128, 3>(g, out_type, fold, ex, s);       // 104 KB
    // Above 48 tokens the tile kernels' order of work is faster (same box, 8
    // shards, us after a read-only flush / warm, 64 tokens, skinny vs 128 x
    // 128 tiles: column 4096 -> 28672 79.8 / 75.1 vs 59.3 / 39.0, 8192 ->
    // 28672 146.1 / 146.9 vs 106.0 / 106.3; row partials + fold 14336 ->
    // 4096 50.7 / 45.8 vs 31.9 / 27.1), so no call reaches here with more.
    return launch_mb<4, 3, 256, 2>(g, out_type, fold, ex, s);                 // 160 KB
}

}  // namespace tpl
