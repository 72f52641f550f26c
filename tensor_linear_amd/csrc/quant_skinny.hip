// Launch of the skinny kernel (gemm_skinny_impl.h) on int8 operands: decode
// shapes, bound by streaming W.  16 tokens, 8 shards, weights from HBM (several in turn
// that no cache holds): 8192 -> 28672 43.9 us (5.4 TB/s), 28672 -> 8192 with the fold 47.3
// (5.0), 4096 -> 28672 26.3 (4.5), 8192 -> 10240 19.3 (4.4).  Few output features leave a
// CU one or two workgroups, whose stages end in a barrier with nothing beside them:
// 14336 -> 4096 with the fold 20.7 (2.8), 4096 -> 6144 8.9 (2.8), 4096 -> 4096 7.3 (2.3).
#include "gemm_skinny_impl.h"

namespace tpl {
namespace {

template <int NB, int MB, int KB, int NST>
hipError_t launch_t(const GemmArgs &g, int out_type, const FoldArgs *fold, const GemmExtra &ex,
                    const QuantArgs &q, hipStream_t s) {
    constexpr int BN = 16 * NB;
    const bool sw = ex.act == ACT_SWIGLU;
    const int64_t tn = (g.N + (sw ? 16 : BN) - 1) / (sw ? 16 : BN);
    const int64_t blocks = fold ? tn : tn * g.P;
    const FoldArgs f = fold ? *fold : FoldArgs{nullptr, 0, 0};
    if (blocks > 0xFFFFFFFFll / SK_THREADS) {
        // One launch has fewer than 2^32 threads: the columns in halves.
        const int64_t n = tn / 2 * (sw ? 16 : BN);
        const int os = out_type == OUT_BF16 ? 2 : 4;
        GemmArgs h = g;
        h.N = n;
        const hipError_t e = launch_t<NB, MB, KB, NST>(h, out_type, fold, ex, q, s);
        if (e != hipSuccess) return e;
        h.N = g.N - n;
        h.B = (const char *)g.B + n * g.ldb;
        GemmExtra x = ex;
        QuantArgs r = q;
        FoldArgs y = f;
        if (ex.bias) x.bias = (const char *)ex.bias + n * os;
        if (out_type != OUT_I32) r.w_scale = q.w_scale + n;
        if (fold) y.Y = (char *)f.Y + n * os;
        else h.C = (char *)g.C + n * os;
        return launch_t<NB, MB, KB, NST>(h, out_type, fold ? &y : nullptr, x, r, s);
    }
    const dim3 grid((unsigned)blocks), block(SK_THREADS);
    if (sw) {
        if constexpr (NB == 2) {
            if (out_type == OUT_BF16) gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, false, true, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
            else gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, false, true, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
        } else {
            return hipErrorInvalidValue;
        }
    } else if (fold) {
        if (out_type == OUT_BF16) gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, true, false, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
        else gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, true, false, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
    } else if (out_type == OUT_I32) {
        gemm_skinny_kernel<NB, MB, KB, NST, OUT_I32, false, false, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
    } else if (out_type == OUT_BF16) {
        gemm_skinny_kernel<NB, MB, KB, NST, OUT_BF16, false, false, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
    } else {
        gemm_skinny_kernel<NB, MB, KB, NST, OUT_F32, false, false, OpI8><<<grid, block, 0, s>>>(g, f, ex, q);
    }
    return hipGetLastError();
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool quant_skinny_supported(const GemmArgs &g, const GemmExtra &ex) {
    return ex.x_rows == 0 && g.M >= 1 && g.M <= (ex.act == ACT_SWIGLU ? SKINNY_MAX_M : 32) && g.K > 0 && g.K % 16 == 0 &&
           g.lda % 16 == 0 && g.ldb % 16 == 0 && g.a_shard % 16 == 0 && g.b_shard % 16 == 0 &&
           aligned16(g.A) && aligned16(g.B);
}

hipError_t launch_quant_skinny(const GemmArgs &g, int out_type, const FoldArgs *fold,
                               const GemmExtra &ex, const QuantArgs &q, hipStream_t s) {
    if (g.M == 0 || g.N == 0 || g.P == 0) return hipSuccess;
    // The bf16 form's blocking: the bytes in flight are the same.  16 tokens, stages
    // of 2 to 6, 16 to 64 W rows and 128 to 512 bytes of K a row were within 3% of it
    // or behind, column and fold.
    if (ex.act == ACT_SWIGLU) {
        if (fold || out_type == OUT_I32) return hipErrorInvalidValue;
        if (g.M <= 16) return launch_t<2, 1, 256, 3>(g, out_type, fold, ex, q, s);
        if (g.M <= 32) return launch_t<2, 2, 256, 2>(g, out_type, fold, ex, q, s);
        return launch_t<2, 4, 256, 2>(g, out_type, fold, ex, q, s);
    }
    if (g.M <= 16) {
        if (fold && g.N >= 32 * (int64_t)device_cu_count())
            return launch_t<2, 1, 256, 4>(g, out_type, fold, ex, q, s);
        if (fold) return launch_t<1, 1, 256, 4>(g, out_type, fold, ex, q, s);
        return launch_t<1, 1, 256, 3>(g, out_type, fold, ex, q, s);
    }
    if (fold) return launch_t<4, 2, 256, 2>(g, out_type, fold, ex, q, s);
    return launch_t<2, 2, 256, 2>(g, out_type, fold, ex, q, s);
}

}  // namespace tpl
