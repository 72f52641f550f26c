// How the attention's work is cut: what host and device share of it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn.h"

namespace tpl {

constexpr int32_t PLAN_FAR = 1 << 29;   // what positions and counts of tokens are below

// x / d = x by >> shift for x < 2^31: 2^(31 + i) / d rounded up, 2^i >= d, times x is too
// large by less than 2^(31 + i) / d, which no quotient feels.
struct Divisor { uint32_t by; int32_t shift; };
inline Divisor divisor(int64_t d) {
    int i = 0;
    while (((int64_t)1 << i) < d) ++i;
    return Divisor{(uint32_t)((((uint64_t)1 << (31 + i)) + (uint64_t)d - 1) / (uint64_t)d), 31 + i};
}

// stream: the tiles of all items in `groups` equal runs; else a workgroup for each of
// the row_tiles * Hkv items.  few: 32 rows a workgroup, else 128.
// last_pos: positions of the table; window: 2 PLAN_FAR at most, excess: what it is longer, 2^32 - 1 at most;
// n_pages: 2^31 at most.
struct AttnPlan { int32_t stream, few, groups, last_pos, window; uint32_t n_pages; int64_t row_tiles; Divisor g, page; uint32_t excess; };

// The plan of a call of these sizes and types (the lengths are on the device: T, B and the
// heads are all that the host knows).
AttnPlan attention_plan(int64_t T, int64_t B, int64_t Hkv, int32_t G, int64_t D, int elem_bytes, bool quant);

hipError_t launch_attention_any(const AttnArgs &a, int elem_bytes, hipStream_t s);
hipError_t launch_attention_bf16(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s);
hipError_t launch_attention_f32(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s);
hipError_t launch_attention_bf16_int8(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s);
hipError_t launch_attention_f32_int8(const AttnArgs &a, const AttnPlan &p, bool dma, hipStream_t s);

// The item that a run begins and does not finish: row tile r of a sequence whose rows (of
// tokens and heads) begin at token `first`, key head h, in `pieces` runs (0: there is none).
struct PlanDesc { int32_t pieces, r, h, rows, first, pad[3]; };

// The workspace: descriptors of the runs, then [slot][row] of maximum and sum, then the
// weighted sums [slot][32 rows][32 features][4][lane] of 4 features each; two slots a run.
constexpr int64_t PLAN_ROWS = 128;      // largest of an item
__host__ __device__ inline int64_t plan_desc_bytes(int64_t W) { return W * (int64_t)sizeof(PlanDesc); }
__host__ __device__ inline int64_t plan_stats_bytes(int64_t W) { return 2 * W * PLAN_ROWS * 8; }

}  // namespace tpl
