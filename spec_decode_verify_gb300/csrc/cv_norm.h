// Internal: parameters and kernel tables of the block norms.
#pragma once

#include <cuda_runtime.h>

namespace cvk {

struct NormParams {
    long long rows;
    int dim, group;
    int gate_act, gate_first;
    float eps, scale;
    const void *y, *gate, *post, *res, *cs, *pre;
    void *out, *res_out;
    long long y_row, gate_row, res_row, res_out_row, out_row;
    int lanes;  // norm_groups: lanes per group (a power of two, at most 32)
    long long ahead;  // norm_row: rows between a row and the one prefetched for it
    int flat;   // norm_groups: rows and groups lie one after the other in every tensor: each group is a row
};

using NormKernel = void (*)(NormParams);

constexpr int kNormGroupThreads = 256;
constexpr int kNormRowThreads = 512;  // norm_row: threads a row, at most
// norm_row: elements a thread, at most, for accesses of v elements.  Single elements and pairs stop at 16: with
// 32 of them a thread spills (6000 odd rows of 9999, bf16: 1257 us; norm_any 682).
constexpr int norm_row_elems(int v) { return v > 2 ? 32 : 16; }
constexpr int kNormAnyThreads = 256;

constexpr int kNormUnroll = 2;        // norm_groups: groups a thread loads at once

// Groups of at most 32 lanes * nv accesses (vec: 16 bytes, nv 1 or 2; else one element, nv up to 4), no residual; unroll 1 or kNormUnroll.
NormKernel norm_groups_kernel(bool bf16, bool vec, int nv, int unroll);
// One block a row, the row in registers (elems = 8, 16 or 32 elements a thread).
// v: elements an access (16 bytes of dtype, 2, or 1).
NormKernel norm_row_kernel(bool bf16, bool res_f32, int v, int elems);
// One block a row, the row read again for each pass: any dim and any group.
NormKernel norm_any_kernel(bool bf16, bool res_f32);

}  // namespace cvk
