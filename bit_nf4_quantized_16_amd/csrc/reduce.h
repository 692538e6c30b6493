// Reductions over a wave and over the waves of a row (gfx950), for the kernels
// that work row by row. Sums are added in a fixed order and every lane gets
// the same bits.
#pragma once

#include "common.h"

namespace qlnf4 {

struct AddOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// Over the 64 lanes, in every lane: four DPP steps inside 16 lanes, then two
// lane-group swaps (no LDS traffic).
template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
    v = op(v, dpp_f<0xB1>(v));   // quad_perm [1,0,3,2]
    v = op(v, dpp_f<0x4E>(v));   // quad_perm [2,3,0,1]
    v = op(v, dpp_f<0x141>(v));  // row_half_mirror
    v = op(v, dpp_f<0x140>(v));  // row_mirror
    const uint32_t b = __float_as_uint(v);
    const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    v = op(__uint_as_float(s[0]), __uint_as_float(s[1]));
    const uint32_t c = __float_as_uint(v);
    const auto t = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return op(__uint_as_float(t[0]), __uint_as_float(t[1]));
}

// Several values over the workgroup's `waves` waves (1 to 16): lds holds
// 16 * N floats that no wave still reads. Every wave has to come here; the
// next use of the same lds needs a barrier in between (or another lds).
template <int N, typename... Op>
__device__ __forceinline__ void block_reduce(float (&v)[N], float* lds, int wave, int waves, Op... ops) {
    static_assert(sizeof...(Op) == N, "one operation a value");
    int i = 0;
    ((v[i] = wave_reduce(v[i], ops), ++i), ...);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int j = 0; j < N; ++j) lds[j * 16 + wave] = v[j];
    __syncthreads();
    i = 0;
    auto join = [&](auto op) {
        float r = lds[i * 16];
        for (int w = 1; w < waves; ++w) r = op(r, lds[i * 16 + w]);
        v[i++] = r;
    };
    (join(ops), ...);
}

}  // namespace qlnf4
