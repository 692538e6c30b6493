// Adapter gradients from an 8-bit checkpoint of the layer's input (gfx950,
// bf16 MFMA): reductions over the tokens
//
//   out[j][c] (dA) or out[c][j] (dB) = scale * sum_t V[t][j] M[t][c]
//
// with M = X (8-bit checkpoint, the dropout mask applied where there is one)
// and V = G = s dY B for dA; M = dY (bf16) and V = U for dB. V comes as fp32
// and is not rounded: it is split into three bf16 terms v = h + m + l (each
// the rounding of what the ones before it leave, 24 bits in all), multiplied
// by the exact bf16 values of M and summed in fp32, so dA and dB carry fp32
// rounding only. One grid holds both problems: workgroups [0, nblk0) take
// 64-column blocks of the first, the rest those of the second.
//
// A workgroup's eight waves take 32-token chunks in turn. A wave expands its
// chunk of M to bf16 in a private LDS tile and reads it back column-wise
// (eight consecutive tokens of one column per lane: the MFMA B operand); its
// chunk of V goes through a second tile, one term at a time, and is read the
// same way (the A operand). With one token split the workgroup writes the
// gradient itself (fixed-order sum of the waves); with several, fp32 partials
// go to the workspace and a second kernel adds them in order.
#include <algorithm>

#include "act8.h"
#include "common.h"
#include "internal.h"
#include "mm_common.h"

namespace qlnf4 {

namespace {

constexpr int kCols = 64;   // columns of M per workgroup
constexpr int kRows = 32;   // tokens per MFMA step
constexpr int kWaves = 8;
constexpr int kLdM = kCols + 8;

// 16-bit lane masks of eight elements from their eight keep bits.
__device__ __forceinline__ uint4 keep_mask(uint32_t bits) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = ((bits >> (2 * q)) & 1u ? 0x0000FFFFu : 0u) | ((bits >> (2 * q + 1)) & 1u ? 0xFFFF0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The next bf16 term of v and what it leaves (exact; nothing once a term is
// infinite or NaN, so that an infinite v stays infinite).
__device__ __forceinline__ float split_term(float& v) {
    const float h = __uint_as_float(pack_bf16x2(v, 0.0f) << 16);
    v = fabsf(h) < __builtin_inff() ? v - h : 0.0f;
    return h;
}

template <int RT>
__global__ __launch_bounds__(64 * kWaves) void act8_grads_kernel(Act8GradArgs a) {
    constexpr int LdV = 16 * RT + 8;
    constexpr int kTile = kRows * (kLdM + LdV);
    __shared__ __attribute__((aligned(16))) uint16_t sm[kWaves][kTile];
    __shared__ float red[kWaves / 2][16][kCols];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g = lane >> 4;
    const bool second = static_cast<int>(blockIdx.x) >= a.nblk0;
    const Act8GradProblem& pb = second ? a.pb[1] : a.pb[0];
    const int64_t C = pb.C;
    const int64_t c0 = static_cast<int64_t>(second ? blockIdx.x - a.nblk0 : blockIdx.x) * kCols;
    const int64_t tb = blockIdx.y * a.t_per;
    const int64_t te = std::min<int64_t>(tb + a.t_per, a.T);
    const int r = a.r;
    f32x4 acc[RT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) acc[rt][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint16_t* const tm = sm[wave];
    uint16_t* const tv = sm[wave] + kRows * kLdM;

    // lane: row (lane / 8) + 8 i of the chunk, columns c0 + 8 (lane % 8) ..
    const int64_t c = c0 + 8 * (lane & 7);
    auto load_m = [&](int64_t t, uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = t + (lane >> 3) + 8 * i;
            v[i] = make_uint4(0, 0, 0, 0);
            if (row < te && c < C) {
                const int64_t e = row * C + c;
                if (pb.scale8 != nullptr) {
                    v[i] = act8_decode8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pb.M) + e),
                                        pb.scale8[e / kAct8Block]);
                    if (pb.keep != nullptr) {
                        const uint4 m = keep_mask(pb.keep[e / 8]);
                        v[i] = make_uint4(v[i].x & m.x, v[i].y & m.y, v[i].z & m.z, v[i].w & m.w);
                    }
                } else {
                    v[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pb.M) + e);
                }
            }
        }
    };
    // V of the chunk: quads of ranks, 4 RT a token (zero past the rank and the tokens)
    auto load_v = [&](int64_t t, float (&v)[2 * RT][4]) {
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) {
            const int q = lane + 64 * i;
            const int64_t row = t + q / (4 * RT);
            const int j = 4 * (q % (4 * RT));
            const float* p = pb.V + row * r + j;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = 0.0f;
            if (row < te) {
                if ((r & 3) == 0) {
                    if (j < r) {
                        const float4 f = *reinterpret_cast<const float4*>(p);
                        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < r) v[i][e] = p[e];
                }
            }
        }
    };

    uint4 mcur[4];
    float vcur[2 * RT][4];
    int64_t t = tb + kRows * wave;
    if (t < te) {
        load_m(t, mcur);
        load_v(t, vcur);
    }
    for (; t < te; t += kWaves * kRows) {
        wave_lds_sync();  // the previous chunk's reads are done
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(tm + ((lane >> 3) + 8 * i) * kLdM + 8 * (lane & 7)) = mcur[i];
        bf16x8_t bv[4];
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            if (term > 0) wave_lds_sync();
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i) {
                const int q = lane + 64 * i;
                float h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = split_term(vcur[i][e]);
                *reinterpret_cast<uint2*>(tv + (q / (4 * RT)) * LdV + 4 * (q % (4 * RT))) =
                    make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
            }
            wave_lds_sync();
            if (term == 0) {
#pragma unroll
                for (int cb = 0; cb < 4; ++cb) bv[cb] = lds_col8(tm, kLdM, 8 * g, 16 * cb, li);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const bf16x8_t av = lds_col8(tv, LdV, 8 * g, 16 * rt, li);
#pragma unroll
                for (int cb = 0; cb < 4; ++cb)
                    acc[rt][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv[cb], acc[rt][cb], 0, 0, 0);
            }
        }
        const int64_t tn = t + kWaves * kRows;
        if (tn < te) {
            load_m(tn, mcur);
            load_v(tn, vcur);
        }
    }
    // D[j = 4 g + q][column li] of each tile: waves 4..7 hand theirs to waves
    // 0..3, whose sums are then added in order
    const bool direct = gridDim.y == 1;
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if ((wave >= kWaves / 2) == (half == 1)) {
                float(*const rw)[kCols] = red[wave % (kWaves / 2)];
#pragma unroll
                for (int cb = 0; cb < 4; ++cb)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float& d = rw[4 * g + q][16 * cb + li];
                        d = half == 1 ? acc[rt][cb][q] : acc[rt][cb][q] + d;
                    }
            }
            __syncthreads();
        }
        for (int e = tid; e < 16 * kCols; e += 64 * kWaves) {
            // consecutive threads along the output's contiguous direction
            const int jl = pb.layout_jc ? e / kCols : e % 16, cl = pb.layout_jc ? e % kCols : e / 16;
            const int j = 16 * rt + jl;
            const int64_t cc = c0 + cl;
            if (cc >= C) continue;
            float v = red[0][jl][cl];
#pragma unroll
            for (int ww = 1; ww < kWaves / 2; ++ww) v += red[ww][jl][cl];
            if (direct) {
                if (j < r) {
                    const int64_t idx = pb.layout_jc ? j * C + cc : cc * r + j;
                    const float o = pb.scale * v;
                    pb.out[idx] = a.accumulate ? pb.out[idx] + o : o;
                }
            } else {
                pb.part[(static_cast<int64_t>(blockIdx.y) * RT * 16 + j) * C + cc] = v;
            }
        }
        __syncthreads();
    }
}

// Sum of the token splits of both problems, in split order.
__global__ __launch_bounds__(256) void act8_grads_final_kernel(Act8GradArgs a, int splits, int rpad) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t n0 = static_cast<int64_t>(a.r) * a.pb[0].C;
    const int64_t n1 = static_cast<int64_t>(a.r) * a.pb[1].C;
    if (idx >= n0 + n1) return;
    const bool second = idx >= n0;
    const Act8GradProblem& pb = second ? a.pb[1] : a.pb[0];
    const int64_t e = second ? idx - n0 : idx;
    const int64_t j = pb.layout_jc ? e / pb.C : e % a.r, c = pb.layout_jc ? e % pb.C : e / a.r;
    float s = 0.0f;
    for (int ts = 0; ts < splits; ++ts) s += pb.part[(static_cast<int64_t>(ts) * rpad + j) * pb.C + c];
    const float v = pb.scale * s;
    pb.out[e] = a.accumulate ? pb.out[e] + v : v;
}

int splits_of(int64_t T, int64_t cols_total) {
    // one split (no second kernel) while a workgroup's token loop stays short
    if (T <= 2048 || cols_total <= 0) return 1;
    const int64_t s = std::min(ceil_div(512, ceil_div(cols_total, kCols)), ceil_div(T, kWaves * kRows));
    return static_cast<int>(std::max<int64_t>(s, 1));
}

}  // namespace

size_t act8_grads_part_bytes(int64_t T, int64_t C0, int64_t C1, int r) {
    const int sp = splits_of(T, C0 + C1);
    return sp == 1 ? 0 : static_cast<size_t>(sp) * lora_grad_rp(r) * (C0 + C1) * sizeof(float);
}

int launch_act8_grads(Act8GradArgs a, float* part, hipStream_t stream) {
    if (a.pb[0].out == nullptr) {  // only the second problem: move it first
        a.pb[0] = a.pb[1];
        a.pb[1] = Act8GradProblem{};
    }
    if (a.pb[0].out == nullptr) return QL_OK;
    if (a.pb[1].out == nullptr) a.pb[1].C = 0;
    const int64_t c0 = a.pb[0].C, c1 = a.pb[1].C;
    const int rp16 = lora_grad_rp(a.r);
    const int splits = splits_of(a.T, c0 + c1);
    a.t_per = ceil_div(ceil_div(a.T, splits), kWaves * kRows) * kWaves * kRows;
    a.nblk0 = static_cast<int>(ceil_div(c0, kCols));
    if (splits > 1) {
        if (part == nullptr) return set_error(QL_ERR_WORKSPACE, "adapter gradients: workspace missing");
        a.pb[0].part = part;
        a.pb[1].part = part + static_cast<size_t>(splits) * rp16 * c0;
    }
    const dim3 grid(static_cast<uint32_t>(a.nblk0 + ceil_div(c1, kCols)), static_cast<uint32_t>(splits));
    timer_begin(QL_KERNEL_ACT8_GRAD, stream);
    switch (rp16 / 16) {
#define QL_CASE(R_)                                                                                  \
    case R_:                                                                                         \
        hipLaunchKernelGGL(act8_grads_kernel<R_>, grid, dim3(64 * kWaves), 0, stream, a);            \
        break;
        QL_CASE(1)
        QL_CASE(2)
        QL_CASE(3)
        QL_CASE(4)
        QL_CASE(5)
        QL_CASE(6)
        QL_CASE(7)
        QL_CASE(8)
#undef QL_CASE
        default:
            return set_error(QL_ERR_SHAPE, "adapter gradients: rank %d out of range", a.r);
    }
    if (splits > 1)
        hipLaunchKernelGGL(act8_grads_final_kernel,
                           dim3(static_cast<uint32_t>(ceil_div(static_cast<int64_t>(a.r) * (c0 + c1), 256))),
                           dim3(256), 0, stream, a, splits, rp16);
    timer_end(QL_KERNEL_ACT8_GRAD, stream);
    return check_launch("adapter gradients from an 8-bit checkpoint");
}

}  // namespace qlnf4
