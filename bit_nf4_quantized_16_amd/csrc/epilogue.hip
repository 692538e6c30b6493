// Backward of the linear layer's epilogue y = act(z) + residual, z = sum + bias
// (gfx950): dz = dy act'(z) and dbias = sum over rows of dz. dz is what the
// layer's own backward takes as dY; the residual's gradient is dy itself.
//
// HBM-bound: dy and z are read, dz is written, once. A lane has eight columns
// (16 bytes) of a row, a workgroup 512 columns (all of a narrower matrix) of a
// run of rows; the column sums stay in registers over its rows, are added over
// the workgroup through LDS and over the runs by a second launch, each in a
// fixed order. The sums take dz before its rounding. 1000 x 11008 with z in fp32
// and GELU: 17.0 us (5.2 TB/s), and 4.2 for the second launch; with z in bf16 2.8
// less for both.
#include "common.h"
#include "internal.h"

namespace qlnf4 {

namespace {

constexpr int kThreads = 256, kUnroll = 4;

template <int ACT, bool SUM, bool ZF32>
__global__ __launch_bounds__(kThreads) void epilogue_bwd_kernel(EpilogueBwdArgs p, int lanes, uint32_t blocks) {
    __shared__ float red[SUM ? kThreads * 8 : 1];
    const int slot = threadIdx.x / lanes, slots = kThreads / lanes, lane = threadIdx.x - slot * lanes;
    const uint32_t run = blockIdx.x / blocks;
    const int64_t col = 8 * (static_cast<int64_t>(blockIdx.x - run * blocks) * lanes + lane);
    const int64_t r0 = run * p.rows_per, r1 = r0 + p.rows_per < p.T ? r0 + p.rows_per : p.T;
    const bool in = col < p.N;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t r = r0 + slot; r < r1 && in; r += slots * kUnroll) {
        uint4 d[kUnroll], z[kUnroll], z2[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t row = r + u * slots < r1 ? r + u * slots : r1 - 1;  // read again, not used
            d[u] = *reinterpret_cast<const uint4*>(p.dY + row * p.N + col);
            if constexpr (ACT != QL_ACT_NONE && ZF32) {
                const uint4* const zp = reinterpret_cast<const uint4*>(static_cast<const float*>(p.Z) + row * p.N + col);
                z[u] = zp[0];
                z2[u] = zp[1];
            } else if constexpr (ACT != QL_ACT_NONE) {
                z[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.Z) + row * p.N + col);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t row = r + u * slots;
            if (row >= r1) continue;
            const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
            float zv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            uint32_t o[4];
            if constexpr (ACT != QL_ACT_NONE) {
                const uint32_t zw[8] = {z[u].x, z[u].y, z[u].z, z[u].w, z2[u].x, z2[u].y, z2[u].z, z2[u].w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    zv[i] = __uint_as_float(ZF32 ? zw[i] : i % 2 ? zw[i / 2] & 0xFFFF0000u : zw[i / 2] << 16);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float g0 = __uint_as_float(dw[q] << 16) * act_slope<ACT>(zv[2 * q]);
                const float g1 = __uint_as_float(dw[q] & 0xFFFF0000u) * act_slope<ACT>(zv[2 * q + 1]);
                o[q] = pack_bf16x2(g0, g1);
                if constexpr (SUM) {
                    s[2 * q] += g0;
                    s[2 * q + 1] += g1;
                }
            }
            if (p.dZ != nullptr) *reinterpret_cast<uint4*>(p.dZ + row * p.N + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    if constexpr (SUM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) red[threadIdx.x * 8 + i] = s[i];
        __syncthreads();
        // 8 lanes sums of `slots` values, row slot first
        const int width = 8 * lanes;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            float t = red[c];
            for (int i = 1; i < slots; ++i) t += red[i * width + c];
            const int64_t n = 8 * static_cast<int64_t>(blockIdx.x - run * blocks) * lanes + c;
            if (n < p.N) p.part[run * p.N + n] = t;
        }
    }
}

// Lanes that take a row of a workgroup's columns, workgroups along a row, runs
// of rows: about eight workgroups a CU.
struct Plan {
    int lanes;
    int64_t blocks, runs, rows_per;
};
Plan plan_of(int64_t T, int64_t N) {
    Plan p{1, 1, 1, 1};
    while (p.lanes < 64 && 8 * p.lanes < N) p.lanes *= 2;
    p.blocks = ceil_div(N, 8 * p.lanes);
    const int64_t turn = kThreads / p.lanes * kUnroll;  // rows a workgroup takes at a time
    const int64_t want = std::max<int64_t>(1, 2048 / p.blocks);
    p.rows_per = ceil_div(ceil_div(T, want), turn) * turn;
    p.runs = ceil_div(T, p.rows_per);
    return p;
}

}  // namespace

size_t epilogue_bwd_ws_bytes(int64_t T, int64_t N) {
    return T > 0 ? static_cast<size_t>(plan_of(T, N).runs) * N * sizeof(float) : 0;
}

int launch_epilogue_bwd(EpilogueBwdArgs a, hipStream_t stream) {
    timer_begin(QL_KERNEL_EPILOGUE, stream);
    int64_t runs = 0;
    if (a.T > 0) {
        const Plan pl = plan_of(a.T, a.N);
        a.rows_per = pl.rows_per;
        runs = pl.runs;
        with_act(a.act, [&](auto act) {
            const dim3 grid(static_cast<uint32_t>(pl.blocks * pl.runs));
            auto launch = [&](auto sum, auto zf32) {
                hipLaunchKernelGGL((epilogue_bwd_kernel<decltype(act)::value, decltype(sum)::value, decltype(zf32)::value>),
                                   grid, dim3(kThreads), 0, stream, a, pl.lanes, static_cast<uint32_t>(pl.blocks));
            };
            auto by_z = [&](auto sum) {
                if (decltype(act)::value != QL_ACT_NONE && a.z_f32)
                    launch(sum, std::true_type{});
                else
                    launch(sum, std::false_type{});
            };
            if (a.dB != nullptr)
                by_z(std::true_type{});
            else
                by_z(std::false_type{});
        });
    }
    if (a.dB != nullptr) launch_column_sums(a.part, runs, a.N, a.dB, nullptr, a.accumulate, stream);
    timer_end(QL_KERNEL_EPILOGUE, stream);
    return check_launch("epilogue backward");
}

}  // namespace qlnf4
