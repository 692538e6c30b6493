// Layer norm and root-mean-square norm, forward and backward (gfx950).
//
//   mu = mean(x) (0 for the root-mean-square form), r = 1 / sqrt(mean((x - mu)^2) + eps)
//   y = h w + b, h = (x - mu) r
//   dx = r (g - mean(g) - h mean(g h)), g = dy w   (no mean(g) without a mean)
//   dw = sum_t dy h, db = sum_t dy
//
// Both are bound by HBM: x is read once and kept in registers between the
// statistics and the output, so the variance is summed from x - mu itself.
// Measured (a large copy: 5.2 TB/s): forward 4096 x 4096 bf16 12.6 us (5.3 TB/s),
// 16384 x 8192 96 (5.6); backward 4096 x 4096 with both sums 26.4 (3.8),
// 16384 x 8192 with dw 150 (5.4). Few rows are bound by their way in and out:
// 1001 x 4096 6.1 and 16.1 us, 3.9 of them the sums' second launch; one row 2.0.
// fp32, both launches, graphs of calls with outputs of their own: 16384 x 4096 103
// and 147 us (5.2 and 5.5 TB/s), 4096 x 4096 29.7 and 43, 1001 x 4096 9.0 and 16.7
// (bf16 by that method: 4096 x 4096 14.8).
#include "common.h"
#include "internal.h"
#include "reduce.h"

namespace qlnf4 {

namespace {

// VEC values of type bf16 (F32 false) or fp32 from p.
template <bool F32, int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t at, float (&v)[VEC]) {
    if constexpr (F32) {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
            const float4 f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[q];
            v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
        }
    } else {
        uint32_t w[VEC / 2];
        if constexpr (VEC == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    }
}

template <bool F32, int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t at, const float (&v)[VEC]) {
    if constexpr (F32) {
        static_assert(VEC == 4, "16 bytes");
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        static_assert(VEC == 8, "16 bytes");
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

template <bool F32, int VEC>
__device__ __forceinline__ void unpack_vec(const uint4& u, float (&v)[VEC]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        v[i] = __uint_as_float(F32 ? w[i] : i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// A row whose squares (or sum) leave fp32's range, or whose squares that count
// and v_rsq_f32's argument are flushed to zero: its values are read again, times the
// power of two that brings the largest (or eps's root) to [2, 4), for each of its
// sums and for its output. Rows of zeros and with infinite values keep what
// they have. All waves of a row come here together, and no wave reads red[2].
template <bool XF32, bool WF32>
__device__ __forceinline__ void norm_fwd_scaled(const NormArgs& p, int64_t row, int first, int step, int wave, int waves,
                                             float (*red)[16]) {
    constexpr int VEC = XF32 ? 4 : 8;
    const int64_t base = row * p.C;
    float k = 1.0f;
    auto sum = [&](auto f, float start, auto op, int at) {
        float s[1] = {start};
#pragma unroll 1
        for (int c = first * VEC; c < p.C; c += step * VEC) {
            float x[VEC];
            load_vec<XF32, VEC>(p.X, base + c, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = f(x[i] * k, s[0]);
        }
        block_reduce(s, red[at], wave, waves, op);
        return s[0];
    };
    const float m = sum([](float x, float s) { return fmaxf(fabsf(x), s); }, __builtin_sqrtf(p.eps), MaxOp{}, 2);
    const int e = static_cast<int>(__float_as_uint(m) >> 23);
    const int up = m > 0.0f && e < 255 ? 128 - max(1, e) : 0;
    k = power2(up);
    const float inv = 1.0f / static_cast<float>(p.C);
    float mu = 0.0f;
    if (!p.rms) mu = inv * sum([](float x, float s) { return s + x; }, 0.0f, AddOp{}, 0);
    const float var = sum([&](float x, float s) { return __builtin_fmaf(x - mu, x - mu, s); }, 0.0f, AddOp{}, 1);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(var, inv, p.eps * k * k));
#pragma unroll 1
    for (int c = first * VEC; c < p.C; c += step * VEC) {
        float x[VEC], w[VEC], b[VEC];
        load_vec<XF32, VEC>(p.X, base + c, x);
        load_vec<WF32, VEC>(p.w, c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = 0.0f;
        if (p.b != nullptr) load_vec<WF32, VEC>(p.b, c, b);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = __builtin_fmaf((x[i] * k - mu) * r, w[i], b[i]);
        store_vec<XF32, VEC>(p.Y, base + c, x);
    }
    if (first == 0) {
        if (p.mean != nullptr) p.mean[row] = ldexpf(mu, -up);
        if (p.rstd != nullptr) p.rstd[row] = ldexpf(r, up);
    }
}

// A row by `waves` waves (the workgroup's, or one of its four), a lane NV
// pieces of 16 bytes of x; weight and bias are on their way with it.
template <bool XF32, bool WF32, int NV>
__global__ __launch_bounds__(1024) void norm_fwd_kernel(NormArgs p, int waves) {
    constexpr int VEC = XF32 ? 4 : 8;
    __shared__ float red[3][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = waves == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + wave : blockIdx.x;
    if (row >= p.T) return;  // a whole wave, and only where no barrier follows
    const int first = waves == 1 ? lane : threadIdx.x, step = 64 * waves;
    const int C = p.C;
    const int64_t base = row * C;

    float x[NV][VEC], w[NV][VEC], b[NV][VEC];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (first + j * step) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[j][i] = b[j][i] = 0.0f;
        if (c < C) {
            load_vec<XF32, VEC>(p.X, base + c, x[j]);
            load_vec<WF32, VEC>(p.w, c, w[j]);
            if (p.b != nullptr) load_vec<WF32, VEC>(p.b, c, b[j]);
        }
    }
    float mu = 0.0f;
    const float inv = 1.0f / static_cast<float>(C);
    if (!p.rms) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += x[j][i];
        block_reduce(s, red[0], wave, waves, AddOp{});
        mu = s[0] * inv;
    }
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const bool in = (first + j * step) * VEC < C;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            x[j][i] = in ? x[j][i] - mu : 0.0f;
            s[0] = __builtin_fmaf(x[j][i], x[j][i], s[0]);
        }
    }
    block_reduce(s, red[1], wave, waves, AddOp{});
    const float var = __builtin_fmaf(s[0], inv, p.eps);
    if (!(var >= 0x1p-100f && var < __builtin_inff()))
        return norm_fwd_scaled<XF32, WF32>(p, row, first, step, wave, waves, red);
    const float r = __builtin_amdgcn_rsqf(var);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (first + j * step) * VEC;
        if (c >= C) continue;
        float y[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[i] = __builtin_fmaf(x[j][i] * r, w[j][i], b[j][i]);
        store_vec<XF32, VEC>(p.Y, base + c, y);
    }
    if (first == 0) {
        if (p.mean != nullptr) p.mean[row] = mu;
        if (p.rstd != nullptr) p.rstd[row] = r;
    }
}

// A workgroup takes `slots` rows at a time, `waves` waves each, and goes on
// gridDim turns further; a row's loads are under way while the one before is
// worked on. A thread keeps its columns' sums of dy h and dy over its rows; the
// slots' are added through LDS, the workgroups' left in part: one array of C
// sums a CU, so that they cost little beside the rows (512 workgroups' sums for
// 1001 x 4096 are two thirds of the rows' bytes: 14.1 and 6.5 us for the two
// launches, with 256 12.4 and 3.9).
// SUMS: none, dw's, dw's and db's.
template <bool XF32, bool WF32, int NV, int SUMS>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(NormArgs p, int waves, int slots) {
    constexpr int VEC = XF32 ? 4 : 8;
    constexpr bool AHEAD = !XF32 || NV < 4;  // else out of registers
    __shared__ float red[2][16][2][16];  // a slot's two sums over its waves
    extern __shared__ __attribute__((aligned(16))) float sums[];  // [slots - 1][C]
    const int tid = threadIdx.x, slot = tid / (64 * waves), first = tid - slot * 64 * waves, wave = first >> 6;
    const int C = p.C, step = 64 * waves;
    const float inv = 1.0f / static_cast<float>(C);
    const bool rms = p.rms;
    float sw[NV][VEC], sb[NV][VEC];
    constexpr int WW = WF32 ? VEC : VEC / 2;  // words of VEC weights, as stored
    uint32_t w[NV][WW];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = min((first + j * step) * VEC, C - VEC);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sw[j][i] = sb[j][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < WW; ++i)
            w[j][i] = reinterpret_cast<const uint32_t*>(static_cast<const char*>(p.w) + c * (WF32 ? 4 : 2))[i];
    }
    auto weight = [&](int j, int i) {
        return __uint_as_float(WF32 ? w[j][i] : i % 2 ? w[j][i / 2] & 0xFFFF0000u : w[j][i / 2] << 16);
    };
    // Loads without a branch (past the edges the last row's or pieces', not
    // used): behind one the compiler waits for them at once.
    uint4 xr[NV], dr[NV];
    float r, mu;
    const float* const means = rms ? p.rstd : p.mean;
    auto load = [&](int64_t row) {
        const int64_t at = (row < p.T ? row : p.T - 1);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t o = (at * C + min((first + j * step) * VEC, C - VEC)) * (XF32 ? 4 : 2);
            xr[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.X) + o);
            dr[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.dY) + o);
        }
        r = p.rstd[at];
        mu = means[at];
    };
    const int64_t turn_rows = static_cast<int64_t>(gridDim.x) * slots;
    int64_t r0 = static_cast<int64_t>(blockIdx.x) * slots;
    if (AHEAD) load(r0 + slot);
    for (int turn = 0; r0 < p.T; r0 += turn_rows, turn ^= 1) {
        const int64_t row = r0 + slot, base = row * C;
        const bool live = row < p.T;
        if (!AHEAD) load(row);
        const float rr = r, m = rms ? 0.0f : mu;
        float h[NV][VEC], g[NV][VEC];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack_vec<XF32, VEC>(xr[j], h[j]);
            unpack_vec<XF32, VEC>(dr[j], g[j]);
        }
        if (AHEAD) load(row + turn_rows);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = live && (first + j * step) * VEC < C;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[j][i] = in ? (h[j][i] - m) * rr : 0.0f;
                g[j][i] = in ? g[j][i] : 0.0f;
                if constexpr (SUMS > 0) sw[j][i] = __builtin_fmaf(g[j][i], h[j][i], sw[j][i]);
                if constexpr (SUMS > 1) sb[j][i] += g[j][i];
                g[j][i] *= weight(j, i);
                s[0] = __builtin_fmaf(g[j][i], h[j][i], s[0]);
                s[1] += g[j][i];
            }
        }
        if (p.dX == nullptr) continue;
        block_reduce(s, red[turn][slot][0], wave, waves, AddOp{}, AddOp{});
        const float gh = s[0] * inv, gm = rms ? 0.0f : s[1] * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (first + j * step) * VEC;
            if (c >= C || !live) continue;
            float d[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) d[i] = rr * (__builtin_fmaf(-gh, h[j][i], g[j][i]) - gm);
            store_vec<XF32, VEC>(p.dX, base + c, d);
        }
    }
    if constexpr (SUMS > 0) {
        // the first slot's threads add the others' to theirs
        auto leave = [&](float* to, const float (&v)[NV][VEC]) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (first + j * step) * VEC;
                if (c >= C) continue;
#pragma unroll
                for (int i = 0; i < VEC; i += 4)
                    *reinterpret_cast<float4*>(to + c + i) = make_float4(v[j][i], v[j][i + 1], v[j][i + 2], v[j][i + 3]);
            }
        };
        auto finish = [&](float (&v)[NV][VEC], bool wanted, int array) {
            if (!wanted) return;
            if (slots > 1) {
                if (slot > 0) leave(sums + (slot - 1) * C, v);
                __syncthreads();
            }
            if (slot == 0) {
                for (int o = 0; o < slots - 1; ++o)
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int c = (first + j * step) * VEC;
                        if (c >= C) continue;
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[j][i] += sums[o * C + c + i];
                    }
                leave(p.part + (static_cast<int64_t>(array) * gridDim.x + blockIdx.x) * C, v);
            }
        };
        finish(sw, p.dW != nullptr, 0);
        if constexpr (SUMS > 1) {
            if (slots > 1 && p.dW != nullptr) __syncthreads();  // dW's sums have been read
            finish(sb, true, 1);
        }
    }
}

// Column sums of part [arrays][parts][C], in order: 32 columns (a line) a
// workgroup by 32 threads each, which have eight loads under way.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* part, int64_t parts, int64_t C, float* out0,
                                                           float* out1, int accumulate) {
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
    float* const out = blockIdx.y == 0 ? out0 : out1;
    if (out == nullptr) return;
    const float* const src = part + blockIdx.y * parts * C;
    float s = 0.0f;
    if (c < C) {
        for (int64_t g = k; g < parts; g += 256) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = g + 32 * u < parts ? src[(g + 32 * u) * C + c] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
    }
    red[k][col] = s;
    __syncthreads();
    if (threadIdx.x < 32 && c < C) {
        float t = red[0][col];
        for (int i = 1; i < 32; ++i) t += red[i][col];
        out[c] = accumulate ? out[c] + t : t;
    }
}

// f(x fp32, w fp32, pieces a lane): at most 16 values a lane, two pieces of bf16
// or four of fp32.
template <typename F>
void norm_dispatch(const NormArgs& a, int nv, F f) {
    auto by_nv = [&](auto xf, auto wf) {
        if (nv == 1) {
            f(xf, wf, std::integral_constant<int, 1>{});
        } else if (nv == 2) {
            f(xf, wf, std::integral_constant<int, 2>{});
        } else if constexpr (decltype(xf)::value) {
            f(xf, wf, std::integral_constant<int, 4>{});
        }
    };
    if (a.x_f32)
        a.w_f32 ? by_nv(std::true_type{}, std::true_type{}) : by_nv(std::true_type{}, std::false_type{});
    else
        a.w_f32 ? by_nv(std::false_type{}, std::true_type{}) : by_nv(std::false_type{}, std::false_type{});
}

// How a row is dealt out: pieces of 16 bytes a lane (`want` where the row is
// long enough, so that few waves have to meet; more where 16 waves ask for it),
// waves.
struct RowPlan {
    int nv, waves;
};
RowPlan row_plan(int64_t C, bool f32, int want) {
    const int pieces = static_cast<int>(ceil_div(C, f32 ? 4 : 8));
    RowPlan r{1, 1};
    while (r.nv < want && 64 * r.nv < pieces) r.nv *= 2;
    while (r.waves < 16 && 64 * r.nv * r.waves < pieces) r.waves *= 2;
    while (64 * r.nv * r.waves < pieces) r.nv *= 2;
    return r;
}

// The backward's: how a row is dealt out, rows at a time of a workgroup,
// workgroups (at most one a CU). Measured (us, slots x waves of a row, pieces a
// lane):
//   1001 x 4096   1x8,1 16.1 | 2x8,1 16.4 | 1x4,2 18.5
//   4096 x 4096   1x8,1 28.9 | 2x8,1 26.6 | 2x4,2 31.2,  16384 x 4096 92.4 | 87.4 | 102.6
//   4096 x 8192   1x16,1 50.1 | 1x8,2 60.9;  dw alone 16384 x 8192 166.6 | 150.6 | 2x8,2 157.3
//   4096 x 1024   1x2,1 18.5 | 2x2,1 13.6 | 4x2,1 12.0 | 8x2,1 12.9
//   8192 x 512    1x1,1 21.4 | 4x1,1 12.1 | 8x1,1 12.1 | 16x1,1 13.0,  600 x 512 6.9 | 6.8 | 7.4 | 9.4
// So one piece a lane where 16 waves then hold the row (two sums spill 13 registers
// with two: layer norm rows over 8192 bf16 values, 2000 x 16384 64 us, 3.1 TB/s), two
// for the root mean square's long rows, whose db is seldom wanted (4096 x 8192 43
// us, with db 62; the plan takes no notice of what is asked for: the same bits
// either way); up to
// four rows and eight waves at a time, 16 where there are many rows of eight.
struct BwdPlan {
    RowPlan row;
    int slots;
    int64_t groups;
};
BwdPlan bwd_plan(int64_t T, int64_t C, bool f32, bool rms) {
    const int64_t pieces = ceil_div(C, f32 ? 4 : 8);
    BwdPlan b{row_plan(C, f32, pieces > (rms ? 512 : 1024) ? 2 : 1), 1, 0};
    const int waves = b.row.waves;
    const int most = waves < 8 ? 8 : b.row.nv == 1 && T >= 4096 ? 16 : 8;
    while (b.slots < 4 && b.slots * waves < most && b.slots < T) b.slots *= 2;
    b.groups = std::min<int64_t>(ceil_div(T, b.slots), 256);
    return b;
}

}  // namespace

void launch_column_sums(const float* part, int64_t parts, int64_t C, float* out0, float* out1, int accumulate,
                        hipStream_t stream) {
    hipLaunchKernelGGL(column_sums_kernel, dim3(static_cast<uint32_t>(ceil_div(C, 32)), out1 != nullptr ? 2 : 1), dim3(1024),
                       0, stream, part, parts, C, out0, out1, accumulate);
}

int launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
    const RowPlan r = row_plan(a.C, a.x_f32, 2);
    const int rows = r.waves == 1 ? 4 : 1;
    timer_begin(QL_KERNEL_NORM, stream);
    norm_dispatch(a, r.nv, [&](auto xf, auto wf, auto nv) {
        hipLaunchKernelGGL((norm_fwd_kernel<decltype(xf)::value, decltype(wf)::value, decltype(nv)::value>),
                           dim3(static_cast<uint32_t>(ceil_div(a.T, rows))), dim3(64 * r.waves * rows), 0, stream, a,
                           r.waves);
    });
    timer_end(QL_KERNEL_NORM, stream);
    return check_launch("norm forward");
}

// (of every plan)
size_t norm_bwd_ws_bytes(int64_t T, int64_t C) {
    return static_cast<size_t>(std::min<int64_t>(T, 256)) * C * 2 * sizeof(float);
}

int launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
    const BwdPlan b = bwd_plan(a.T, a.C, a.x_f32, a.rms);
    const RowPlan r = b.row;
    const int slots = b.slots;
    const int64_t groups = b.groups;
    const bool grads = a.dW != nullptr || a.dB != nullptr;
    timer_begin(QL_KERNEL_NORM, stream);
    if (groups > 0)
        norm_dispatch(a, r.nv, [&](auto xf, auto wf, auto nv) {
            const dim3 grid(static_cast<uint32_t>(groups)), block(64 * r.waves * slots);
            const uint32_t lds = grads ? (slots - 1) * a.C * sizeof(float) : 0;  // at most 16 KiB
            auto launch = [&](auto sums) {
                hipLaunchKernelGGL((norm_bwd_kernel<decltype(xf)::value, decltype(wf)::value, decltype(nv)::value,
                                                    decltype(sums)::value>),
                                   grid, block, lds, stream, a, r.waves, slots);
            };
            if (a.dB != nullptr) launch(std::integral_constant<int, 2>{});
            else if (grads) launch(std::integral_constant<int, 1>{});
            else launch(std::integral_constant<int, 0>{});
        });
    if (grads) launch_column_sums(a.part, groups, a.C, a.dW, a.dB, a.accumulate, stream);
    timer_end(QL_KERNEL_NORM, stream);
    return check_launch("norm backward");
}

}  // namespace qlnf4
