// Losses on logits [T, V] with their gradients (gfx950): the preference loss on
// paired log ratios of packed sequences, and distillation from a teacher's top
// logits. All are bound by HBM: a row of logits is V values to read and V to
// write, with a maximum and a sum of exponentials in between.
//
// A row starts at any element: up to seven values before the first 16-byte
// boundary and after the last one (the edges) go to single lanes, the pieces of
// 16 bytes between them to whole lanes. Exponentials are 2^((z - m) log2 e):
// the difference first, so that logits near the type's limits do not overflow
// in the product.
#include "common.h"
#include "internal.h"
#include "reduce.h"

namespace qlnf4 {

namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// Where the pieces of a row lie.
struct RowShape {
    const char* body;  // the first piece
    int head, pieces, tail;
};

template <bool F32>
__device__ __forceinline__ RowShape row_shape(const char* row, int V) {
    constexpr int E = F32 ? 4 : 8, B = F32 ? 4 : 2;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / B;
    RowShape s;
    s.head = off == 0 ? 0 : min(E - off, V);
    s.pieces = (V - s.head) / E;
    s.tail = V - s.head - s.pieces * E;
    s.body = row + s.head * B;
    return s;
}

template <bool F32>
__device__ __forceinline__ float load_one(const char* row, int64_t j) {
    if constexpr (F32) return reinterpret_cast<const float*>(row)[j];
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[j]);
}
template <bool F32>
__device__ __forceinline__ void store_one(char* row, int64_t j, float v) {
    if constexpr (F32)
        reinterpret_cast<float*>(row)[j] = v;
    else
        reinterpret_cast<uint16_t*>(row)[j] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Column of the edge value that this thread has, or -1: head values to
// threads 0.., tail values to threads 8...
__device__ __forceinline__ int edge_column(const RowShape& s, int V, int tid) {
    if (tid < s.head) return tid;
    if (tid >= 8 && tid - 8 < s.tail) return V - s.tail + (tid - 8);
    return -1;
}

// The values of a piece.
template <bool F32>
struct Piece {
    static constexpr int E = F32 ? 4 : 8;
    uint4 u;
    __device__ __forceinline__ float at(int i) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (F32) return __uint_as_float(w[i]);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    // all -inf: neutral to the maximum and the sum
    __device__ __forceinline__ void clear() {
        const uint32_t n = F32 ? 0xFF800000u : 0xFF80FF80u;
        u = make_uint4(n, n, n, n);
    }
};
template <bool F32>
__device__ __forceinline__ uint4 pack_piece(const float (&g)[F32 ? 4 : 8]) {
    if constexpr (F32)
        return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
    else
        return make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// What exponentials are taken against: the maximum, or zero for a row of
// -inf (whose sum then is zero, not NaN).
__device__ __forceinline__ float reference(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// A running maximum and sum of 2^((z - m) c).
struct Running {
    float m = -__builtin_inff(), s = 0.0f;
};
__device__ __forceinline__ void rescale(Running& r, float m, float c) {
    if (m > r.m) {
        r.s = r.s == 0.0f ? 0.0f : r.s * exp2_((r.m - m) * c);
        r.m = m;
    }
}

// ---------------------------------------------------------------------------
// Preference loss. Rows of the logits are tokens, sequences are runs of rows,
// pairs are neighbouring sequences.
//   l_t = z_t[label] - lse(z_t)       a launch over rows (and slices of them)
//   L_s, the loss and dloss / dl_t    a workgroup per pair
//   dz_t = dloss dl_t (onehot - softmax)   a launch over rows
// ---------------------------------------------------------------------------
constexpr int kStatThreads = 256, kStatUnroll = 4;

// From the label's logit, the reference and the sum: the log probability, and
// what the gradient takes softmax from (not their sum, the row's log-sum-exp,
// whose rounding would cost softmax half a unit in the last place of it).
__device__ __forceinline__ void finish_row(const LogpArgs& p, int64_t t, float z, float ref, float s) {
    p.logp[t] = (z - ref) - kLn2 * __builtin_amdgcn_logf(s);
    if (p.ref == nullptr) return;
    p.ref[t] = ref;
    p.inv[t] = 1.0f / s;
}

template <bool F32>
__global__ __launch_bounds__(kStatThreads) void logp_kernel(LogpArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E;
    __shared__ float red[2][16];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int64_t t = blockIdx.x / p.slices;
    const int slice = static_cast<int>(blockIdx.x - t * p.slices);
    const int64_t label = p.labels[t];
    if (tid == 0 && slice == 0 && p.dlogp != nullptr) {
        p.dlogp[t] = 0.0f;  // until its pair says otherwise
        p.pair[t] = 0;
    }
    if (label < 0 || label >= p.V) {
        if (tid == 0 && slice == 0) p.logp[t] = 0.0f;
        return;
    }
    const char* const row = static_cast<const char*>(p.z) + t * p.ld * (F32 ? 4 : 2);
    const RowShape sh = row_shape<F32>(row, p.V);
    const int per = (sh.pieces + p.slices - 1) / p.slices;
    const int first = slice * per, last = min(first + per, sh.pieces);
    Running r;
    const int edge = slice == 0 ? edge_column(sh, p.V, tid) : -1;
    if (edge >= 0) {
        r.m = load_one<F32>(row, edge);
        r.s = exp2_((r.m - reference(r.m)) * kLog2e);
    }
    for (int c0 = first + tid; c0 < last; c0 += kStatThreads * kStatUnroll) {
        P v[kStatUnroll];
#pragma unroll
        for (int j = 0; j < kStatUnroll; ++j) {
            v[j].clear();
            const int c = c0 + j * kStatThreads;
            if (c < last) v[j].u = *reinterpret_cast<const uint4*>(sh.body + 16 * static_cast<int64_t>(c));
        }
        float m = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < kStatUnroll; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) m = fmaxf(m, v[j].at(i));
        rescale(r, m, kLog2e);
        const float ref = reference(r.m);
#pragma unroll
        for (int j = 0; j < kStatUnroll; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) r.s += exp2_((v[j].at(i) - ref) * kLog2e);
    }
    float m[1] = {r.m};
    block_reduce(m, red[0], wave, kStatThreads / 64, MaxOp{});
    rescale(r, m[0], kLog2e);
    float s[1] = {r.s};
    block_reduce(s, red[1], wave, kStatThreads / 64, AddOp{});
    if (tid != 0) return;
    if (p.slices > 1) {
        p.part[2 * (t * p.slices + slice)] = m[0];
        p.part[2 * (t * p.slices + slice) + 1] = s[0];
        return;
    }
    finish_row(p, t, load_one<F32>(row, label), reference(m[0]), s[0]);
}

// The slices of a row joined, a thread a row.
template <bool F32>
__global__ __launch_bounds__(256) void logp_join_kernel(LogpArgs p) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (t >= p.T) return;
    const int64_t label = p.labels[t];
    if (label < 0 || label >= p.V) return;  // written already
    Running r;
    for (int i = 0; i < p.slices; ++i) r.m = fmaxf(r.m, p.part[2 * (t * p.slices + i)]);
    const float ref = reference(r.m);
    for (int i = 0; i < p.slices; ++i) {
        const float m = p.part[2 * (t * p.slices + i)], s = p.part[2 * (t * p.slices + i) + 1];
        r.s += s == 0.0f ? 0.0f : s * exp2_((m - ref) * kLog2e);
    }
    finish_row(p, t, load_one<F32>(static_cast<const char*>(p.z) + t * p.ld * (F32 ? 4 : 2), label), ref, r.s);
}

constexpr int kPairThreads = 1024;

// log(1 + e^-|x|) and the two logistic values in 64 bits: one thread a pair.
__device__ void pair_loss(const PairArgs& p, double d, double& loss, double& slope) {
    const double x = p.beta * d;
    if (p.kind == QL_PREF_SIGMOID) {
        const double e = exp(-fabs(x)), soft = log1p(e);
        const double lo = e / (1.0 + e), hi = 1.0 / (1.0 + e);  // sigmoid(-|x|), sigmoid(|x|)
        const double up = x >= 0 ? hi : lo, down = x >= 0 ? lo : hi;  // sigmoid(x), sigmoid(-x)
        // -log sigmoid(x) = soft + max(-x, 0)
        loss = (1.0 - p.smooth) * (soft + fmax(-x, 0.0)) + (p.smooth > 0.0f ? p.smooth * (soft + fmax(x, 0.0)) : 0.0);
        slope = p.beta * (p.smooth * up - (1.0 - p.smooth) * down);
        if (x != x) loss = slope = x;
    } else if (p.kind == QL_PREF_HINGE) {
        loss = x < 1.0 ? 1.0 - x : (x != x ? x : 0.0);
        slope = x < 1.0 ? -static_cast<double>(p.beta) : (x != x ? x : 0.0);
    } else {
        const double e = d - 0.5 / p.beta;
        loss = e * e;
        slope = 2.0 * e;
    }
}

__global__ __launch_bounds__(kPairThreads) void pair_kernel(PairArgs p) {
    __shared__ double sums[2][kPairThreads / 64];
    __shared__ int64_t counts[2][kPairThreads / 64];
    __shared__ float slopes[2];
    const int tid = threadIdx.x, wave = tid >> 6, pair = blockIdx.x;
    int64_t at[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t a = p.start[2 * pair + i];
        at[i] = a < 0 ? 0 : (a > p.T ? p.T : a);
    }
    for (int q = 0; q < 2; ++q) {
        double s = 0.0;
        int64_t n = 0;
        for (int64_t t = at[q] + tid; t < at[q + 1]; t += kPairThreads) {
            const int64_t label = p.labels[t];
            if (label < 0 || label >= p.V) continue;
            s += p.logp[t];
            ++n;
        }
        for (int d = 32; d > 0; d >>= 1) {
            s += __shfl_xor(s, d);
            n += __shfl_xor(n, d);
        }
        if ((tid & 63) == 0) {
            sums[q][wave] = s;
            counts[q][wave] = n;
        }
    }
    __syncthreads();
    if (tid == 0) {
        double L[2], per[2];
        for (int q = 0; q < 2; ++q) {
            double s = 0.0;
            int64_t n = 0;
            for (int w = 0; w < kPairThreads / 64; ++w) {
                s += sums[q][w];
                n += counts[q][w];
            }
            per[q] = p.average && n > 0 ? 1.0 / static_cast<double>(n) : 1.0;
            L[q] = s * per[q];
            p.seq_logp[2 * pair + q] = static_cast<float>(L[q]);
        }
        double loss, slope;
        pair_loss(p, (L[0] - p.ref[2 * pair]) - (L[1] - p.ref[2 * pair + 1]), loss, slope);
        p.loss[pair] = static_cast<float>(loss);
        slopes[0] = static_cast<float>(slope * per[0]);
        slopes[1] = static_cast<float>(-slope * per[1]);
    }
    __syncthreads();
    for (int q = 0; q < 2; ++q)
        for (int64_t t = at[q] + tid; t < at[q + 1]; t += kPairThreads) {
            const int64_t label = p.labels[t];
            if (label < 0 || label >= p.V) continue;
            p.dlogp[t] = slopes[q];
            p.pair[t] = pair;
        }
}

// dz = f (onehot - softmax), f = dloss dlogp; a row that counts nothing is
// written as zeros without being read.
constexpr int kGradThreads = 256, kGradUnroll = 4;

template <bool F32>
__global__ __launch_bounds__(kGradThreads) void logp_grad_kernel(LogpGradArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E;
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / p.slices;
    const int slice = static_cast<int>(blockIdx.x - t * p.slices);
    const int64_t bytes = t * p.ld * (F32 ? 4 : 2);
    const char* const row = static_cast<const char*>(p.z) + bytes;
    char* const out = static_cast<char*>(p.dz) + bytes;
    const int64_t label = p.labels[t];
    const bool on = label >= 0 && label < p.V && p.pairs > 0;
    const float f = on ? p.dlogp[t] * p.dloss[p.pair[t]] : 0.0f;
    const float ref = on ? p.ref[t] : 0.0f, fq = on ? -f * p.inv[t] : 0.0f;
    const RowShape sh = row_shape<F32>(out, p.V);
    const int64_t body = sh.body - out;
    const int per = (sh.pieces + p.slices - 1) / p.slices;
    const int first = slice * per, last = min(first + per, sh.pieces);
    const int edge = slice == 0 ? edge_column(sh, p.V, tid) : -1;
    auto value = [&](float z, int col) {
        return __builtin_fmaf(fq, exp2_((z - ref) * kLog2e), col == label ? f : 0.0f);
    };
    const bool zero = !on || f == 0.0f;
    if (edge >= 0) store_one<F32>(out, edge, zero ? 0.0f : value(load_one<F32>(row, edge), edge));
    for (int c0 = first + tid; c0 < last; c0 += kGradThreads * kGradUnroll) {
        P v[kGradUnroll];
        if (!zero) {
#pragma unroll
            for (int j = 0; j < kGradUnroll; ++j) {
                const int c = c0 + j * kGradThreads;
                if (c < last) v[j].u = *reinterpret_cast<const uint4*>(row + body + 16 * static_cast<int64_t>(c));
            }
        }
#pragma unroll
        for (int j = 0; j < kGradUnroll; ++j) {
            const int c = c0 + j * kGradThreads;
            if (c >= last) continue;
            uint4 o = make_uint4(0, 0, 0, 0);
            if (!zero) {
                float g[E];
#pragma unroll
                for (int i = 0; i < E; ++i) g[i] = value(v[j].at(i), sh.head + c * E + i);
                o = pack_piece<F32>(g);
            }
            *reinterpret_cast<uint4*>(out + body + 16 * static_cast<int64_t>(c)) = o;
        }
    }
}

// Slices of a row where there are few rows.
int logp_slices(int64_t T, int64_t V, bool f32) {
    const int64_t pieces = V / (f32 ? 4 : 8);
    const int64_t most = std::max<int64_t>(1, pieces / (kStatThreads * 2));
    return static_cast<int>(std::min(most, std::max<int64_t>(1, 512 / std::max<int64_t>(T, 1))));
}
int grad_slices(int64_t V, bool f32) {
    const int64_t pieces = V / (f32 ? 4 : 8);
    return static_cast<int>(std::max<int64_t>(1, pieces / (kGradThreads * kGradUnroll)));
}

// ---------------------------------------------------------------------------
// Distillation. p = softmax over the teacher's K logits / tau, q = softmax of
// the row / tau:
//   loss = (1 - a) tau^2 sum_k p_k (log p_k - log q_k) + a (lse(z) - z[label])
//   dz   = w ((1 - a) tau (q - p) + a (softmax(z) - onehot))
// A workgroup a row, the row in registers (NV pieces a thread) between its
// sums and its gradient, so it is read once; NV = 0 reads a longer one again.
// The gradient is written without the p and the onehot first; then a thread
// per teacher entry (and one for the label) writes its column's value with
// everything that falls on this column, so that equal entries write equal
// values.
// ---------------------------------------------------------------------------
constexpr int kTop = QL_DISTILL_MAX_TOP;

// BOTH: the row's softmax at temperature 1 besides the one at tau.
template <bool F32, int NV, bool BOTH>
__global__ __launch_bounds__(1024) void distill_kernel(DistillArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E;
    __shared__ float red[3][48];
    __shared__ float s_p[kTop + 1];
    __shared__ int s_k[kTop + 1];
    const int tid = threadIdx.x, wave = tid >> 6, threads = blockDim.x, waves = threads >> 6;
    const int64_t t = blockIdx.x, bytes = t * p.ld * (F32 ? 4 : 2);
    const char* const row = static_cast<const char*>(p.z) + bytes;
    char* const out = p.dz != nullptr ? static_cast<char*>(p.dz) + bytes : nullptr;
    const RowShape sh = row_shape<F32>(row, p.V);
    const int64_t body = sh.body - row;
    const int edge = edge_column(sh, p.V, tid);
    const int64_t label = p.labels != nullptr ? p.labels[t] : 0;
    if (label < 0 || label >= p.V) {  // not counted
        if (tid == 0 && p.loss != nullptr) p.loss[t] = 0.0f;
        if (out != nullptr) {
            if (edge >= 0) store_one<F32>(out, edge, 0.0f);
            for (int c = tid; c < sh.pieces; c += threads)
                *reinterpret_cast<uint4*>(out + body + 16 * static_cast<int64_t>(c)) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const float ninf = -__builtin_inff();
    const float ct = kLog2e / p.tau;
    P v[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j].clear();
            const int c = tid + j * threads;
            if (c < sh.pieces) v[j].u = *reinterpret_cast<const uint4*>(sh.body + 16 * static_cast<int64_t>(c));
        }
    }
    const float ze = edge >= 0 ? load_one<F32>(row, edge) : ninf;
    // the teacher's entry of this thread; the thread after them has the label
    float top = ninf, zk = 0.0f;
    int k = -1;
    if (tid < p.K) {
        const int64_t at = p.index[t * p.K + tid];
        if (at >= 0 && at < p.V) {
            k = static_cast<int>(at);
            top = p.top_f32 ? static_cast<const float*>(p.top)[t * p.K + tid]
                            : bf16_to_f32(static_cast<const uint16_t*>(p.top)[t * p.K + tid]);
        }
    } else if (tid == p.K && p.alpha > 0.0f) {
        k = static_cast<int>(label);
    }
    if (k >= 0) zk = load_one<F32>(row, k);

    float mx[2] = {ze, top};
    Running r1, rt;  // NV = 0: running sums
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) mx[0] = fmaxf(mx[0], v[j].at(i));
    } else {
        constexpr int U = 4;
        for (int c0 = tid; c0 < sh.pieces; c0 += threads * U) {
            P u[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                u[j].clear();
                const int c = c0 + j * threads;
                if (c < sh.pieces) u[j].u = *reinterpret_cast<const uint4*>(sh.body + 16 * static_cast<int64_t>(c));
            }
            float m = ninf;
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) m = fmaxf(m, u[j].at(i));
            rescale(rt, m, ct);
            rescale(r1, m, kLog2e);
            const float ref = reference(rt.m);
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = u[j].at(i) - ref;
                    rt.s += exp2_(d * ct);
                    if constexpr (BOTH) r1.s += exp2_(d * kLog2e);
                }
        }
        mx[0] = fmaxf(mx[0], rt.m);
    }
    block_reduce(mx, red[0], wave, waves, MaxOp{}, MaxOp{});
    const float m = reference(mx[0]);
    // sums: at tau, at 1, of the teacher's exponentials
    float s[3] = {exp2_((ze - m) * ct), BOTH ? exp2_((ze - m) * kLog2e) : 0.0f, 0.0f};
    const float lt = (top - reference(mx[1])) * ct;  // log2 of the unnormalised p
    const float et = exp2_(lt);
    s[2] = tid < p.K ? et : 0.0f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float d = v[j].at(i) - m;
                s[0] += exp2_(d * ct);
                if constexpr (BOTH) s[1] += exp2_(d * kLog2e);
            }
    } else {
        rescale(rt, mx[0], ct);
        s[0] += rt.s;
        if constexpr (BOTH) {
            rescale(r1, mx[0], kLog2e);
            s[1] += r1.s;
        }
    }
    block_reduce(s, red[1], wave, waves, AddOp{}, AddOp{}, AddOp{});
    if constexpr (!BOTH) s[1] = s[0];  // tau = 1, or not used
    const float kl = s[2] != 0.0f ? (1.0f - p.alpha) * p.tau : 0.0f;  // no entry: no such term
    // this thread's part of the loss, and what its column's gradient loses
    float part[1] = {0.0f}, loses = 0.0f;
    if (tid < p.K && et != 0.0f && kl != 0.0f) {
        const float pk = et / s[2];
        const float log_p = lt - __builtin_amdgcn_logf(s[2]), log_q = (zk - m) * ct - __builtin_amdgcn_logf(s[0]);
        part[0] = kl * p.tau * pk * ((log_p - log_q) * kLn2);
        loses = kl * pk;
    } else if (tid == p.K && k >= 0) {
        part[0] = p.alpha * (kLn2 * __builtin_amdgcn_logf(s[1]) - (zk - m));
        loses = p.alpha;
    }
    if (tid <= p.K) {
        s_p[tid] = loses;
        s_k[tid] = k;
    }
    block_reduce(part, red[2], wave, waves, AddOp{});
    if (waves == 1) __syncthreads();
    if (tid == 0 && p.loss != nullptr) p.loss[t] = part[0];
    if (out == nullptr) return;

    const float w = p.weight != nullptr ? p.weight[t] : 1.0f;
    const float ft = w * (BOTH || p.alpha == 0.0f ? kl : kl + p.alpha) / s[0], f1 = BOTH ? w * p.alpha / s[1] : 0.0f;
    auto value = [&](float z) {
        const float d = z - m;
        float g = ft * exp2_(d * ct);
        if constexpr (BOTH) g = __builtin_fmaf(f1, exp2_(d * kLog2e), g);
        return g;
    };
    auto put = [&](const P& u, int c) {
        float g[E];
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] = value(u.at(i));
        *reinterpret_cast<uint4*>(out + body + 16 * static_cast<int64_t>(c)) = pack_piece<F32>(g);
    };
    if (edge >= 0) store_one<F32>(out, edge, value(ze));
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = tid + j * threads;
            if (c < sh.pieces) put(v[j], c);
        }
    } else {
        for (int c = tid; c < sh.pieces; c += threads) {
            P u;
            u.u = *reinterpret_cast<const uint4*>(sh.body + 16 * static_cast<int64_t>(c));
            put(u, c);
        }
    }
    __syncthreads();  // the row's values before its entries'
    if (k >= 0) {
        float sum = 0.0f;
        for (int i = 0; i <= p.K; ++i) sum += s_k[i] == k ? s_p[i] : 0.0f;
        store_one<F32>(out, k, __builtin_fmaf(-w, sum, value(zk)));
    }
}

template <bool F32, bool BOTH>
void launch_distill_nv(const DistillArgs& a, hipStream_t stream) {
    const int64_t pieces = a.V / (F32 ? 4 : 8);
    const int threads = pieces <= 1024 ? 512 : 1024;
    const int64_t need = std::max<int64_t>(1, ceil_div(pieces, threads));
    const dim3 grid(static_cast<uint32_t>(a.T)), block(threads);
    if (need <= 1) hipLaunchKernelGGL((distill_kernel<F32, 1, BOTH>), grid, block, 0, stream, a);
    else if (need <= 2) hipLaunchKernelGGL((distill_kernel<F32, 2, BOTH>), grid, block, 0, stream, a);
    else if (need <= 4) hipLaunchKernelGGL((distill_kernel<F32, 4, BOTH>), grid, block, 0, stream, a);
    else if (need <= 8) hipLaunchKernelGGL((distill_kernel<F32, 8, BOTH>), grid, block, 0, stream, a);
    else if (need <= 16) hipLaunchKernelGGL((distill_kernel<F32, 16, BOTH>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((distill_kernel<F32, 0, BOTH>), grid, block, 0, stream, a);
}

}  // namespace

size_t logp_ws_bytes(int64_t T, int64_t V, bool f32) {
    const int n = logp_slices(T, V, f32);
    return n > 1 ? static_cast<size_t>(T) * n * 2 * sizeof(float) : 0;
}

int launch_logp(LogpArgs a, hipStream_t stream) {
    a.slices = logp_slices(a.T, a.V, a.f32);
    timer_begin(QL_KERNEL_LOGP, stream);
    const dim3 grid(static_cast<uint32_t>(a.T * a.slices)), rows(static_cast<uint32_t>(ceil_div(a.T, 256)));
    if (a.f32) {
        hipLaunchKernelGGL(logp_kernel<true>, grid, dim3(kStatThreads), 0, stream, a);
        if (a.slices > 1) hipLaunchKernelGGL(logp_join_kernel<true>, rows, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(logp_kernel<false>, grid, dim3(kStatThreads), 0, stream, a);
        if (a.slices > 1) hipLaunchKernelGGL(logp_join_kernel<false>, rows, dim3(256), 0, stream, a);
    }
    timer_end(QL_KERNEL_LOGP, stream);
    return check_launch("token log probabilities");
}

int launch_pairs(const PairArgs& a, int pairs, hipStream_t stream) {
    timer_begin(QL_KERNEL_PREFERENCE, stream);
    hipLaunchKernelGGL(pair_kernel, dim3(static_cast<uint32_t>(pairs)), dim3(kPairThreads), 0, stream, a);
    timer_end(QL_KERNEL_PREFERENCE, stream);
    return check_launch("preference loss");
}

int launch_logp_grad(LogpGradArgs a, hipStream_t stream) {
    a.slices = grad_slices(a.V, a.f32);
    timer_begin(QL_KERNEL_LOGP_GRAD, stream);
    const dim3 grid(static_cast<uint32_t>(a.T * a.slices));
    if (a.f32)
        hipLaunchKernelGGL(logp_grad_kernel<true>, grid, dim3(kGradThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(logp_grad_kernel<false>, grid, dim3(kGradThreads), 0, stream, a);
    timer_end(QL_KERNEL_LOGP_GRAD, stream);
    return check_launch("preference loss backward");
}

int launch_distill(const DistillArgs& a, hipStream_t stream) {
    timer_begin(QL_KERNEL_DISTILL, stream);
    const bool both = a.alpha > 0.0f && a.tau != 1.0f;
    if (a.f32)
        both ? launch_distill_nv<true, true>(a, stream) : launch_distill_nv<true, false>(a, stream);
    else
        both ? launch_distill_nv<false, true>(a, stream) : launch_distill_nv<false, false>(a, stream);
    timer_end(QL_KERNEL_DISTILL, stream);
    return check_launch("distillation loss");
}

}  // namespace qlnf4
