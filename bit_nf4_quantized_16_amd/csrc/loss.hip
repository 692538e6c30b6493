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

// Streaming (nontemporal) accesses, for gradients, which nothing here reads
// again, and for the last reading of logits: they leave the last-level cache to
// the logits between the preference loss's passes (us; plain, stores, loads too:
// 3500 x 32000 bf16 114, 96, 90; 6001 x 50257 fp32 495, 473, 460; distillation at
// 4000 x 128000 bf16 461, 442, 433).
typedef uint32_t u32x4_stream __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_stream(char* p, const uint4& v) {
    __builtin_nontemporal_store(u32x4_stream{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_stream*>(p));
}
__device__ __forceinline__ uint4 load_stream(const char* p) {
    const u32x4_stream v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_stream*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
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

// Exponentials against the maximum m: 2^(z c - m c), one multiply-add. The
// rounding of m c is the same for all and is taken off the logarithm of their
// sum (delta). Up to |m c| = 2^30 that rounding is at most 32, so the sum keeps
// its bits. Past it, values next to each other (an fp32 step is over 2^-24 of the
// value) are at least 64 apart in z c, so that only those equal to m count (a
// row's others together are under 2^30 2^-64): a power of two that brings m to
// 2^30 or more in c's place gives them exactly 1 and the others as little.
struct Scale {
    float c, mc, delta;
};
__device__ __forceinline__ Scale scale_of(float m, float c) {
    Scale s;
    const float mc = m * c;
    const bool far = !(fabsf(mc) <= 0x1p30f);
    s.c = far ? __uint_as_float((284u - (__float_as_uint(m) >> 23 & 255u)) << 23) : c;
    s.mc = far ? m * s.c : mc;
    s.delta = far ? 0.0f : __builtin_fmaf(m, c, -mc);
    return s;
}
__device__ __forceinline__ float exp_of(float z, const Scale& s) { return exp2_(__builtin_fmaf(z, s.c, -s.mc)); }
// A running sum of such exponentials, which carries 2^delta of its maximum's
// scale, brought to a new maximum: delta changes with it. (fp32 logits around
// 1e6 have deltas of up to 2^-4; without them the sums of rows that a maximum
// rises over many times were off by 1e-3.) Two maxima lie at least a delta apart
// in z c, so the exponent's roundings are under 2^-21 of that distance.
__device__ __forceinline__ void rescale(Running& r, Scale& s, float m, float c) {
    if (!(m > r.m)) return;
    const Scale to = scale_of(reference(m), c);
    r.s = r.s == 0.0f ? 0.0f : r.s * exp2_((r.m - m) * c - s.delta + to.delta);
    r.m = m;
    s = to;
}

// The largest of m and a piece's values.
template <bool F32>
__device__ __forceinline__ float piece_max(const Piece<F32>& v, float m) {
#pragma unroll
    for (int i = 0; i < Piece<F32>::E; ++i) m = fmaxf(m, v.at(i));
    return m;
}

// ---------------------------------------------------------------------------
// Preference loss. Rows of the logits are tokens, sequences are runs of rows,
// pairs are neighbouring sequences.
//   l_t = z_t[label] - lse(z_t)       a wave per 512 pieces of a row
//   L_s, the loss and dloss / dl_t    a workgroup per pair
//   dz_t = dloss dl_t (onehot - softmax)   workgroups of 1024 pieces of a row
// A pair's sums must be known before any of its gradient, so the logits are
// read twice. The second pass takes the rows from the last to the first, which
// the first pass has left in the last-level cache.
// ---------------------------------------------------------------------------
constexpr int kLogpThreads = 256, kLogpPieces = 8;  // pieces a lane
constexpr int kLogpRun = 64 * kLogpPieces;          // and a wave

// Maximum and sum of 2^((z - m) log2 e) of a row's runs of pieces, a wave
// each, all its loads in flight at once; no wave waits for another. HBM-bound:
// 2450 rows of 32000 bf16 27.6 us (5.7 TB/s), 3000 of 50257 fp32 99 (6.1). (A row
// a workgroup of 256, two barriers: 45.8 us for the first.) A workgroup's waves
// take the same run of neighbouring rows, whose results lie side by side (four
// runs of a row each: 1 to 2 us more for the loss and its gradient).
template <bool F32>
__global__ __launch_bounds__(kLogpThreads) void logp_kernel(LogpArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E;
    const int lane = threadIdx.x & 63;
    const uint32_t rows = blockIdx.x / p.runs;
    const int run = static_cast<int>(blockIdx.x - rows * p.runs);
    const int64_t t = static_cast<int64_t>(rows) * (kLogpThreads / 64) + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const int64_t label = p.labels[t];
    if (run == 0 && lane == 0 && p.dlogp != nullptr) {
        p.dlogp[t] = 0.0f;  // until its pair says otherwise
        p.pair[t] = 0;
        p.pair_logp[t] = 0.0f;
    }
    if (label < 0 || label >= p.V) return;
    const char* const row = static_cast<const char*>(p.z) + t * p.ld * (F32 ? 4 : 2);
    const RowShape sh = row_shape<F32>(row, p.V);
    const int first = run * kLogpRun + lane;
    P v[kLogpPieces];
#pragma unroll
    for (int j = 0; j < kLogpPieces; ++j) {
        v[j].clear();
        const int c = first + 64 * j;
        if (c < sh.pieces) v[j].u = *reinterpret_cast<const uint4*>(sh.body + 16 * static_cast<int64_t>(c));
    }
    float m = -__builtin_inff();
    const int edge = run == 0 ? edge_column(sh, p.V, lane) : -1;
    const float ze = edge >= 0 ? load_one<F32>(row, edge) : m;
#pragma unroll
    for (int j = 0; j < kLogpPieces; ++j) m = piece_max(v[j], m);
    m = wave_reduce(fmaxf(m, ze), MaxOp{});
    const Scale sc = scale_of(reference(m), kLog2e);
    float s = exp_of(ze, sc);
#pragma unroll
    for (int j = 0; j < kLogpPieces; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) s += exp_of(v[j].at(i), sc);
    s = wave_reduce(s, AddOp{});
    // of the exact argument: the scale's rounding off
    if (lane == 0) reinterpret_cast<float2*>(p.part)[run * p.T + t] = make_float2(m, s * exp2_(-sc.delta));
}

// A row's runs joined, eight loads under way at a time: what exponentials are
// taken against, their sum. Neighbouring threads have neighbouring rows, and the
// runs lie [run][row] so that a wave's load is a few lines (as [row][run] the
// join of 3000 rows of 25 took 18 us, so 11).
__device__ __forceinline__ float2 join_runs(const float* part, int runs, int64_t T, int64_t t) {
    const float2* const v = reinterpret_cast<const float2*>(part) + t;
    Running r;
    for (int i0 = 0; i0 < runs; i0 += 8) {
        float2 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i0 + i < runs ? v[(i0 + i) * T] : make_float2(-__builtin_inff(), 0.0f);
        float m = r.m;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, u[i].x);
        rescale(r, m, kLog2e);
        const float ref = reference(m);
#pragma unroll
        for (int i = 0; i < 8; ++i) r.s += u[i].y == 0.0f ? 0.0f : u[i].y * exp2_((u[i].x - ref) * kLog2e);
    }
    return make_float2(reference(r.m), r.s < __builtin_inff() ? r.s : __builtin_nanf(""));
}
__device__ __forceinline__ float label_logit(const void* z, int f32, int64_t at) {
    return f32 ? static_cast<const float*>(z)[at] : bf16_to_f32(static_cast<const uint16_t*>(z)[at]);
}

// The log probabilities alone: both launches 28.9 us for 2048 x 32000 bf16 (4.5
// TB/s), 176 for 4000 x 128000 (5.8), 106 for 3000 x 50257 fp32, 5.7 for one row.
__global__ __launch_bounds__(256) void logp_join_kernel(LogpArgs p) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (t >= p.T) return;
    const int64_t label = p.labels[t];
    float l = 0.0f;
    if (label >= 0 && label < p.V) {
        const float z = label_logit(p.z, p.f32, t * p.ld + label);
        const float2 r = join_runs(p.part, p.runs, p.T, t);
        l = (z - r.x) - kLn2 * __builtin_amdgcn_logf(r.y);
    }
    p.logp[t] = l;
}

constexpr int kPairThreads = 1024;

// The loss of x = beta d and dloss / dd.
__device__ __forceinline__ void pair_loss(const PairArgs& p, double d, float& loss, double& slope) {
    const double x = p.beta * d;
    if (p.kind == QL_PREF_SIGMOID) {
        // with e = e^-|x|: -log sigmoid(x) = log1p(e) + max(-x, 0), sigmoid(-|x|) = e / (1 + e)
        const float xf = static_cast<float>(x), e = expf(-fabsf(xf)), soft = log1pf(e);
        const float lo = e / (1.0f + e), hi = 1.0f / (1.0f + e);
        const float up = xf >= 0 ? hi : lo, down = xf >= 0 ? lo : hi;  // sigmoid(x), sigmoid(-x)
        // a term of weight 0 is none, also where it is infinite
        loss = (p.smooth < 1.0f ? (1.0f - p.smooth) * (soft + fmaxf(-xf, 0.0f)) : 0.0f) +
               (p.smooth > 0.0f ? p.smooth * (soft + fmaxf(xf, 0.0f)) : 0.0f);
        slope = p.beta * (p.smooth * up - (1.0f - p.smooth) * down);
        if (xf != xf) loss = xf, slope = x;
    } else if (p.kind == QL_PREF_HINGE) {
        loss = static_cast<float>(x < 1.0 ? 1.0 - x : (x != x ? x : 0.0));
        slope = x < 1.0 ? -static_cast<double>(p.beta) : (x != x ? x : 0.0);
    } else {
        const double e = d - 0.5 / p.beta;
        loss = static_cast<float>(e * e);
        slope = 2.0 * e;
    }
}

// Joins its rows' runs (their log probabilities, references and sums are kept
// for the caller and the gradient), sums them, and hands each row its share of
// the loss's slope. Bound by latency, a chain of few loads and sums on one CU a
// pair: one pair of 16 rows 4.0 us, four of 875 (8 runs) 7.5, eight of 750 (25)
// 11.1; more CUs would take one more launch, 3 us.
__global__ __launch_bounds__(kPairThreads) void pair_kernel(PairArgs p) {
    __shared__ double sums[2][kPairThreads / 64];
    __shared__ int counts[2][kPairThreads / 64];
    __shared__ float slopes[2];
    const int tid = threadIdx.x, wave = tid >> 6, pair = blockIdx.x;
    int64_t at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int64_t a = p.start[2 * pair + i];
        at[i] = a < 0 ? 0 : (a > p.T ? p.T : a);
    }
    const float ref0 = p.ref_logp[2 * pair], ref1 = p.ref_logp[2 * pair + 1];
    // both sequences' rows in one go
    double s[2] = {0.0, 0.0};
    int n[2] = {0, 0};
    for (int64_t t = at[0] + tid; t < at[2]; t += kPairThreads) {
        const int64_t label = p.labels[t];
        const int q = t >= at[1];
        float l = 0.0f;
        if (label >= 0 && label < p.V) {
            const float z = label_logit(p.z, p.f32, t * p.ld + label);
            const float2 r = join_runs(p.part, p.runs, p.T, t);
            l = (z - r.x) - kLn2 * __builtin_amdgcn_logf(r.y);
            p.ref[t] = r.x;
            p.inv[t] = 1.0f / r.y;
            n[0] += q == 0;
            n[1] += q;
        }
        p.logp[t] = l;
        s[0] += q == 0 ? l : 0.0f;
        s[1] += q == 0 ? 0.0f : l;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        for (int d = 32; d > 0; d >>= 1) {
            s[q] += __shfl_xor(s[q], d);
            n[q] += __shfl_xor(n[q], d);
        }
        if ((tid & 63) == 0) {
            sums[q][wave] = s[q];
            counts[q][wave] = n[q];
        }
    }
    __syncthreads();
    if (tid == 0) {
        double L[2], per[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            double s = 0.0;
            int n = 0;
            for (int w = 0; w < kPairThreads / 64; ++w) {
                s += sums[q][w];
                n += counts[q][w];
            }
            per[q] = p.average && n > 0 ? 1.0 / static_cast<double>(n) : 1.0;
            L[q] = s * per[q];
            p.seq_logp[2 * pair + q] = static_cast<float>(L[q]);
        }
        float loss;
        double slope;
        pair_loss(p, (L[0] - ref0) - (L[1] - ref1), loss, slope);
        p.loss[pair] = loss;
        slopes[0] = static_cast<float>(slope * per[0]);
        slopes[1] = static_cast<float>(-slope * per[1]);
    }
    __syncthreads();
    for (int64_t t = at[0] + tid; t < at[2]; t += kPairThreads) {
        const int64_t label = p.labels[t];
        if (label < 0 || label >= p.V) continue;
        p.dlogp[t] = slopes[t >= at[1]];
        p.pair[t] = pair;
    }
}

// dz = f (onehot - softmax), f = dloss dlogp; a row that counts nothing is
// written as zeros without being read. HBM-bound, each value on its own, 16 KiB
// of a row a workgroup: 3500 x 32000 bf16 with 2450 rows read 54 us (7.0 TB/s,
// the last rows' reads from the last-level cache), 6001 x 50257 fp32 with 3000
// read 340 (5.3).
constexpr int kGradThreads = 256, kGradUnroll = 4;

template <bool F32>
__global__ __launch_bounds__(kGradThreads) void logp_grad_kernel(LogpGradArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E;
    const int tid = threadIdx.x;
    const int64_t back = blockIdx.x / p.slices, t = p.T - 1 - back;
    const int slice = static_cast<int>(blockIdx.x - back * p.slices);
    const int64_t bytes = t * p.ld * (F32 ? 4 : 2);
    const char* const row = static_cast<const char*>(p.z) + bytes;
    char* const out = static_cast<char*>(p.dz) + bytes;
    const int64_t label = p.labels[t];
    const bool on = label >= 0 && label < p.V && p.pairs > 0;
    const RowShape sh = row_shape<F32>(out, p.V);
    const int64_t body = sh.body - out;
    const int first = slice * kGradThreads * kGradUnroll + tid;
    const int edge = slice == 0 ? edge_column(sh, p.V, tid) : -1;
    P v[kGradUnroll];
    float ze = 0.0f;
    if (on) {
#pragma unroll
        for (int j = 0; j < kGradUnroll; ++j) {
            const int c = first + j * kGradThreads;
            if (c < sh.pieces) v[j].u = load_stream(row + body + 16 * static_cast<int64_t>(c));
        }
        if (edge >= 0) ze = load_one<F32>(row, edge);
    }
    // a row in no sequence has no slope and no pair, whatever dloss holds
    const float slope = on ? p.dlogp[t] : 0.0f;
    const int pair = on ? p.pair[t] : 0;
    const float f = slope != 0.0f && pair >= 0 && pair < p.pairs ? slope * p.dloss[pair] : 0.0f;
    const bool zero = f == 0.0f;
    const Scale sc = scale_of(zero ? 0.0f : p.ref[t], kLog2e);
    const float fq = zero ? 0.0f : -f * p.inv[t] * exp2_(-sc.delta);
    const int at = on ? static_cast<int>(label) : -1;
    auto value = [&](float z, int col) { return __builtin_fmaf(fq, exp_of(z, sc), col == at ? f : 0.0f); };
    if (edge >= 0) store_one<F32>(out, edge, zero ? 0.0f : value(ze, edge));
#pragma unroll
    for (int j = 0; j < kGradUnroll; ++j) {
        const int c = first + j * kGradThreads;
        if (c >= sh.pieces) continue;
        uint4 o = make_uint4(0, 0, 0, 0);
        if (!zero) {
            float g[E];
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = value(v[j].at(i), sh.head + c * E + i);
            o = pack_piece<F32>(g);
        }
        store_stream(out + body + 16 * static_cast<int64_t>(c), o);
    }
}

// Waves and workgroups along a row.
int logp_runs(int64_t V, bool f32) { return static_cast<int>(std::max<int64_t>(1, ceil_div(V / (f32 ? 4 : 8), kLogpRun))); }
int grad_slices(int64_t V, bool f32) {
    return static_cast<int>(std::max<int64_t>(1, ceil_div(V / (f32 ? 4 : 8), kGradThreads * kGradUnroll)));
}

// ---------------------------------------------------------------------------
// Distillation. p = softmax over the teacher's K logits / tau, q = softmax of
// the row / tau:
//   loss = (1 - a) tau^2 sum_k p_k (log p_k - log q_k) + a (lse(z) - z[label])
//   dz   = w ((1 - a) tau (q - p) + a (softmax(z) - onehot))
// A workgroup takes a row at a time, the row in registers (NV pieces a thread)
// between its sums and its gradient, so it is read once; NV = 0 reads a longer
// one again. As a piece's gradient is written, the next row's piece is loaded
// into its registers, so that the CU's memory works while its sums are formed.
// The gradient is written without the p and the onehot first; then a thread
// per teacher entry (and one for the label) writes its column's value with
// everything that falls on this column, so that equal entries write equal
// values. HBM-bound where there are many rows (2048 x 32000 bf16, K = 64, 63 us,
// 4.1 TB/s; 4000 x 128000, K = 32 with the cross entropy, 433, 4.7), one row by
// its barriers and loads in a row (32000: 6.9 us).
// ---------------------------------------------------------------------------
constexpr int kTop = QL_DISTILL_MAX_TOP;

// Keeps the compiler from holding a piece's values unpacked from one use to
// the next, which takes twice the registers.
template <bool F32>
__device__ __forceinline__ void forget(Piece<F32>& v) {
    if constexpr (!F32) asm volatile("" : "+v"(v.u.x), "+v"(v.u.y), "+v"(v.u.z), "+v"(v.u.w));
}

// What a thread has of a row besides its pieces.
struct RowEnds {
    RowShape sh;
    bool on;   // the row counts
    int edge;  // column of its edge value or -1
    float ze;  // and the value
    int k;     // column of its teacher entry (or the label's), or -1
    float zk;  // the row's value there
    float top; // the teacher's
};

// One workgroup a CU with the chip's longest rows in registers: a workgroup goes
// from row to row. Shorter rows leave room for several workgroups, which hide
// each other's sums, and a workgroup a row is faster (us, a row each | in turns):
// bf16 8192 x 32000 205 | 226 to 248, 2000 x 65536 114 | 117, 4000 x 128000 474 |
// 454.
// A row past 16 pieces a thread is read for its sums and again for its gradient
// (from the last-level cache where that holds it), eight waves a SIMD: 2000 x
// 151936 bf16 265 us, 286 with two softmaxes (4.6 and 4.3 TB/s of one reading and
// one writing), 1000 x 262144 248, 2000 x 128000 fp32 466. Rows in turns beside the
// same rows read again (us, one softmax, two; in turns | read again): bf16 2000 x
// 70000 160, 194 | 130, 146; 1000 x 128000 122, 141 | 113, 123; 4000 x 128000 434,
// 495 | 430, 462; fp32 2000 x 50257 186, 199 | 190, 190; 3000 x 65000 342, 367 | 363,
// 365. So turns gain for fp32 with one softmax and lose for bf16, whose two
// softmaxes spill 11 registers (one: 2).
constexpr bool distill_loops(int threads, int nv) { return threads == 1024 && nv == 16; }

// GRAD: the gradient too. BOTH: the row's softmax at temperature 1 besides the
// one at tau.
template <bool F32, int THREADS, int NV, bool GRAD, bool BOTH>
__global__ __launch_bounds__(THREADS, NV == 16 || NV == 0 ? 4 : NV == 8 ? (BOTH ? 6 : 7) : 8) void distill_kernel(DistillArgs p) {
    using P = Piece<F32>;
    constexpr int E = P::E, WAVES = THREADS / 64, B = F32 ? 4 : 2;
    constexpr bool LOOP = distill_loops(THREADS, NV);
    __shared__ float red[3][48];
    __shared__ float s_p[kTop + 1];
    __shared__ int s_k[kTop + 1];
    const int tid = threadIdx.x, wave = tid >> 6;
    const uint32_t mine = 16u * tid;
    const float ninf = -__builtin_inff();
    const float ct = kLog2e / p.tau;

    auto begin_row = [&](int64_t t) {
        RowEnds r;
        const char* const row = static_cast<const char*>(p.z) + t * p.ld * B;
        r.sh = row_shape<F32>(row, p.V);
        const int64_t label = p.labels != nullptr ? p.labels[t] : 0;
        r.on = label >= 0 && label < p.V;
        r.edge = edge_column(r.sh, p.V, tid);
        r.ze = ninf;
        r.k = -1;
        r.top = ninf;
        r.zk = 0.0f;
        if (r.on) {
            if (r.edge >= 0) r.ze = load_one<F32>(row, r.edge);
            if (tid < p.K) {
                const int64_t at = p.index[t * p.K + tid];
                if (at >= 0 && at < p.V) {
                    r.k = static_cast<int>(at);
                    r.top = p.top_f32 ? static_cast<const float*>(p.top)[t * p.K + tid]
                                      : bf16_to_f32(static_cast<const uint16_t*>(p.top)[t * p.K + tid]);
                }
            } else if (tid == p.K && p.alpha > 0.0f) {
                r.k = static_cast<int>(label);
            }
            if (r.k >= 0) r.zk = load_one<F32>(row, r.k);
        }
        return r;
    };
    // piece j of this thread: a base that is the same for all and 32 bits of its own
    // (streaming unless it is read again, by the second pass over a long row)
    auto load_piece = [&](const RowEnds& r, int j, bool again = false) {
        P u;
        u.clear();
        if (r.on && tid + j * THREADS < r.sh.pieces)
            u.u = again ? *reinterpret_cast<const uint4*>(r.sh.body + static_cast<int64_t>(j) * THREADS * 16 + mine)
                        : load_stream(r.sh.body + static_cast<int64_t>(j) * THREADS * 16 + mine);
        return u;
    };

    int64_t t = blockIdx.x;
    RowEnds cur = begin_row(t);
    P v[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = load_piece(cur, j);
    }
    while (true) {
        const int64_t tn = t + gridDim.x;
        const bool more = LOOP && tn < p.T;
        float loss = 0.0f, ft = 0.0f, f1 = 0.0f, w = 0.0f;
        Scale st{}, s1{};
        if (cur.on) {
            float mx[2] = {cur.ze, cur.top};
            Running r1, rt;  // NV = 0: running sums and their scales
            Scale u1 = scale_of(0.0f, kLog2e), ut = scale_of(0.0f, ct);
            if constexpr (NV > 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j) mx[0] = piece_max(v[j], mx[0]);
#pragma unroll
                for (int j = 0; j < NV; ++j) forget(v[j]);
            } else {
                constexpr int U = 4;
                for (int c0 = 0; c0 * THREADS < cur.sh.pieces; c0 += U) {
                    P u[U];
#pragma unroll
                    for (int j = 0; j < U; ++j) u[j] = load_piece(cur, c0 + j, GRAD);
                    float m = ninf;
#pragma unroll
                    for (int j = 0; j < U; ++j) m = piece_max(u[j], m);
                    rescale(rt, ut, m, ct);
                    if constexpr (BOTH) rescale(r1, u1, m, kLog2e);
#pragma unroll
                    for (int j = 0; j < U; ++j)
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            rt.s += exp_of(u[j].at(i), ut);
                            if constexpr (BOTH) r1.s += exp_of(u[j].at(i), u1);
                        }
                }
                mx[0] = fmaxf(mx[0], rt.m);
            }
            block_reduce(mx, red[0], wave, WAVES, MaxOp{}, MaxOp{});
            const float m = reference(mx[0]);
            st = scale_of(m, ct);
            if constexpr (BOTH) s1 = scale_of(m, kLog2e);
            // sums: at tau, at 1, of the teacher's exponentials
            float s[3] = {exp_of(cur.ze, st), BOTH ? exp_of(cur.ze, s1) : 0.0f, 0.0f};
            const float lt = (cur.top - reference(mx[1])) * ct;  // log2 of the unnormalised p
            const float et = exp2_(lt);
            s[2] = tid < p.K ? et : 0.0f;
            if constexpr (NV > 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        s[0] += exp_of(v[j].at(i), st);
                        if constexpr (BOTH) s[1] += exp_of(v[j].at(i), s1);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int j = 0; j < NV; ++j) forget(v[j]);
            } else {
                // a thread's sums against its own maximum, brought to the row's
                rescale(rt, ut, m, ct);
                s[0] += rt.s;
                if constexpr (BOTH) {
                    rescale(r1, u1, m, kLog2e);
                    s[1] += r1.s;
                }
            }
            block_reduce(s, red[1], wave, WAVES, AddOp{}, AddOp{}, AddOp{});
            if constexpr (!BOTH) s[1] = s[0];  // tau = 1, or not used
            if (!(s[0] < __builtin_inff())) s[0] = s[1] = __builtin_nanf("");  // an infinite logit
            const float kl = s[2] != 0.0f ? (1.0f - p.alpha) * p.tau : 0.0f;  // no entry: no such term
            // this thread's part of the loss, and what its column's gradient loses
            float part[1] = {0.0f}, loses = 0.0f;
            if (tid < p.K && et != 0.0f && kl != 0.0f) {
                const float pk = et / s[2];
                const float log_p = lt - __builtin_amdgcn_logf(s[2]);
                const float log_q = (cur.zk - m) * ct - (__builtin_amdgcn_logf(s[0]) - st.delta);
                part[0] = kl * p.tau * pk * ((log_p - log_q) * kLn2);
                loses = kl * pk;
            } else if (tid == p.K && cur.k >= 0) {
                part[0] = p.alpha * (kLn2 * (__builtin_amdgcn_logf(s[1]) - (BOTH ? s1.delta : st.delta)) - (cur.zk - m));
                loses = p.alpha;
            }
            if (GRAD && tid <= p.K) {
                s_p[tid] = loses;
                s_k[tid] = cur.k;
            }
            block_reduce(part, red[2], wave, WAVES, AddOp{});
            loss = part[0];
            if constexpr (GRAD) {
                w = p.weight != nullptr ? p.weight[t] : 1.0f;
                ft = w * (BOTH || p.alpha == 0.0f ? kl : kl + p.alpha) / s[0];
                if constexpr (BOTH) f1 = w * p.alpha / s[1];
            }
        }
        if (tid == 0 && p.loss != nullptr) p.loss[t] = loss;

        RowEnds nxt = cur;
        if constexpr (LOOP) {
            nxt.on = false;
            if (more) nxt = begin_row(tn);
        }
        char* const out = GRAD ? static_cast<char*>(p.dz) + t * p.ld * B : nullptr;
        char* const obody = GRAD ? out + (cur.sh.body - (static_cast<const char*>(p.z) + t * p.ld * B)) : nullptr;
        auto value = [&](float z) {
            float g = ft * exp_of(z, st);
            if constexpr (BOTH) g = __builtin_fmaf(f1, exp_of(z, s1), g);
            return g;
        };
        auto put = [&](const P& u, int j) {
            if (tid + j * THREADS >= cur.sh.pieces) return;
            uint4 o = make_uint4(0, 0, 0, 0);
            if (cur.on) {
                float g[E];
#pragma unroll
                for (int i = 0; i < E; ++i) g[i] = value(u.at(i));
                o = pack_piece<F32>(g);
            }
            store_stream(obody + static_cast<int64_t>(j) * THREADS * 16 + mine, o);
        };
        if (GRAD && cur.edge >= 0) store_one<F32>(out, cur.edge, cur.on ? value(cur.ze) : 0.0f);
        if constexpr (NV > 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if constexpr (GRAD) put(v[j], j);
                __builtin_amdgcn_sched_barrier(0);  // a piece at a time: few registers besides the row's
                if constexpr (LOOP) v[j] = load_piece(nxt, j);
            }
        } else if constexpr (GRAD) {
            for (int j = 0; j * THREADS < cur.sh.pieces; ++j) put(load_piece(cur, j), j);
        }
        if constexpr (GRAD) {
            __syncthreads();  // the row's values before its entries'
            if (cur.on && cur.k >= 0) {
                float sum = 0.0f;
                for (int i = 0; i <= p.K; ++i) sum += s_k[i] == cur.k ? s_p[i] : 0.0f;
                store_one<F32>(out, cur.k, __builtin_fmaf(-w, sum, value(cur.zk)));
            }
        }
        if (!more) return;
        if constexpr (LOOP) {
            cur = nxt;
            t = tn;
        }
    }
}

template <bool F32, int THREADS, int NV, bool BOTH>
void launch_distill_as(const DistillArgs& a, hipStream_t stream) {
    // in turns: a workgroup a CU, each the same number of rows
    const int64_t rounds = distill_loops(THREADS, NV) ? ceil_div(a.T, 256) : 1;
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.T, rounds))), block(THREADS);
    if (a.dz != nullptr)
        hipLaunchKernelGGL((distill_kernel<F32, THREADS, NV, true, BOTH>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((distill_kernel<F32, THREADS, NV, false, BOTH>), grid, block, 0, stream, a);
}

// The fewest threads that hold the row and have one for every entry and the
// label. A wave alone meets no barrier: 8192 x 300 bf16, K = 32, 12.0 us, with
// four waves 27.9. Four to sixteen waves keep the row's registers under 128
// each, so that two workgroups and more share a CU (2048 x 32000: 8 waves 64.8
// us, 4 waves 63.3, 16 waves 86; 2000 x 65536: 8 waves 114, 16 waves 134; fp32
// 2000 x 32000: 108 and 115).
template <bool F32, bool BOTH>
void launch_distill_nv(const DistillArgs& a, hipStream_t stream) {
    const int64_t pieces = a.V / (F32 ? 4 : 8);
    if (pieces <= 64 && a.K < 64) launch_distill_as<F32, 64, 1, BOTH>(a, stream);
    else if (pieces <= 256 && a.K < 64) launch_distill_as<F32, 64, 4, BOTH>(a, stream);
    else if (pieces <= 256 && a.K < 256) launch_distill_as<F32, 256, 1, BOTH>(a, stream);
    else if (pieces <= 1024 && a.K < 256) launch_distill_as<F32, 256, 4, BOTH>(a, stream);
    else if (pieces <= 2048) launch_distill_as<F32, 512, 4, BOTH>(a, stream);
    else if (pieces <= 4096) launch_distill_as<F32, 512, 8, BOTH>(a, stream);
    else if (pieces <= 8192) launch_distill_as<F32, 512, 16, BOTH>(a, stream);
    else if (pieces <= 16384) launch_distill_as<F32, 1024, 16, BOTH>(a, stream);
    else launch_distill_as<F32, 1024, 0, BOTH>(a, stream);
}

}  // namespace

size_t logp_ws_bytes(int64_t T, int64_t V, bool f32) {
    return static_cast<size_t>(T) * logp_runs(V, f32) * 2 * sizeof(float);
}

int launch_logp(LogpArgs& a, hipStream_t stream) {
    a.runs = logp_runs(a.V, a.f32);
    timer_begin(QL_KERNEL_LOGP, stream);
    const dim3 grid(static_cast<uint32_t>(ceil_div(a.T, kLogpThreads / 64) * a.runs));
    if (a.f32)
        hipLaunchKernelGGL(logp_kernel<true>, grid, dim3(kLogpThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(logp_kernel<false>, grid, dim3(kLogpThreads), 0, stream, a);
    if (a.logp != nullptr)
        hipLaunchKernelGGL(logp_join_kernel, dim3(static_cast<uint32_t>(ceil_div(a.T, 256))), dim3(256), 0, stream, a);
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
