// C ABI of the operators around the linear layer in a training step: norms, the
// backward of its epilogue, and the losses on logits. Validation before any launch, as in api.cpp. No C++
// exception crosses this file's extern "C" functions.
#include <hip/hip_runtime.h>

#include <cmath>

#include "common.h"
#include "internal.h"
#include "qlora_nf4.h"

namespace qlnf4 {
namespace {

int check_dtype(int dtype, const char* name) {
    if (dtype != QL_F32 && dtype != QL_BF16) return set_error(QL_ERR_UNSUPPORTED, "%s dtype %d", name, dtype);
    return QL_OK;
}

int check_flag(int v, const char* name) {
    if (v != 0 && v != 1) return set_error(QL_ERR_UNSUPPORTED, "%s = %d", name, v);
    return QL_OK;
}

// Device arrays of 4- or 8-byte values that are read one by one.
int check_array(const void* p, const char* name, unsigned bytes) {
    if (p == nullptr) return set_error(QL_ERR_NULL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return set_error(QL_ERR_ALIGN, "%s is not %u-byte aligned", name, bytes);
    return QL_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
    if (need == 0) return QL_OK;
    if (ws == nullptr || have < need)
        return set_error(QL_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws == nullptr ? 0 : have, need);
    if (!aligned16(ws)) return set_error(QL_ERR_ALIGN, "workspace is not 16-byte aligned");
    return QL_OK;
}

int check_norm(int64_t rows, int64_t cols, int x_dtype, int w_dtype) {
    // one row a workgroup of up to 1024 threads, fewer than 2^32 threads a launch
    if (rows < 0 || rows >= (int64_t{1} << 22)) return set_error(QL_ERR_SHAPE, "rows = %lld", (long long)rows);
    if (cols <= 0 || cols % 8 != 0 || cols > QL_NORM_MAX_COLS)
        return set_error(QL_ERR_SHAPE, "cols = %lld (a multiple of 8, at most %d)", (long long)cols, QL_NORM_MAX_COLS);
    int s;
    if ((s = check_dtype(x_dtype, "activation")) != QL_OK) return s;
    return check_dtype(w_dtype, "weight");
}

int check_epilogue_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || rows > (int64_t{1} << 31)) return set_error(QL_ERR_SHAPE, "rows = %lld", (long long)rows);
    // 1024 threads per 32 column sums, fewer than 2^32 threads a launch
    if (cols <= 0 || cols % 8 != 0 || cols >= (int64_t{1} << 27))
        return set_error(QL_ERR_SHAPE, "cols = %lld (a multiple of 8 under 2^27)", (long long)cols);
    if (rows > 0 && cols > (int64_t{1} << 40) / rows)
        return set_error(QL_ERR_SHAPE, "%lld x %lld", (long long)rows, (long long)cols);
    return QL_OK;
}

int check_logits_shape(int64_t T, int64_t V, int64_t ld, int dtype) {
    int s;
    if ((s = check_dtype(dtype, "logits")) != QL_OK) return s;
    // workgroups: a row's slices are at most one and one per 4096 values
    if (T < 0 || T > (int64_t{1} << 22)) return set_error(QL_ERR_SHAPE, "T = %lld", (long long)T);
    if (V <= 0 || V >= (int64_t{1} << 30)) return set_error(QL_ERR_SHAPE, "V = %lld", (long long)V);
    if (T * V > (int64_t{1} << 35)) return set_error(QL_ERR_SHAPE, "%lld x %lld logits", (long long)T, (long long)V);
    if (ld < V || ld > (int64_t{1} << 34)) return set_error(QL_ERR_SHAPE, "row stride %lld, V = %lld", (long long)ld, (long long)V);
    return QL_OK;
}

int check_logits(const void* z, int dtype) { return check_array(z, "logits", dtype == QL_F32 ? 4 : 2); }

int check_dlogits(const void* dz, const void* z, int dtype) {
    int s;
    if ((s = check_array(dz, "dlogits", dtype == QL_F32 ? 4 : 2)) != QL_OK) return s;
    if ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15u)
        return set_error(QL_ERR_ALIGN, "dlogits and logits lie differently in their 16-byte lines");
    return QL_OK;
}

}  // namespace
}  // namespace qlnf4

using namespace qlnf4;

extern "C" {

int qlora_norm_fwd(const void* X, int x_dtype, int64_t rows, int64_t cols, const void* weight, const void* bias,
                   int w_dtype, float eps, int rms, void* Y, float* mean, float* rstd, void* stream) {
    clear_error();
    int s;
    if ((s = check_norm(rows, cols, x_dtype, w_dtype)) != QL_OK) return s;
    if (!(eps >= 0.0f) || std::isinf(eps)) return set_error(QL_ERR_UNSUPPORTED, "eps = %g", (double)eps);
    if ((s = check_flag(rms, "rms")) != QL_OK) return s;
    if (rows == 0) return QL_OK;
    if ((s = check_ptr(X, "X")) != QL_OK) return s;
    if ((s = check_ptr(weight, "weight")) != QL_OK) return s;
    if (bias != nullptr && (s = check_ptr(bias, "bias")) != QL_OK) return s;
    if ((s = check_ptr(Y, "Y")) != QL_OK) return s;
    if (mean != nullptr && (s = check_array(mean, "mean", 4)) != QL_OK) return s;
    if (rstd != nullptr && (s = check_array(rstd, "rstd", 4)) != QL_OK) return s;
    NormArgs a{};
    a.X = X;
    a.T = rows;
    a.C = static_cast<int>(cols);
    a.w = weight;
    a.b = bias;
    a.x_f32 = x_dtype == QL_F32;
    a.w_f32 = w_dtype == QL_F32;
    a.rms = rms;
    a.eps = eps;
    a.Y = Y;
    a.mean = mean;
    a.rstd = rstd;
    return launch_norm_fwd(a, static_cast<hipStream_t>(stream));
}

size_t qlora_norm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || rows >= (int64_t{1} << 22) || cols <= 0 || cols > QL_NORM_MAX_COLS) return 0;
    return norm_bwd_ws_bytes(rows, cols);
}

int qlora_norm_bwd(const void* X, int x_dtype, int64_t rows, int64_t cols, const void* weight, int w_dtype,
                   const void* dY, const float* mean, const float* rstd, void* dX, float* dweight, float* dbias,
                   int accumulate, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int s;
    if ((s = check_norm(rows, cols, x_dtype, w_dtype)) != QL_OK) return s;
    if ((s = check_flag(accumulate, "accumulate")) != QL_OK) return s;
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (!sums && (dX == nullptr || rows == 0)) return QL_OK;
    if (dweight != nullptr && (s = check_ptr(dweight, "dweight")) != QL_OK) return s;
    if (dbias != nullptr && (s = check_ptr(dbias, "dbias")) != QL_OK) return s;
    if (rows > 0) {
        if ((s = check_ptr(X, "X")) != QL_OK) return s;
        if ((s = check_ptr(weight, "weight")) != QL_OK) return s;
        if ((s = check_ptr(dY, "dY")) != QL_OK) return s;
        if (mean != nullptr && (s = check_array(mean, "mean", 4)) != QL_OK) return s;
        if ((s = check_array(rstd, "rstd", 4)) != QL_OK) return s;
        if (dX != nullptr && (s = check_ptr(dX, "dX")) != QL_OK) return s;
        if (sums && (s = check_ws(ws, ws_bytes, norm_bwd_ws_bytes(rows, cols))) != QL_OK) return s;
    }
    NormArgs a{};
    a.X = X;
    a.T = rows;
    a.C = static_cast<int>(cols);
    a.w = weight;
    a.x_f32 = x_dtype == QL_F32;
    a.w_f32 = w_dtype == QL_F32;
    a.rms = mean == nullptr;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dY = dY;
    a.dX = dX;
    a.dW = dweight;
    a.dB = dbias;
    a.accumulate = accumulate;
    a.part = static_cast<float*>(ws);
    return launch_norm_bwd(a, static_cast<hipStream_t>(stream));
}

size_t qlora_epilogue_bwd_workspace(int64_t rows, int64_t cols) {
    if (check_epilogue_shape(rows, cols) != QL_OK) return 0;
    return epilogue_bwd_ws_bytes(rows, cols);
}

int qlora_epilogue_bwd(const uint16_t* dY, const void* Z, int z_dtype, int64_t rows, int64_t cols, int act, uint16_t* dZ,
                       float* dbias, int accumulate, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int s;
    if ((s = check_epilogue_shape(rows, cols)) != QL_OK) return s;
    if (act < QL_ACT_NONE || act > QL_ACT_GELU_TANH) return set_error(QL_ERR_UNSUPPORTED, "activation %d", act);
    if ((s = check_dtype(z_dtype, "Z")) != QL_OK) return s;
    if ((s = check_flag(accumulate, "accumulate")) != QL_OK) return s;
    if (dbias == nullptr && (dZ == nullptr || rows == 0)) return QL_OK;
    if (dbias != nullptr && (s = check_ptr(dbias, "dbias")) != QL_OK) return s;
    if (rows > 0) {
        if ((s = check_ptr(dY, "dY")) != QL_OK) return s;
        if (act != QL_ACT_NONE && (s = check_ptr(Z, "Z")) != QL_OK) return s;
        if (dZ != nullptr && (s = check_ptr(dZ, "dZ")) != QL_OK) return s;
        if (dbias != nullptr && (s = check_ws(ws, ws_bytes, epilogue_bwd_ws_bytes(rows, cols))) != QL_OK) return s;
    }
    EpilogueBwdArgs a{};
    a.dY = dY;
    a.Z = Z;
    a.z_f32 = z_dtype == QL_F32;
    a.T = rows;
    a.N = cols;
    a.act = act;
    a.dZ = dZ;
    a.dB = dbias;
    a.accumulate = accumulate;
    a.part = static_cast<float*>(ws);
    return launch_epilogue_bwd(a, static_cast<hipStream_t>(stream));
}

size_t qlora_token_logp_workspace(int64_t T, int64_t V, int dtype) {
    if (check_logits_shape(T, V, V, dtype) != QL_OK || T == 0) return 0;
    return logp_ws_bytes(T, V, dtype == QL_F32);
}

int qlora_token_logp(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const int64_t* labels,
                     float* logp, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int s;
    if ((s = check_logits_shape(T, V, ld, dtype)) != QL_OK) return s;
    if (T == 0) return QL_OK;
    if ((s = check_logits(logits, dtype)) != QL_OK) return s;
    if ((s = check_array(labels, "labels", 8)) != QL_OK) return s;
    if ((s = check_array(logp, "logp", 4)) != QL_OK) return s;
    if ((s = check_ws(ws, ws_bytes, logp_ws_bytes(T, V, dtype == QL_F32))) != QL_OK) return s;
    LogpArgs a{};
    a.z = logits;
    a.f32 = dtype == QL_F32;
    a.T = T;
    a.ld = ld;
    a.V = static_cast<int>(V);
    a.labels = labels;
    a.logp = logp;
    a.part = static_cast<float*>(ws);
    return launch_logp(a, static_cast<hipStream_t>(stream));
}

int qlora_preference_loss_fwd(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const int64_t* labels,
                              const int64_t* seq_start, int64_t pairs, const float* ref_logp, float beta,
                              float label_smoothing, int kind, int average, float* loss, float* seq_logp, float* state,
                              void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    int s;
    if ((s = check_logits_shape(T, V, ld, dtype)) != QL_OK) return s;
    if (pairs < 0 || pairs > (int64_t{1} << 21)) return set_error(QL_ERR_SHAPE, "pairs = %lld", (long long)pairs);
    if (!(beta > 0.0f) || std::isinf(beta)) return set_error(QL_ERR_UNSUPPORTED, "beta = %g", (double)beta);
    if (!(label_smoothing >= 0.0f && label_smoothing <= 1.0f))
        return set_error(QL_ERR_UNSUPPORTED, "label_smoothing = %g", (double)label_smoothing);
    if (kind != QL_PREF_SIGMOID && kind != QL_PREF_HINGE && kind != QL_PREF_SQUARED)
        return set_error(QL_ERR_UNSUPPORTED, "kind = %d", kind);
    if (kind != QL_PREF_SIGMOID && label_smoothing != 0.0f)
        return set_error(QL_ERR_UNSUPPORTED, "label_smoothing = %g with kind %d", (double)label_smoothing, kind);
    if ((s = check_flag(average, "average")) != QL_OK) return s;
    if (T > 0) {
        if ((s = check_logits(logits, dtype)) != QL_OK) return s;
        if ((s = check_array(labels, "labels", 8)) != QL_OK) return s;
        if ((s = check_array(state, "state", 4)) != QL_OK) return s;
        if ((s = check_ws(ws, ws_bytes, logp_ws_bytes(T, V, dtype == QL_F32))) != QL_OK) return s;
    }
    if (pairs > 0) {
        if ((s = check_array(seq_start, "seq_start", 8)) != QL_OK) return s;
        if ((s = check_array(ref_logp, "ref_logp", 4)) != QL_OK) return s;
        if ((s = check_array(loss, "loss", 4)) != QL_OK) return s;
        if ((s = check_array(seq_logp, "seq_logp", 4)) != QL_OK) return s;
    }
    float* const dlogp = state + 2 * T;
    int* const pair = reinterpret_cast<int*>(state + 3 * T);
    float* const logp = state + 4 * T;
    static_assert(QL_PREF_STATE_ROWS == 5, "references, sums, slopes, pairs, log probabilities");
    LogpArgs a{};
    a.z = logits;
    a.f32 = dtype == QL_F32;
    a.T = T;
    a.ld = ld;
    a.V = static_cast<int>(V);
    a.labels = labels;
    a.dlogp = dlogp;
    a.pair = pair;
    a.pair_logp = logp;
    a.part = static_cast<float*>(ws);
    if (T > 0 && (s = launch_logp(a, static_cast<hipStream_t>(stream))) != QL_OK) return s;
    if (pairs == 0) return QL_OK;
    PairArgs q{};
    q.z = logits;
    q.f32 = a.f32;
    q.T = T;
    q.ld = ld;
    q.V = a.V;
    q.labels = labels;
    q.part = a.part;
    q.runs = a.runs;
    q.start = seq_start;
    q.ref_logp = ref_logp;
    q.beta = beta;
    q.smooth = label_smoothing;
    q.kind = kind;
    q.average = average;
    q.loss = loss;
    q.seq_logp = seq_logp;
    q.logp = logp;
    q.ref = state;
    q.inv = state + T;
    q.dlogp = dlogp;
    q.pair = pair;
    return launch_pairs(q, static_cast<int>(pairs), static_cast<hipStream_t>(stream));
}

int qlora_preference_loss_bwd(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const int64_t* labels,
                              const float* state, const float* dloss, int64_t pairs, void* dlogits, void* stream) {
    clear_error();
    int s;
    if ((s = check_logits_shape(T, V, ld, dtype)) != QL_OK) return s;
    if (pairs < 0 || pairs > (int64_t{1} << 21)) return set_error(QL_ERR_SHAPE, "pairs = %lld", (long long)pairs);
    if (T == 0) return QL_OK;
    if ((s = check_logits(logits, dtype)) != QL_OK) return s;
    if ((s = check_array(labels, "labels", 8)) != QL_OK) return s;
    if ((s = check_array(state, "state", 4)) != QL_OK) return s;
    if (pairs > 0 && (s = check_array(dloss, "dloss", 4)) != QL_OK) return s;
    if ((s = check_dlogits(dlogits, logits, dtype)) != QL_OK) return s;
    LogpGradArgs a{};
    a.z = logits;
    a.dz = dlogits;
    a.f32 = dtype == QL_F32;
    a.T = T;
    a.ld = ld;
    a.V = static_cast<int>(V);
    a.labels = labels;
    a.ref = state;
    a.inv = state + T;
    a.dlogp = state + 2 * T;
    a.pair = reinterpret_cast<const int*>(state + 3 * T);
    a.dloss = dloss;
    a.pairs = pairs;
    return launch_logp_grad(a, static_cast<hipStream_t>(stream));
}

int qlora_distill_loss(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const int64_t* top_index,
                       const void* top_logits, int top_dtype, int64_t K, const int64_t* labels, float tau, float a,
                       const float* weight, float* loss, void* dlogits, void* stream) {
    clear_error();
    int s;
    if ((s = check_logits_shape(T, V, ld, dtype)) != QL_OK) return s;
    if ((s = check_dtype(top_dtype, "top_logits")) != QL_OK) return s;
    if (K < 1 || K > QL_DISTILL_MAX_TOP)
        return set_error(QL_ERR_SHAPE, "K = %lld outside [1, %d]", (long long)K, QL_DISTILL_MAX_TOP);
    if (!(tau >= 0x1p-20f && tau <= 0x1p20f)) return set_error(QL_ERR_UNSUPPORTED, "tau = %g outside [2^-20, 2^20]", (double)tau);
    if (!(a >= 0.0f && a <= 1.0f)) return set_error(QL_ERR_UNSUPPORTED, "a = %g outside [0, 1]", (double)a);
    if (T == 0 || (loss == nullptr && dlogits == nullptr)) return QL_OK;
    if ((s = check_logits(logits, dtype)) != QL_OK) return s;
    if ((s = check_array(top_index, "top_index", 8)) != QL_OK) return s;
    if ((s = check_array(top_logits, "top_logits", top_dtype == QL_F32 ? 4 : 2)) != QL_OK) return s;
    if ((labels != nullptr || a > 0.0f) && (s = check_array(labels, "labels", 8)) != QL_OK) return s;
    if (weight != nullptr && (s = check_array(weight, "weight", 4)) != QL_OK) return s;
    if (loss != nullptr && (s = check_array(loss, "loss", 4)) != QL_OK) return s;
    if (dlogits != nullptr && (s = check_dlogits(dlogits, logits, dtype)) != QL_OK) return s;
    DistillArgs d{};
    d.z = logits;
    d.dz = dlogits;
    d.f32 = dtype == QL_F32;
    d.T = T;
    d.ld = ld;
    d.V = static_cast<int>(V);
    d.K = static_cast<int>(K);
    d.index = top_index;
    d.top = top_logits;
    d.top_f32 = top_dtype == QL_F32;
    d.labels = labels;
    d.weight = weight;
    d.tau = tau;
    d.alpha = a;
    d.loss = loss;
    return launch_distill(d, static_cast<hipStream_t>(stream));
}

}  // extern "C"
