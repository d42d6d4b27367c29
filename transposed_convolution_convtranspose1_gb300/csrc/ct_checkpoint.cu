// ct_checkpoint.cu -- 8-bit activation checkpoints: a matrix kept as codes
// and group scales (the format of ct_rows.cuh), read back, and the (gated)
// activation that keeps its inputs so and differentiates from them.
//
//   forward    y = act(gate) * up   (up absent: y = act(gate)), gate and up kept
//   backward   dgate = dy * up^ * act'(gate^),  dup = dy * act(gate^)
// with gate^, up^ the values the codes stand for.  The gradient is that of
// the activation at the kept values: no second copy of the inputs exists.
#include <algorithm>

#include "ct_internal.h"
#include "ct_rows.cuh"

namespace ct {
namespace {

using namespace rows;

constexpr int kThreads = 256;

struct ActFwd {
    const void *gate, *up;
    void* y;
    uint8_t *gc, *uc;
    float *gsc, *usc;
    int64_t gs, us, ys;
    int64_t rows;
    int cols, group, n_groups;
    float alpha;
};

struct ActBwd {
    const void* dy;
    const uint8_t *gc, *uc;
    const float *gsc, *usc;
    void *dgate, *dup, *y;
    int64_t dys, dgs, dus, ys;
    int64_t rows;
    int cols, group, n_groups;
    float alpha;
};

// Codes and scale of one group held four values a lane.
template <int Q>
__device__ __forceinline__ void keep(const float (&v)[4], unsigned amax, int n, int lane, uint8_t* codes, float* scale_out) {
    amax = __reduce_max_sync(0xffffffffu, amax);
    float scale, inv;
    group_scale<Q>(amax, scale, inv);
    if (lane == 0) *scale_out = scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        if (k < n) codes[k] = encode<Q>(v[j], inv);
    }
}

// Simple form: a warp per group of a row; any size and alignment.
template <typename T, int Q, int A>
__global__ void __launch_bounds__(kThreads) act_fwd_groups(ActFwd P) {
    const int lane = threadIdx.x & 31;
    const int64_t n_work = P.rows * P.n_groups;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n_work;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t row = i / P.n_groups;
        const int c0 = (int)(i - row * P.n_groups) * P.group, n = min(P.group, P.cols - c0);
        const T* g = static_cast<const T*>(P.gate) + row * P.gs + c0;
        const T* u = P.up ? static_cast<const T*>(P.up) + row * P.us + c0 : nullptr;
        T* y = P.y ? static_cast<T*>(P.y) + row * P.ys + c0 : nullptr;
        float a[4], b[4];
        unsigned amax = 0, bmax = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = j * 32 + lane;
            a[j] = b[j] = 0.f;
            if (k < n) {
                a[j] = to_f32(g[k]);
                amax = max(amax, abs_bits(a[j]));
                if (u) {
                    b[j] = to_f32(u[k]);
                    bmax = max(bmax, abs_bits(b[j]));
                }
                if (y) {
                    const float v = act_fixed<A>(a[j], P.alpha);
                    y[k] = from_f32<T>(u ? v * b[j] : v);
                }
            }
        }
        keep<Q>(a, amax, n, lane, P.gc + row * P.cols + c0, P.gsc + i);
        if (u) keep<Q>(b, bmax, n, lane, P.uc + row * P.cols + c0, P.usc + i);
    }
}

// Simple form of the gradient, and of reading a checkpoint back (no dy).
template <typename T, int Q, int A>
__global__ void __launch_bounds__(kThreads) act_bwd_groups(ActBwd P) {
    const int lane = threadIdx.x & 31;
    const int64_t n_work = P.rows * P.n_groups;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n_work;
         i += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t row = i / P.n_groups;
        const int c0 = (int)(i - row * P.n_groups) * P.group, n = min(P.group, P.cols - c0);
        const uint8_t* gc = P.gc + row * P.cols + c0;
        const uint8_t* uc = P.uc ? P.uc + row * P.cols + c0 : nullptr;
        const float gsc = P.gsc[i], usc = uc ? P.usc[i] : 1.f;
        const T* dy = P.dy ? static_cast<const T*>(P.dy) + row * P.dys + c0 : nullptr;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = j * 32 + lane;
            if (k >= n) continue;
            const float a = decode<Q>(gc[k]) * gsc, b = uc ? decode<Q>(uc[k]) * usc : 1.f;
            const float f = act_fixed<A>(a, P.alpha);
            if (P.y) static_cast<T*>(P.y)[row * P.ys + c0 + k] = from_f32<T>(uc ? f * b : f);
            if (!dy) continue;
            const float d = to_f32(dy[k]);
            if (P.dgate) {
                const float t = d * act_slope<A>(a, P.alpha);
                static_cast<T*>(P.dgate)[row * P.dgs + c0 + k] = from_f32<T>(uc ? t * b : t);
            }
            if (P.dup) static_cast<T*>(P.dup)[row * P.dus + c0 + k] = from_f32<T>(d * f);
        }
    }
}

unsigned warps_grid(int64_t work) {
    return (unsigned)std::min<int64_t>((work + kThreads / 32 - 1) / (kThreads / 32), 1 << 20);
}

template <typename T, int Q>
cudaError_t launch_fwd(const ActFwd& P, int act, cudaStream_t s) {
    const unsigned grid = warps_grid(P.rows * P.n_groups);
    switch (act) {
#define CASE(A) case A: act_fwd_groups<T, Q, A><<<grid, kThreads, 0, s>>>(P); break
        CASE(1); CASE(2); CASE(3); CASE(4); CASE(5); CASE(6);
        default: act_fwd_groups<T, Q, 0><<<grid, kThreads, 0, s>>>(P);
#undef CASE
    }
    return cudaGetLastError();
}

template <typename T, int Q>
cudaError_t launch_bwd(const ActBwd& P, int act, cudaStream_t s) {
    const unsigned grid = warps_grid(P.rows * P.n_groups);
    switch (act) {
#define CASE(A) case A: act_bwd_groups<T, Q, A><<<grid, kThreads, 0, s>>>(P); break
        CASE(1); CASE(2); CASE(3); CASE(4); CASE(5); CASE(6);
        default: act_bwd_groups<T, Q, 0><<<grid, kThreads, 0, s>>>(P);
#undef CASE
    }
    return cudaGetLastError();
}

cudaError_t run_fwd(const ActFwd& P, int act, int dtype, int quant, cudaStream_t s) {
    const bool i8 = quant == CT_Q_INT8;
    switch (dtype) {
        case CT_F32: return i8 ? launch_fwd<float, CT_Q_INT8>(P, act, s) : launch_fwd<float, CT_Q_E4M3>(P, act, s);
        case CT_F16: return i8 ? launch_fwd<__half, CT_Q_INT8>(P, act, s) : launch_fwd<__half, CT_Q_E4M3>(P, act, s);
        default: return i8 ? launch_fwd<__nv_bfloat16, CT_Q_INT8>(P, act, s) : launch_fwd<__nv_bfloat16, CT_Q_E4M3>(P, act, s);
    }
}

cudaError_t run_bwd(const ActBwd& P, int act, int dtype, int quant, cudaStream_t s) {
    const bool i8 = quant == CT_Q_INT8;
    switch (dtype) {
        case CT_F32: return i8 ? launch_bwd<float, CT_Q_INT8>(P, act, s) : launch_bwd<float, CT_Q_E4M3>(P, act, s);
        case CT_F16: return i8 ? launch_bwd<__half, CT_Q_INT8>(P, act, s) : launch_bwd<__half, CT_Q_E4M3>(P, act, s);
        default: return i8 ? launch_bwd<__nv_bfloat16, CT_Q_INT8>(P, act, s) : launch_bwd<__nv_bfloat16, CT_Q_E4M3>(P, act, s);
    }
}

bool bad_ptr(const void* p, size_t a) { return p && (uintptr_t)p % a != 0; }

int check(int64_t rows, int64_t cols, int activation, int dtype, int quant, int group) {
    if (dtype != CT_F32 && dtype != CT_F16 && dtype != CT_BF16)
        return report_error(CT_ERR_DTYPE, "dtype %d is not a supported floating type (CT_F32, CT_F16, CT_BF16)", dtype);
    if (rows < 0 || cols < 0)
        return report_error(CT_ERR_SHAPE, "rows and cols must be >= 0 (got %lld, %lld)", (long long)rows, (long long)cols);
    if (cols > (1ll << 30) || rows > (1ll << 40) || (double)rows * (double)cols > 4e18)
        return report_error(CT_ERR_TOO_LARGE, "cols <= 2^30, rows <= 2^40 and rows * cols <= 4e18 supported");
    if (quant != CT_Q_INT8 && quant != CT_Q_E4M3) return report_error(CT_ERR_PARAM, "quant must be CT_Q_INT8 or CT_Q_E4M3 (got %d)", quant);
    if (group != 32 && group != 64 && group != 128) return report_error(CT_ERR_PARAM, "group must be 32, 64 or 128 (got %d)", group);
    if (activation < CT_ACT_NONE || activation > CT_ACT_SIGMOID)
        return report_error(CT_ERR_PARAM, "activation %d is not a ct_activation", activation);
    return CT_OK;
}

int done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? CT_OK : report_error(CT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace ct

using namespace ct;

extern "C" int ct_checkpointed_activation_forward(const void* gate, int64_t gate_stride, const void* up,
                                                  int64_t up_stride, void* y, int64_t y_stride, void* gate_codes,
                                                  float* gate_scales, void* up_codes, float* up_scales, int64_t rows,
                                                  int64_t cols, int activation, float alpha, int dtype, int quant,
                                                  int group, void* stream) {
    int rc = check(rows, cols, activation, dtype, quant, group);
    if (rc != CT_OK) return rc;
    if (rows == 0 || cols == 0) return CT_OK;
    if (!gate || !gate_codes || !gate_scales || (up && (!up_codes || !up_scales)))
        return report_error(CT_ERR_NULL, "gate and the codes and scales of each input must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(gate, eb) || bad_ptr(up, eb) || bad_ptr(y, eb) || bad_ptr(gate_scales, 4) || bad_ptr(up_scales, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    ActFwd P{gate, up, y, static_cast<uint8_t*>(gate_codes), static_cast<uint8_t*>(up_codes), gate_scales, up_scales,
             gate_stride, up_stride, y_stride, rows, (int)cols, group, (int)((cols + group - 1) / group), alpha};
    return done(run_fwd(P, activation, dtype, quant, (cudaStream_t)stream), "checkpointed activation");
}

extern "C" int ct_checkpointed_activation_backward(const void* dy, int64_t dy_stride, const void* gate_codes,
                                                   const float* gate_scales, const void* up_codes,
                                                   const float* up_scales, void* dgate, int64_t dgate_stride, void* dup,
                                                   int64_t dup_stride, void* y, int64_t y_stride, int64_t rows,
                                                   int64_t cols, int activation, float alpha, int dtype, int quant,
                                                   int group, void* stream) {
    int rc = check(rows, cols, activation, dtype, quant, group);
    if (rc != CT_OK) return rc;
    if (rows == 0 || cols == 0) return CT_OK;
    if (!gate_codes || !gate_scales || (up_codes && !up_scales) || (dup && !up_codes) || ((dgate || dup) && !dy))
        return report_error(CT_ERR_NULL, "codes and scales of each input, dy for a gradient and up for dup must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(dy, eb) || bad_ptr(dgate, eb) || bad_ptr(dup, eb) || bad_ptr(y, eb) || bad_ptr(gate_scales, 4) || bad_ptr(up_scales, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    if (!dgate && !dup && !y) return CT_OK;
    ActBwd P{dgate || dup ? dy : nullptr, static_cast<const uint8_t*>(gate_codes), static_cast<const uint8_t*>(up_codes),
             gate_scales, up_scales, dgate, dup, y, dy_stride, dgate_stride, dup_stride, y_stride, rows, (int)cols, group,
             (int)((cols + group - 1) / group), alpha};
    return done(run_bwd(P, activation, dtype, quant, (cudaStream_t)stream), "checkpointed activation backward");
}

extern "C" int ct_checkpoint_store(const void* x, int64_t x_stride, void* codes, float* scales, int64_t rows,
                                   int64_t cols, int dtype, int quant, int group, void* stream) {
    return ct_checkpointed_activation_forward(x, x_stride, nullptr, 0, nullptr, 0, codes, scales, nullptr, nullptr, rows,
                                              cols, CT_ACT_NONE, 0.f, dtype, quant, group, stream);
}

extern "C" int ct_checkpoint_load(const void* codes, const float* scales, void* y, int64_t y_stride, int64_t rows,
                                  int64_t cols, int dtype, int quant, int group, void* stream) {
    if (rows > 0 && cols > 0 && !y) return report_error(CT_ERR_NULL, "y must not be NULL");
    return ct_checkpointed_activation_backward(nullptr, 0, codes, scales, nullptr, nullptr, nullptr, 0, nullptr, 0, y,
                                               y_stride, rows, cols, CT_ACT_NONE, 0.f, dtype, quant, group, stream);
}
