// ct_norm.cu -- root-mean-square norm of the rows of a matrix, with the
// residual's addition before it and an 8-bit output, and its gradient.
//
//   s = x + residual             (fp32, not rounded before the norm)
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y = s * rstd * weight        (also or instead in 8 bits, see ct_rows.cuh)
//   h = s rounded once to the element type: the residual stream's new value
//
// Gradient, with u = h * rstd:
//   c  = mean(weight * dy * u)
//   dx = rstd * (weight * dy - u * c) + dresidual     (also the residual's)
//   dw = sum over rows of dy * u
#include <algorithm>

#include "ct_internal.h"
#include "ct_rows.cuh"

namespace ct {
namespace {

using namespace rows;

constexpr int kThreads = 256;

struct NormFwd {
    const void *x, *res, *w;
    void *y, *h;
    float* rstd;
    uint8_t* codes;
    float* scales;
    int64_t xs, rs, ys, hs;  // row strides, elements
    int64_t rows;
    int cols, group, quant;
    float eps;
};

struct NormBwd {
    const void *dy, *h, *w, *dres;
    const float* rstd;
    void *dx, *dw;
    float* part;  // [blocks][cols] partial sums of dw
    int64_t dys, hs, drs, dxs;
    int64_t rows;
    int cols, blocks;
};

template <typename T>
__device__ __forceinline__ float sum_at(const T* x, const T* r, int i) {
    return r ? to_f32(x[i]) + to_f32(r[i]) : to_f32(x[i]);
}

// Simple form: a block per row, two passes over it; any size and alignment.
template <typename T, int Q>
__global__ void __launch_bounds__(kThreads) norm_fwd_rows(NormFwd A) {
    __shared__ float part[32];
    const T* w = static_cast<const T*>(A.w);
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(A.x) + row * A.xs;
        const T* r = A.res ? static_cast<const T*>(A.res) + row * A.rs : nullptr;
        float ss = 0.f;
        for (int i = threadIdx.x; i < A.cols; i += kThreads) {
            const float s = sum_at(x, r, i);
            ss = fmaf(s, s, ss);
        }
        ss = block_sum<kThreads>(ss, part);
        const float rstd = 1.f / sqrtf(ss / (float)A.cols + A.eps);
        if (threadIdx.x == 0 && A.rstd) A.rstd[row] = rstd;
        T* y = A.y ? static_cast<T*>(A.y) + row * A.ys : nullptr;
        T* h = A.h ? static_cast<T*>(A.h) + row * A.hs : nullptr;
        const int lane = threadIdx.x & 31;
        const int n_groups = (A.cols + A.group - 1) / A.group;
        for (int g = threadIdx.x >> 5; g < n_groups; g += kThreads / 32) {
            float v[4];
            unsigned amax = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = j * 32 + lane, i = g * A.group + k;
                v[j] = 0.f;
                if (k < A.group && i < A.cols) {
                    const float s = sum_at(x, r, i);
                    v[j] = s * rstd * (w ? to_f32(w[i]) : 1.f);
                    if (h) h[i] = from_f32<T>(s);
                    if (y) y[i] = from_f32<T>(v[j]);
                    amax = max(amax, abs_bits(v[j]));
                }
            }
            if constexpr (Q != CT_Q_NONE) {
                amax = __reduce_max_sync(0xffffffffu, amax);
                float scale, inv;
                group_scale<Q>(amax, scale, inv);
                if (lane == 0) A.scales[row * n_groups + g] = scale;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = j * 32 + lane, i = g * A.group + k;
                    if (k < A.group && i < A.cols) A.codes[row * A.cols + i] = encode<Q>(v[j], inv);
                }
            }
        }
    }
}

// Simple form: a block takes a contiguous run of rows and keeps its share of
// dw in its own row of the workspace.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_rows(NormBwd A) {
    __shared__ float part[32];
    const T* w = static_cast<const T*>(A.w);
    const int64_t r0 = A.rows * blockIdx.x / A.blocks, r1 = A.rows * (blockIdx.x + 1) / A.blocks;
    float* mine = A.part + (int64_t)blockIdx.x * A.cols;
    if (A.dw)
        for (int i = threadIdx.x; i < A.cols; i += kThreads) mine[i] = 0.f;
    for (int64_t row = r0; row < r1; ++row) {
        const T* dy = static_cast<const T*>(A.dy) + row * A.dys;
        const T* h = static_cast<const T*>(A.h) + row * A.hs;
        const T* dres = A.dres ? static_cast<const T*>(A.dres) + row * A.drs : nullptr;
        const float rstd = A.rstd[row];
        float c = 0.f;
        for (int i = threadIdx.x; i < A.cols; i += kThreads) {
            const float u = to_f32(h[i]) * rstd, d = to_f32(dy[i]);
            c = fmaf(d * (w ? to_f32(w[i]) : 1.f), u, c);
            if (A.dw) mine[i] = fmaf(d, u, mine[i]);
        }
        c = block_sum<kThreads>(c, part) / (float)A.cols;
        if (A.dx) {
            T* dx = static_cast<T*>(A.dx) + row * A.dxs;
            for (int i = threadIdx.x; i < A.cols; i += kThreads) {
                const float u = to_f32(h[i]) * rstd, d = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.f);
                dx[i] = from_f32<T>(rstd * (d - u * c) + (dres ? to_f32(dres[i]) : 0.f));
            }
        }
    }
}

// dw: the blocks' partial sums added in their order, a warp's lanes on 32
// neighbouring columns.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dw_sum(const float* part, T* dw, int cols, int blocks) {
    __shared__ float s[kThreads / 32][32];
    const int i = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float v = 0.f;
    if (i < cols)
        for (int b = w; b < blocks; b += kThreads / 32) v += part[(int64_t)b * cols + i];
    s[w][threadIdx.x & 31] = v;
    __syncthreads();
    if (w == 0 && i < cols) {
#pragma unroll
        for (int k = 1; k < kThreads / 32; ++k) v += s[k][threadIdx.x & 31];
        dw[i] = from_f32<T>(v);
    }
}

int bwd_blocks(int64_t rows, int sm_count) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)sm_count * 4));
}

template <typename T>
cudaError_t launch_fwd(const NormFwd& A, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>(A.rows, 1 << 20);
    if (A.quant == CT_Q_INT8) norm_fwd_rows<T, CT_Q_INT8><<<grid, kThreads, 0, s>>>(A);
    else if (A.quant == CT_Q_E4M3) norm_fwd_rows<T, CT_Q_E4M3><<<grid, kThreads, 0, s>>>(A);
    else norm_fwd_rows<T, CT_Q_NONE><<<grid, kThreads, 0, s>>>(A);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const NormBwd& A, cudaStream_t s) {
    if (A.rows > 0) {
        norm_bwd_rows<T><<<A.blocks, kThreads, 0, s>>>(A);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (A.dw) norm_dw_sum<T><<<(A.cols + 31) / 32, kThreads, 0, s>>>(A.part, static_cast<T*>(A.dw), A.cols,
                                                                   A.rows > 0 ? A.blocks : 0);
    return cudaGetLastError();
}

bool bad_ptr(const void* p, size_t a) { return p && (uintptr_t)p % a != 0; }

int check_matrix(int64_t rows, int64_t cols, int dtype) {
    if (dtype != CT_F32 && dtype != CT_F16 && dtype != CT_BF16)
        return report_error(CT_ERR_DTYPE, "dtype %d is not a supported floating type (CT_F32, CT_F16, CT_BF16)", dtype);
    if (rows < 0 || cols < 1) return report_error(CT_ERR_SHAPE, "rows must be >= 0 and cols >= 1 (got %lld, %lld)",
                                                  (long long)rows, (long long)cols);
    if (cols > (1 << 24) || rows > (1ll << 40)) return report_error(CT_ERR_TOO_LARGE, "cols <= 2^24 and rows <= 2^40 supported");
    return CT_OK;
}

}  // namespace
}  // namespace ct

using namespace ct;

extern "C" int ct_rms_norm_forward(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                   const void* weight, void* y, int64_t y_stride, void* h, int64_t h_stride,
                                   float* rstd, void* codes, float* scales, int64_t rows, int64_t cols, float eps,
                                   int dtype, int quant, int group, void* stream) {
    int rc = check_matrix(rows, cols, dtype);
    if (rc != CT_OK) return rc;
    if (quant != CT_Q_NONE && quant != CT_Q_INT8 && quant != CT_Q_E4M3)
        return report_error(CT_ERR_PARAM, "quant %d is not a ct_quant", quant);
    if (quant != CT_Q_NONE && group != 32 && group != 64 && group != 128)
        return report_error(CT_ERR_PARAM, "group must be 32, 64 or 128 (got %d)", group);
    if (!(eps >= 0.f)) return report_error(CT_ERR_PARAM, "eps must be >= 0");
    if (rows == 0) return CT_OK;
    if (!x || (quant != CT_Q_NONE && (!codes || !scales)))
        return report_error(CT_ERR_NULL, "x (and codes and scales with an 8-bit output) must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(x, eb) || bad_ptr(residual, eb) || bad_ptr(weight, eb) || bad_ptr(y, eb) || bad_ptr(h, eb) ||
        bad_ptr(rstd, 4) || bad_ptr(scales, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    NormFwd A{x, residual, weight, y, h, rstd, static_cast<uint8_t*>(codes), scales, x_stride, residual_stride,
              y_stride, h_stride, rows, (int)cols, quant != CT_Q_NONE ? group : 128, quant, eps};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = dtype == CT_F32 ? launch_fwd<float>(A, s) : dtype == CT_F16 ? launch_fwd<__half>(A, s)
                                                                              : launch_fwd<__nv_bfloat16>(A, s);
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "rms norm: %s", cudaGetErrorString(e));
    return CT_OK;
}

extern "C" int ct_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols, int dtype, size_t* bytes) {
    if (!bytes) return report_error(CT_ERR_NULL, "bytes is NULL");
    int rc = check_matrix(rows, cols, dtype);
    if (rc != CT_OK) return rc;
    DeviceInfo d;
    int sm = 152;
    if (device_info(&d) == cudaSuccess) sm = d.sm_count;
    *bytes = (size_t)bwd_blocks(rows, sm) * cols * sizeof(float);
    return CT_OK;
}

extern "C" int ct_rms_norm_backward(const void* dy, int64_t dy_stride, const void* h, int64_t h_stride,
                                    const float* rstd, const void* weight, const void* dresidual,
                                    int64_t dresidual_stride, void* dx, int64_t dx_stride, void* dw, void* workspace,
                                    size_t workspace_bytes, int64_t rows, int64_t cols, int dtype, void* stream) {
    size_t need = 0;
    int rc = ct_rms_norm_backward_workspace_bytes(rows, cols, dtype, &need);
    if (rc != CT_OK) return rc;
    if (!dw) need = 0;
    if (rows > 0 && (dx || dw) && (!dy || !h || !rstd)) return report_error(CT_ERR_NULL, "dy, h and rstd must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(dy, eb) || bad_ptr(h, eb) || bad_ptr(weight, eb) || bad_ptr(dresidual, eb) || bad_ptr(dx, eb) ||
        bad_ptr(dw, eb) || bad_ptr(rstd, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    if (!dx && !dw) return CT_OK;
    if (rows == 0 && !dw) return CT_OK;
    DeviceInfo d;
    cudaError_t e = device_info(&d);
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "rms norm backward: %s", cudaGetErrorString(e));
    cudaStream_t s = (cudaStream_t)stream;
    void* ws = workspace;
    bool owned = false;
    if (need > 0) {
        if (ws) {
            if (workspace_bytes < need)
                return report_error(CT_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes, need);
            if (bad_ptr(ws, 256)) return report_error(CT_ERR_ALIGN, "workspace must be 256-byte aligned");
        } else {
            e = cudaMallocAsync(&ws, need, s);
            if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "cudaMallocAsync(workspace): %s", cudaGetErrorString(e));
            owned = true;
        }
    }
    NormBwd A{dy, h, weight, dresidual, rstd, dx, dw, static_cast<float*>(ws), dy_stride, h_stride, dresidual_stride,
              dx_stride, rows, (int)cols, bwd_blocks(rows, d.sm_count)};
    e = dtype == CT_F32 ? launch_bwd<float>(A, s) : dtype == CT_F16 ? launch_bwd<__half>(A, s) : launch_bwd<__nv_bfloat16>(A, s);
    if (owned) {
        cudaError_t e2 = cudaFreeAsync(ws, s);
        if (e == cudaSuccess) e = e2;
    }
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "rms norm backward: %s", cudaGetErrorString(e));
    return CT_OK;
}
