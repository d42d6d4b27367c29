// ct_linear_attention.cu -- causal linear attention with a decay for each
// head: host side (checks, the four uses of the recurrence) and the kernel
// that runs the recurrence token by token.
#include <algorithm>
#include <cmath>

#include "ct_linear_attention.h"
#include "ct_types.cuh"

namespace ct {
namespace {

constexpr int kWarps = 4;
constexpr int kCols = 32;    // columns of M a block owns
constexpr int kTokens = 16;  // tokens staged at a time

// A block owns 32 columns of one head's matrix: columns of M never meet, so
// the only sum across threads is out = M^T z over the rows.  Lane = 4 row
// runs x 8 column quads, each thread RX consecutive rows x 4 columns in
// registers; partial outputs are joined by two shuffles and, across the four
// warps, through shared memory once per 16 tokens.
template <typename T, int RX>
__global__ void __launch_bounds__(kWarps * 32) la_scan(LaCore A, const int* only, const float* kept) {
    constexpr int D = kWarps * 4 * RX;  // rows held (>= Da)
    __shared__ __align__(16) float xs[kTokens][D];
    __shared__ __align__(16) float zs[kTokens][D];
    __shared__ __align__(16) float ys[kTokens][kCols];
    __shared__ __align__(16) float part[kWarps][kTokens][kCols];
    __shared__ float first_gamma;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane >> 3, c4 = (lane & 7) * 4;
    const int a0 = (warp * 4 + sub) * RX, b0 = blockIdx.y * kCols;
    const int64_t bh = blockIdx.x;
    const int b = (int)(bh / A.H), h = (int)(bh % A.H);
    const int n = A.lengths ? max(0, min(A.T, A.lengths[b])) : A.T;
    // exp(0 * g) must be 1 for a decay of zero (g = -infinity) too
    const float gamma = expf(fmaxf(A.log_decay[h], -1e30f));
    const T* z = static_cast<const T*>(A.z) + b * A.zs[0] + h * A.zs[2];
    const T* x = static_cast<const T*>(A.x) + b * A.xs[0] + h * A.xs[2];
    const T* y = static_cast<const T*>(A.y) + b * A.ys[0] + h * A.ys[2];
    T* out = static_cast<T*>(A.out) + b * A.os[0] + h * A.os[2];
    const int64_t msize = (int64_t)A.Da * A.Db;
    if (only && !only[bh]) {
        if (kept)
            for (int i = tid; i < A.Da * kCols; i += kWarps * 32) {
                const int c = b0 + i % kCols;
                if (c < A.Db) A.m_out[bh * msize + (int64_t)(i / kCols) * A.Db + c] = kept[bh * msize + (int64_t)(i / kCols) * A.Db + c];
            }
        return;
    }

    float m[RX][4];
#pragma unroll
    for (int i = 0; i < RX; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int a = a0 + i, c = b0 + c4 + j;
            m[i][j] = 0.f;
            if (A.m_in && a < A.Da && c < A.Db)
                m[i][j] = A.m_in[bh * msize + (A.m_in_t ? (int64_t)c * A.Da + a : (int64_t)a * A.Db + c)];
        }
    // gamma is rounded, and its t-th power is off by t times that: 7e-6 of the
    // result after 300 tokens.  So the first step of every further round of 16
    // takes what makes the round's product exp(16 g).
    if (tid == 0 && n > kTokens) {
        const double e = gamma, e2 = e * e, e4 = e2 * e2, e8 = e4 * e4;
        first_gamma = gamma > 1e-10f ? (float)(exp(16.0 * (double)A.log_decay[h]) / (e8 * e4 * e2 * e)) : gamma;
    }
    for (int t0 = 0; t0 < n; t0 += kTokens) {
        const int nt = min(kTokens, n - t0);
        for (int i = tid; i < nt * D; i += kWarps * 32) {
            const int t = i / D, a = i % D;
            const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
            xs[t][a] = a < A.Da ? to_f32(x[tok * A.xs[1] + a]) : 0.f;
            zs[t][a] = a < A.Da ? to_f32(z[tok * A.zs[1] + a]) : 0.f;
        }
        for (int i = tid; i < nt * kCols; i += kWarps * 32) {
            const int t = i / kCols, c = i % kCols;
            const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
            ys[t][c] = b0 + c < A.Db ? to_f32(y[tok * A.ys[1] + b0 + c]) * A.mscale : 0.f;
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float g = t > 0 ? gamma : t0 > 0 ? first_gamma : A.reverse ? 1.f : gamma;
            float yv[4], acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yv[j] = ys[t][c4 + j];
                acc[j] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < RX; ++i) {
                const float xv = xs[t][a0 + i], zv = zs[t][a0 + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    m[i][j] = fmaf(xv, yv[j], g * m[i][j]);
                    acc[j] = fmaf(m[i][j], zv, acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 8);
                acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 16);
                if (sub == 0) part[warp][t][c4 + j] = acc[j];
            }
        }
        __syncthreads();
        if (A.out)
            for (int i = tid; i < nt * kCols; i += kWarps * 32) {
                const int t = i / kCols, c = i % kCols;
                const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += part[w][t][c];
                if (b0 + c < A.Db) out[tok * A.os[1] + b0 + c] = from_f32<T>(s * A.oscale);
            }
        // the next round's staging writes xs, ys and zs only, and its partial
        // sums come after its own barrier
    }
    if (A.out)
        for (int64_t i = tid; i < (int64_t)(A.T - n) * kCols; i += kWarps * 32) {
            const int c = (int)(i % kCols);
            if (b0 + c < A.Db) out[(n + i / kCols) * A.os[1] + b0 + c] = from_f32<T>(0.f);
        }
    if (A.m_out) {
        const float g = A.reverse && n > 0 ? gamma : 1.f;
#pragma unroll
        for (int i = 0; i < RX; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (a0 + i < A.Da && b0 + c4 + j < A.Db)
                    A.m_out[bh * msize + (int64_t)(a0 + i) * A.Db + b0 + c4 + j] = g * m[i][j];
    }
}

template <typename T>
cudaError_t launch_t(const LaCore& A, cudaStream_t s, const int* only, const float* kept) {
    const dim3 grid((unsigned)(A.B * A.H), (unsigned)((A.Db + kCols - 1) / kCols));
    if (A.Da <= 32) la_scan<T, 2><<<grid, kWarps * 32, 0, s>>>(A, only, kept);
    else if (A.Da <= 64) la_scan<T, 4><<<grid, kWarps * 32, 0, s>>>(A, only, kept);
    else if (A.Da <= 128) la_scan<T, 8><<<grid, kWarps * 32, 0, s>>>(A, only, kept);
    else la_scan<T, 16><<<grid, kWarps * 32, 0, s>>>(A, only, kept);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_scan(const LaCore& A, cudaStream_t s, const int* only, const float* kept) {
    if (A.B * A.H == 0) return cudaSuccess;
    switch (A.dtype) {
        case CT_F32: return launch_t<float>(A, s, only, kept);
        case CT_F16: return launch_t<__half>(A, s, only, kept);
        default: return launch_t<__nv_bfloat16>(A, s, only, kept);
    }
}

namespace {

bool bad_ptr(const void* p, size_t a) { return p && (uintptr_t)p % a != 0; }

int check(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, int dtype) {
    if (dtype != CT_F32 && dtype != CT_F16 && dtype != CT_BF16)
        return report_error(CT_ERR_DTYPE, "dtype %d is not a supported floating type (CT_F32, CT_F16, CT_BF16)", dtype);
    if (B < 0 || T < 0 || H < 0 || Dk < 1 || Dv < 1)
        return report_error(CT_ERR_SHAPE, "B, T and H must be >= 0 and the head sizes >= 1");
    if (Dk > kLaMaxD || Dv > kLaMaxD) return report_error(CT_ERR_TOO_LARGE, "head sizes up to %d are supported", kLaMaxD);
    if (T > (1ll << 30) || H > (1 << 20) || B > (1ll << 30) || B * H > (1ll << 31) - 1)
        return report_error(CT_ERR_TOO_LARGE, "T <= 2^30 and B * H < 2^31 supported");
    return CT_OK;
}

void set3(int64_t* d, const int64_t* s) { for (int i = 0; i < 3; ++i) d[i] = s[i]; }

int done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? CT_OK : report_error(CT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Workspace of a call: the caller's, checked, or the call's own.
struct Workspace {
    void* p = nullptr;
    bool owned = false;
    int take(void* given, size_t bytes, size_t need, cudaStream_t s) {
        if (need == 0) return CT_OK;
        if (given) {
            if (bytes < need)
                return report_error(CT_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", bytes, need);
            if (bad_ptr(given, 256)) return report_error(CT_ERR_ALIGN, "workspace must be 256-byte aligned");
            p = given;
            return CT_OK;
        }
        cudaError_t e = cudaMallocAsync(&p, need, s);
        if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "cudaMallocAsync(workspace): %s", cudaGetErrorString(e));
        owned = true;
        return CT_OK;
    }
    cudaError_t give_back(cudaError_t e, cudaStream_t s) {
        const cudaError_t e2 = owned ? cudaFreeAsync(p, s) : cudaSuccess;
        return e == cudaSuccess ? e2 : e;
    }
};

cudaError_t launch_core(const LaCore& c, void* workspace, cudaStream_t s) {
    return la_tc_supports(c) ? launch_la_tc(&c, 1, workspace, s) : launch_la_scan(c, s);
}

LaCore core_of(const float* log_decay, const int32_t* lengths, int64_t B, int64_t T, int64_t H, int dtype) {
    LaCore c{};
    c.log_decay = log_decay;
    c.lengths = lengths;
    c.mscale = c.oscale = 1.f;
    c.B = B;
    c.T = (int)T;
    c.H = (int)H;
    c.dtype = dtype;
    return c;
}

}  // namespace
}  // namespace ct

using namespace ct;

extern "C" int ct_linear_attention_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, int dtype,
                                                   int backward, size_t* bytes) {
    if (backward != 0 && backward != 1) return report_error(CT_ERR_PARAM, "backward must be 0 or 1");
    if (!bytes) return report_error(CT_ERR_NULL, "bytes is NULL");
    int rc = check(B, T, H, Dk, Dv, dtype);
    if (rc != CT_OK) return rc;
    *bytes = la_tc_workspace_bytes(B, T, H, Dk, Dv, dtype, backward);
    return CT_OK;
}

extern "C" int ct_linear_attention_forward(const void* q, const int64_t* q_strides, const void* k,
                                           const int64_t* k_strides, const void* v, const int64_t* v_strides, void* o,
                                           const int64_t* o_strides, const float* log_decay, const float* state_in,
                                           float* state_out, const int32_t* lengths, void* workspace,
                                           size_t workspace_bytes, int64_t B, int64_t T, int64_t H, int64_t Dk,
                                           int64_t Dv, float scale, int dtype, void* stream) {
    int rc = check(B, T, H, Dk, Dv, dtype);
    if (rc != CT_OK) return rc;
    if (B * H == 0) return CT_OK;
    if (!log_decay || (T > 0 && (!q || !k || !v || !o)) || !q_strides || !k_strides || !v_strides || !o_strides)
        return report_error(CT_ERR_NULL, "q, k, v, o, their strides and log_decay must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(q, eb) || bad_ptr(k, eb) || bad_ptr(v, eb) || bad_ptr(o, eb) || bad_ptr(log_decay, 4) ||
        bad_ptr(state_in, 4) || bad_ptr(state_out, 4) || bad_ptr(lengths, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    LaCore c = core_of(log_decay, lengths, B, T, H, dtype);
    c.x = k; c.y = v; c.z = q; c.out = o;
    set3(c.xs, k_strides); set3(c.ys, v_strides); set3(c.zs, q_strides); set3(c.os, o_strides);
    c.Da = (int)Dk; c.Db = (int)Dv;
    c.m_in = state_in; c.m_out = state_out;
    c.oscale = scale;
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    rc = ws.take(workspace, workspace_bytes, la_tc_supports(c) ? la_tc_workspace_bytes(B, T, H, Dk, Dv, dtype, 0) : 0, s);
    if (rc != CT_OK) return rc;
    return done(ws.give_back(launch_core(c, ws.p, s), s), "linear attention");
}

extern "C" int ct_linear_attention_backward(const void* q, const int64_t* q_strides, const void* k,
                                            const int64_t* k_strides, const void* v, const int64_t* v_strides,
                                            const void* dout, const int64_t* do_strides, const float* log_decay,
                                            const float* state_in, const float* dstate_out, const int32_t* lengths,
                                            void* dq, const int64_t* dq_strides, void* dk, const int64_t* dk_strides,
                                            void* dv, const int64_t* dv_strides, float* dstate_in, void* workspace,
                                            size_t workspace_bytes, int64_t B, int64_t T, int64_t H, int64_t Dk,
                                            int64_t Dv, float scale, int dtype, void* stream) {
    int rc = check(B, T, H, Dk, Dv, dtype);
    if (rc != CT_OK) return rc;
    if (B * H == 0) return CT_OK;
    if (!log_decay || (T > 0 && (!q || !k || !v || !dout)) || !q_strides || !k_strides || !v_strides || !do_strides ||
        (dq && !dq_strides) || (dk && !dk_strides) || (dv && !dv_strides))
        return report_error(CT_ERR_NULL, "q, k, v, dout, log_decay and the strides of each tensor must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(q, eb) || bad_ptr(k, eb) || bad_ptr(v, eb) || bad_ptr(dout, eb) || bad_ptr(dq, eb) || bad_ptr(dk, eb) ||
        bad_ptr(dv, eb) || bad_ptr(log_decay, 4) || bad_ptr(state_in, 4) || bad_ptr(dstate_out, 4) ||
        bad_ptr(dstate_in, 4) || bad_ptr(lengths, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    rc = ws.take(workspace, workspace_bytes, la_tc_workspace_bytes(B, T, H, Dk, Dv, dtype, 1), s);
    if (rc != CT_OK) return rc;
    // dstate_in may be dstate_out's own buffer: the walk that writes it is the
    // last to read it
    LaCore walks[3];
    int n = 0;
    if (dq && T > 0) {
        LaCore& c = walks[n++] = core_of(log_decay, lengths, B, T, H, dtype);
        c.x = v; c.y = k; c.z = dout; c.out = dq;
        set3(c.xs, v_strides); set3(c.ys, k_strides); set3(c.zs, do_strides); set3(c.os, dq_strides);
        c.Da = (int)Dv; c.Db = (int)Dk;
        c.m_in = state_in; c.m_in_t = 1;
        c.oscale = scale;
    }
    if (dk && T > 0) {
        LaCore& c = walks[n++] = core_of(log_decay, lengths, B, T, H, dtype);
        c.x = dout; c.y = q; c.z = v; c.out = dk;
        set3(c.xs, do_strides); set3(c.ys, q_strides); set3(c.zs, v_strides); set3(c.os, dk_strides);
        c.Da = (int)Dv; c.Db = (int)Dk;
        c.m_in = dstate_out; c.m_in_t = 1;
        c.mscale = scale;
        c.reverse = 1;
    }
    if ((dv && T > 0) || dstate_in) {
        LaCore& c = walks[n++] = core_of(log_decay, lengths, B, T, H, dtype);
        c.x = q; c.y = dout; c.z = k; c.out = T > 0 ? dv : nullptr;
        set3(c.xs, q_strides); set3(c.ys, do_strides); set3(c.zs, k_strides);
        if (dv) set3(c.os, dv_strides);
        c.Da = (int)Dk; c.Db = (int)Dv;
        c.m_in = dstate_out; c.m_out = dstate_in;
        c.mscale = scale;
        c.reverse = 1;
    }
    // together where their tiles are alike: three times the CTAs.  In one
    // launch nothing orders the walks, so a shared buffer keeps them apart.
    bool together = n > 1 && (dstate_in == nullptr || dstate_in != dstate_out) && (Dk <= 64) == (Dv <= 64);
    for (int i = 0; i < n; ++i) together = together && walks[i].out && la_tc_supports(walks[i]);
    cudaError_t e = cudaSuccess;
    if (together) e = launch_la_tc(walks, n, ws.p, s);
    else
        for (int i = 0; i < n && e == cudaSuccess; ++i) e = launch_core(walks[i], ws.p, s);
    return done(ws.give_back(e, s), "linear attention backward");
}
