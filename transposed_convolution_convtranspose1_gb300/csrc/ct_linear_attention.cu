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

struct ScanArgs {
    LaCore c;
    const int* only;         // heads with flag 0 are left alone ...
    const float* kept;       // ... but for m_out, copied from here
    int seg_tokens;          // of a segment (blockIdx.z)
    int m_in_seg, m_out_seg; // a matrix for each segment; m_out: its own sum
};

// A block owns 32 columns of one head's matrix: columns of M never meet, so
// the only sum across threads is out = M^T z over the rows.  Lane = 4 row
// runs x 8 column quads, each thread RX consecutive rows x 4 columns in
// registers.  A token's partial sums are joined by three shuffles (each halves
// the columns a lane still carries) and, across the four warps, through shared
// memory once per TB tokens; the next TB tokens' values are on their way in
// registers meanwhile.  A streaming step (one token) is bound by memory, the
// state read and written: 64 x 8 heads of 128 x 128, 67 MB, 15 us, 66% of the
// copy rate (256 x 8 heads 52 us, 77%).  Longer sequences are bound by each
// token's chain of sums.
template <typename T, int RX, int TB>
__global__ void __launch_bounds__(kWarps * 32) la_scan(const __grid_constant__ ScanArgs S) {
    const LaCore& A = S.c;
    constexpr int D = kWarps * 4 * RX, kThreads = kWarps * 32;  // D: rows held (>= Da)
    constexpr int NX = TB * D / kThreads, NY = TB * kCols / kThreads;
    static_assert(NX > 0 && NY > 0, "a thread stages whole elements");
    __shared__ __align__(16) float xs[TB][D];
    __shared__ __align__(16) float zs[TB][D];
    __shared__ __align__(16) float ys[TB][kCols];
    __shared__ __align__(16) float part[kWarps][TB][kCols];
    __shared__ float first_gamma;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane >> 3, c4 = (lane & 7) * 4;
    const int a0 = (warp * 4 + sub) * RX, b0 = blockIdx.y * kCols;
    const int64_t bh = blockIdx.x, BH = gridDim.x;
    const int b = (int)(bh / A.H), h = (int)(bh % A.H);
    const int len = A.lengths ? max(0, min(A.T, A.lengths[b])) : A.T;
    const int s0 = blockIdx.z * S.seg_tokens, s1 = min(A.T, s0 + S.seg_tokens);
    const int n = max(0, min(len, s1) - s0);  // tokens of this segment
    // backward in time the sequence's last token takes the matrix undecayed
    const bool holds_end = A.reverse && n > 0 && s0 + n == len;
    const float gamma = expf(la_log_decay(A.log_decay[h]));
    const T* z = static_cast<const T*>(A.z) + b * A.zs[0] + s0 * A.zs[1] + h * A.zs[2];
    const T* x = static_cast<const T*>(A.x) + b * A.xs[0] + s0 * A.xs[1] + h * A.xs[2];
    const T* y = static_cast<const T*>(A.y) + b * A.ys[0] + s0 * A.ys[1] + h * A.ys[2];
    T* out = A.out ? static_cast<T*>(A.out) + b * A.os[0] + s0 * A.os[1] + h * A.os[2] : nullptr;
    const int64_t msize = (int64_t)A.Da * A.Db;
    const float* m_in = A.m_in ? A.m_in + (bh + (S.m_in_seg ? blockIdx.z * BH : 0)) * msize : nullptr;
    float* m_out = A.m_out ? A.m_out + (bh + (S.m_out_seg ? blockIdx.z * BH : 0)) * msize : nullptr;
    if (S.only && !S.only[bh]) {
        if (S.kept)
            for (int i = tid; i < A.Da * kCols; i += kThreads) {
                const int c = b0 + i % kCols;
                const int64_t e = (int64_t)(i / kCols) * A.Db + c;
                if (c < A.Db) m_out[e] = S.kept[bh * msize + e];
            }
        return;
    }

    // four columns as one access where a row's quads lie on 16 bytes
    const bool quads = A.Db % 4 == 0 && !A.m_in_t && ((uintptr_t)m_in | (uintptr_t)m_out) % 16 == 0;
    float m[RX][4];
#pragma unroll
    for (int i = 0; i < RX; ++i) {
        const int a = a0 + i, c0 = b0 + c4;
        if (quads) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m_in && a < A.Da && c0 < A.Db) v = *reinterpret_cast<const float4*>(m_in + (int64_t)a * A.Db + c0);
            m[i][0] = v.x; m[i][1] = v.y; m[i][2] = v.z; m[i][3] = v.w;
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + j;
            m[i][j] = 0.f;
            if (m_in && a < A.Da && c < A.Db) m[i][j] = m_in[A.m_in_t ? (int64_t)c * A.Da + a : (int64_t)a * A.Db + c];
        }
    }
    // gamma is rounded, and its t-th power is off by t times that: 7e-6 of the
    // result after 300 tokens.  So the first step of every further round of TB
    // takes what makes the round's product exp(TB g).
    if (tid == 0 && n > TB) {
        double p = 1.0;
#pragma unroll 1
        for (int i = 1; i < TB; ++i) p *= (double)gamma;
        first_gamma = gamma > 1e-10f ? (float)(exp((double)TB * (double)A.log_decay[h]) / p) : gamma;
    }
    float px[NX], pz[NX], py[NY];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int t = (i * kThreads + tid) / D, a = (i * kThreads + tid) % D;
            const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
            const bool in = t0 + t < n && a < A.Da;
            px[i] = in ? to_f32(x[tok * A.xs[1] + a]) : 0.f;
            pz[i] = in && out ? to_f32(z[tok * A.zs[1] + a]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int t = (i * kThreads + tid) / kCols, c = (i * kThreads + tid) % kCols;
            const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
            py[i] = t0 + t < n && b0 + c < A.Db ? to_f32(y[tok * A.ys[1] + b0 + c]) * A.mscale : 0.f;
        }
    };
    if (n > 0) fetch(0);
    for (int t0 = 0; t0 < n; t0 += TB) {
        const int nt = min(TB, n - t0);
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int e = i * kThreads + tid;
            xs[e / D][e % D] = px[i];
            zs[e / D][e % D] = pz[i];
        }
#pragma unroll
        for (int i = 0; i < NY; ++i) ys[(i * kThreads + tid) / kCols][(i * kThreads + tid) % kCols] = py[i];
        __syncthreads();
        if (t0 + TB < n) fetch(t0 + TB);
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
            const float g = t > 0 ? gamma : t0 > 0 ? first_gamma : holds_end ? 1.f : gamma;
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
            // lanes 8 apart keep two columns each, lanes 16 apart one
            const bool odd = sub & 1, high = sub & 2;
            float k0 = odd ? acc[2] : acc[0], k1 = odd ? acc[3] : acc[1];
            k0 += __shfl_xor_sync(0xffffffffu, odd ? acc[0] : acc[2], 8);
            k1 += __shfl_xor_sync(0xffffffffu, odd ? acc[1] : acc[3], 8);
            const float k = (high ? k1 : k0) + __shfl_xor_sync(0xffffffffu, high ? k0 : k1, 16);
            part[warp][t][c4 + (odd ? 2 : 0) + (high ? 1 : 0)] = k;
        }
        __syncthreads();
        if (out)
            for (int i = tid; i < nt * kCols; i += kThreads) {
                const int t = i / kCols, c = i % kCols;
                const int64_t tok = A.reverse ? n - 1 - (t0 + t) : t0 + t;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += part[w][t][c];
                if (b0 + c < A.Db) out[tok * A.os[1] + b0 + c] = from_f32<T>(s * A.oscale);
            }
        // the next round writes xs, ys and zs at once, which nothing reads
        // any more, and its partial sums after its own barrier
    }
    if (out)
        for (int64_t i = tid; i < (int64_t)(s1 - s0 - n) * kCols; i += kThreads) {
            const int c = (int)(i % kCols);
            if (b0 + c < A.Db) out[(n + i / kCols) * A.os[1] + b0 + c] = from_f32<T>(0.f);
        }
    if (m_out) {
        const float g = A.reverse && !S.m_out_seg && n > 0 ? gamma : 1.f;
#pragma unroll
        for (int i = 0; i < RX; ++i) {
            if (a0 + i >= A.Da) continue;
            float* to = m_out + (int64_t)(a0 + i) * A.Db + b0 + c4;
            if (quads) {
                if (b0 + c4 < A.Db) *reinterpret_cast<float4*>(to) = make_float4(g * m[i][0], g * m[i][1], g * m[i][2], g * m[i][3]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (b0 + c4 + j < A.Db) to[j] = g * m[i][j];
        }
    }
}

template <typename T, int TB>
cudaError_t launch_tb(const ScanArgs& S, int segs, cudaStream_t s) {
    const LaCore& A = S.c;
    const dim3 grid((unsigned)(A.B * A.H), (unsigned)((A.Db + kCols - 1) / kCols), (unsigned)segs);
    if (A.Da <= 32) la_scan<T, 2, TB><<<grid, kWarps * 32, 0, s>>>(S);
    else if (A.Da <= 64) la_scan<T, 4, TB><<<grid, kWarps * 32, 0, s>>>(S);
    else if (A.Da <= 128) la_scan<T, 8, TB><<<grid, kWarps * 32, 0, s>>>(S);
    else la_scan<T, 16, TB < 8 ? TB : 8><<<grid, kWarps * 32, 0, s>>>(S);
    return cudaGetLastError();
}

// Streaming steps stage four tokens: fewer registers, so more of the state in
// flight (512 heads of 128 x 128 on the GPU, one state again and again, which
// L2 keeps: 11.7 us; 20.4 with sixteen).
template <typename T>
cudaError_t launch_t(const ScanArgs& S, int segs, cudaStream_t s) {
    return S.c.T <= 4 ? launch_tb<T, 4>(S, segs, s) : launch_tb<T, 16>(S, segs, s);
}

cudaError_t launch(const ScanArgs& S, int segs, cudaStream_t s) {
    if (S.c.B * S.c.H == 0) return cudaSuccess;
    switch (S.c.dtype) {
        case CT_F32: return launch_t<float>(S, segs, s);
        case CT_F16: return launch_t<__half>(S, segs, s);
        default: return launch_t<__nv_bfloat16>(S, segs, s);
    }
}

// Segments of the scan and the tokens of one.  A segment is walked twice, and
// the matrices between cost as much again where they are many (64 heads of
// 128 x 128, 128 tokens: 127 us in several, 39 in one), so sequences are cut
// only where two blocks to an SM leave room for four segments of at least 64
// tokens (f32, heads of 64: 38 heads of 512 tokens in four 61 us, 39 in one 78;
// of 256 tokens 40 and 41; 15 heads of 40 x 72, 333 tokens in five 41, in one
// 78).
void scan_split(int64_t BH, int64_t T, int64_t Db, int* segs, int* tokens) {
    DeviceInfo d;
    const int64_t room = 2 * (device_info(&d) == cudaSuccess ? d.sm_count : 152);
    const int64_t blocks = std::max<int64_t>(1, BH * ((Db + kCols - 1) / kCols));
    int64_t want = std::min<int64_t>(std::min<int64_t>(room / blocks, T / 64), 4096);
    if (want < 4) want = 1;
    *tokens = (int)std::max<int64_t>(1, (T + want - 1) / want);
    *segs = (int)std::max<int64_t>(1, (T + *tokens - 1) / *tokens);
}

}  // namespace

size_t la_scan_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Da, int64_t Db) {
    int segs, tokens;
    scan_split(B * H, T, Db, &segs, &tokens);
    return segs > 1 ? ((size_t)B * H * Da * Db * segs * sizeof(float) + 255) / 256 * 256 : 0;
}

cudaError_t launch_la_scan(const LaCore& c, void* workspace, cudaStream_t s) {
    ScanArgs S{c, nullptr, nullptr, 0, 0, 0};
    int segs;
    scan_split(c.B * c.H, c.T, c.Db, &segs, &S.seg_tokens);
    if (segs == 1) return launch(S, 1, s);
    float* sums = static_cast<float*>(workspace);
    S.c.out = nullptr;
    S.c.m_in = nullptr;
    S.c.m_out = sums;
    S.m_out_seg = 1;
    cudaError_t e = launch(S, segs, s);
    if (e != cudaSuccess) return e;
    LaChainBatch C{};
    C.core[0] = {sums, c.m_in, c.m_out, c.m_in_t, c.reverse, c.Da, c.Db};
    C.log_decay = c.log_decay;
    C.lengths = c.lengths;
    C.T = c.T;
    C.H = c.H;
    C.BH = (int)(c.B * c.H);
    C.seg_tokens = S.seg_tokens;
    C.segs = segs;
    e = launch_la_chain(C, 1, s);
    if (e != cudaSuccess || !c.out) return e;
    S.c = c;
    S.c.m_in = sums;
    S.c.m_in_t = 0;
    S.c.m_out = nullptr;
    S.m_in_seg = 1;
    S.m_out_seg = 0;
    return launch(S, segs, s);
}

cudaError_t launch_la_scan_again(const LaCore& c, const int* flags, const float* kept, cudaStream_t s) {
    return launch(ScanArgs{c, flags, kept, std::max(1, c.T), 0, 0}, 1, s);
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

// Whichever kernel the strides lead to.
size_t workspace_of(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, int dtype, int backward) {
    size_t n = std::max(la_tc_workspace_bytes(B, T, H, Dk, Dv, dtype, backward), la_scan_workspace_bytes(B, T, H, Dk, Dv));
    if (backward) n = std::max(n, la_scan_workspace_bytes(B, T, H, Dv, Dk));
    return n;
}

cudaError_t launch_core(const LaCore& c, void* workspace, cudaStream_t s) {
    return la_tc_supports(c) ? launch_la_tc(&c, 1, workspace, s) : launch_la_scan(c, workspace, s);
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
    *bytes = workspace_of(B, T, H, Dk, Dv, dtype, backward);
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
    rc = ws.take(workspace, workspace_bytes, workspace_of(B, T, H, Dk, Dv, dtype, 0), s);
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
    rc = ws.take(workspace, workspace_bytes, workspace_of(B, T, H, Dk, Dv, dtype, 1), s);
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
