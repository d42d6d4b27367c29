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
constexpr int kUnroll = 2;  // vectors a thread has in flight

struct ActFwd {
    const void *gate, *up;
    void* y;
    uint8_t *gc, *uc;
    float *gsc, *usc;
    int64_t gs, us, ys;
    int64_t rows;
    int cols, group, group_shift, n_groups;
    float alpha;
};

struct ActBwd {
    const void* dy;
    const uint8_t *gc, *uc;
    const float *gsc, *usc;
    void *dgate, *dup, *y;
    int64_t dys, dgs, dus, ys;
    int64_t rows;
    int cols, group, group_shift, n_groups;
    float alpha;
};

// Work is cut per row into pieces: one thread's vector (rows aligned to 16
// bytes) or one warp's 128 values (any alignment).  Piece i of the launch
// belongs to row i / per_row; a launch covers fewer than 2^31 pieces.
struct Pieces {
    Divider per_row;
    unsigned n;
};

// Forward on 16-byte vectors: a group is 4 to 32 neighbouring lanes, whose
// maxima meet by shuffles; a row is padded to whole groups, so groups of
// short rows share a warp.  Bound by memory: 2 bytes read and 2 + 1 written
// (gated: 4 and 2 + 2) for an element of a 16-bit tensor.  Measured: gated silu
// of 16384 x 4096 bf16, both inputs kept in int8, 90 us, 6000 GB/s, 90% of the
// copy rate; two vectors a thread in flight.
template <typename T, int VEC, int Q, int A, int U>
__global__ void __launch_bounds__(kThreads) act_fwd_vec(ActFwd P, Pieces W) {
    const int lanes = P.group / VEC;
    int64_t row[U];
    int col[U];
    bool in[U];
    Vec<T, VEC> gv[U], uv[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const unsigned i = (blockIdx.x * U + j) * kThreads + threadIdx.x;
        unsigned piece;
        row[j] = divide(i, W.per_row, &piece);
        col[j] = (int)piece * VEC;
        in[j] = i < W.n && col[j] < P.cols;
        gv[j].zero();
        uv[j].zero();
        if (in[j]) {
            gv[j].load(static_cast<const T*>(P.gate) + row[j] * P.gs + col[j]);
            if (P.up) uv[j].load(static_cast<const T*>(P.up) + row[j] * P.us + col[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        float a[VEC], b[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            a[k] = gv[j].get(k);
            b[k] = uv[j].get(k);
        }
        if (in[j] && P.y) {
            float o[VEC];
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                float2 f = act_value2<A, sizeof(T) == 2>(pair(a + k), P.alpha);
                if (P.up) f = __fmul2_rn(f, pair(b + k));
                put(o + k, f);
            }
            Vec<T, VEC> ov;
            ov.set(o);
            ov.store(static_cast<T*>(P.y) + row[j] * P.ys + col[j]);
        }
        unsigned amax = gv[j].top_bits(), bmax = uv[j].top_bits();
        if constexpr (sizeof(T) == 2) {  // both inputs' maxima in one word
            const uint32_t both = lanes_max2(amax | bmax << 16, lanes);
            amax = both & 0xffffu;
            bmax = both >> 16;
        } else {
            amax = lanes_max(amax, lanes);
            if (P.up) bmax = lanes_max(bmax, lanes);
        }
        if (!in[j]) continue;
        const bool first = (threadIdx.x & (lanes - 1)) == 0;
        const int64_t at = row[j] * P.n_groups + (col[j] >> P.group_shift);
        float scale, inv;
        group_scale<Q>(Vec<T, VEC>::to_abs_bits(amax), scale, inv);
        store_codes<Q, VEC>(P.gc + row[j] * P.cols + col[j], a, inv);
        if (first) P.gsc[at] = scale;
        if (P.up) {
            group_scale<Q>(Vec<T, VEC>::to_abs_bits(bmax), scale, inv);
            store_codes<Q, VEC>(P.uc + row[j] * P.cols + col[j], b, inv);
            if (first) P.usc[at] = scale;
        }
    }
}

// The gradient (and, without dy, reading a checkpoint back) on 16-byte
// vectors.  Bound by memory: dy and the codes read, one or two gradients
// written.  Measured: the two gradients of the case above 84 us, 6450 GB/s,
// 96% of the copy rate.
template <typename T, int VEC, int Q, int A, int U>
__global__ void __launch_bounds__(kThreads) act_bwd_vec(ActBwd P, Pieces W) {
    int64_t row[U];
    int col[U];
    bool in[U];
    Vec<T, VEC> dv[U];
    uint32_t gw[U][VEC / 4], uw[U][VEC / 4];
    float gsc[U], usc[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const unsigned i = (blockIdx.x * U + j) * kThreads + threadIdx.x;
        unsigned piece;
        row[j] = divide(i, W.per_row, &piece);
        col[j] = (int)piece * VEC;
        in[j] = i < W.n;
        usc[j] = 1.f;
        if (in[j]) {
            const int64_t at = row[j] * P.n_groups + (col[j] >> P.group_shift);
            if (P.dy) dv[j].load(static_cast<const T*>(P.dy) + row[j] * P.dys + col[j]);
            code_words<VEC>(P.gc + row[j] * P.cols + col[j], gw[j]);
            if (P.uc) code_words<VEC>(P.uc + row[j] * P.cols + col[j], uw[j]);
            gsc[j] = P.gsc[at];
            if (P.uc) usc[j] = P.usc[at];
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (!in[j]) continue;
        float a[VEC], b[VEC], f[VEC], slope[VEC], o[VEC];
        Vec<T, VEC> ov;
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            decode4<Q>(gw[j][k], a + 4 * k);
            if (P.uc) decode4<Q>(uw[j][k], b + 4 * k);
        }
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
            put(a + k, __fmul2_rn(pair(a + k), twice(gsc[j])));
            if (P.uc) put(b + k, __fmul2_rn(pair(b + k), twice(usc[j])));
            float2 f2, s2;
            act_both2<A, sizeof(T) == 2>(pair(a + k), P.alpha, f2, s2);
            put(f + k, f2);
            put(slope + k, s2);
        }
        if (P.y) {
#pragma unroll
            for (int k = 0; k < VEC; k += 2) put(o + k, P.uc ? __fmul2_rn(pair(f + k), pair(b + k)) : pair(f + k));
            ov.set(o);
            ov.store(static_cast<T*>(P.y) + row[j] * P.ys + col[j]);
        }
        if (P.dgate) {
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                float2 d = __fmul2_rn(make_float2(dv[j].get(k), dv[j].get(k + 1)), pair(slope + k));
                if (P.uc) d = __fmul2_rn(d, pair(b + k));
                put(o + k, d);
            }
            ov.set(o);
            ov.store(static_cast<T*>(P.dgate) + row[j] * P.dgs + col[j]);
        }
        if (P.dup) {
#pragma unroll
            for (int k = 0; k < VEC; k += 2) put(o + k, __fmul2_rn(make_float2(dv[j].get(k), dv[j].get(k + 1)), pair(f + k)));
            ov.set(o);
            ov.store(static_cast<T*>(P.dup) + row[j] * P.dus + col[j]);
        }
    }
}

// Maximum of each group of a warp's 128 values, slot j of every lane being
// value j * 32 + lane: groups are 1, 2 or 4 slots.
__device__ __forceinline__ void slot_max(unsigned (&m)[4], int group) {
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = __reduce_max_sync(0xffffffffu, m[j]);
    if (group >= 64) {
        m[0] = m[1] = max(m[0], m[1]);
        m[2] = m[3] = max(m[2], m[3]);
    }
    if (group == 128) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
}

// Codes and scales of a warp's 128 values (n of them inside the row).
template <int Q>
__device__ __forceinline__ void keep(const float (&v)[4], const unsigned (&m)[4], int n, int lane, int group, int shift,
                                     uint8_t* codes, float* scales) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        float scale, inv;
        group_scale<Q>(m[j], scale, inv);
        if (k < n) {
            codes[k] = encode<Q>(v[j], inv);
            if ((k & (group - 1)) == 0) scales[k >> shift] = scale;
        }
    }
}

// Forward for rows of any alignment: a warp takes 128 consecutive values,
// four a lane, all loads before the first use.  Bound by the instructions of
// single elements: 16384 x 2048 bf16, gated, 115 us against 49 on vectors.
template <typename T, int Q, int A>
__global__ void __launch_bounds__(kThreads) act_fwd_any(ActFwd P, Pieces W) {
    const int lane = threadIdx.x & 31;
    const unsigned i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= W.n) return;
    unsigned piece;
    const unsigned r32 = divide(i, W.per_row, &piece);
    const int c0 = (int)piece * 128, n = min(128, P.cols - c0);
    const int64_t row = r32;
    const T* g = static_cast<const T*>(P.gate) + row * P.gs + c0;
    const T* u = P.up ? static_cast<const T*>(P.up) + row * P.us + c0 : nullptr;
    T* y = P.y ? static_cast<T*>(P.y) + row * P.ys + c0 : nullptr;
    float a[4], b[4];
    unsigned amax[4], bmax[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        a[j] = k < n ? to_f32(g[k]) : 0.f;
        b[j] = u && k < n ? to_f32(u[k]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        amax[j] = abs_bits(a[j]);
        bmax[j] = abs_bits(b[j]);
        if (y && k < n) {
            const float v = act_value<A, sizeof(T) == 2>(a[j], P.alpha);
            y[k] = from_f32<T>(u ? v * b[j] : v);
        }
    }
    const int64_t at = row * P.n_groups + (c0 >> P.group_shift);
    slot_max(amax, P.group);
    keep<Q>(a, amax, n, lane, P.group, P.group_shift, P.gc + row * P.cols + c0, P.gsc + at);
    if (u) {
        slot_max(bmax, P.group);
        keep<Q>(b, bmax, n, lane, P.group, P.group_shift, P.uc + row * P.cols + c0, P.usc + at);
    }
}

// The gradient for rows of any alignment (16384 x 2048 bf16, gated: 88 us
// against 46 on vectors).
template <typename T, int Q, int A>
__global__ void __launch_bounds__(kThreads) act_bwd_any(ActBwd P, Pieces W) {
    const int lane = threadIdx.x & 31;
    const unsigned i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= W.n) return;
    unsigned piece;
    const unsigned r32 = divide(i, W.per_row, &piece);
    const int c0 = (int)piece * 128, n = min(128, P.cols - c0);
    const int64_t row = r32, at = row * P.n_groups + (c0 >> P.group_shift);
    const uint8_t* gc = P.gc + row * P.cols + c0;
    const uint8_t* uc = P.uc ? P.uc + row * P.cols + c0 : nullptr;
    const T* dy = P.dy ? static_cast<const T*>(P.dy) + row * P.dys + c0 : nullptr;
    float a[4], b[4], d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        const bool in = k < n;
        a[j] = in ? decode<Q>(gc[k]) * P.gsc[at + (k >> P.group_shift)] : 0.f;
        b[j] = uc && in ? decode<Q>(uc[k]) * P.usc[at + (k >> P.group_shift)] : 1.f;
        d[j] = dy && in ? to_f32(dy[k]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = j * 32 + lane;
        if (k >= n) continue;
        float f, slope;
        act_both<A, sizeof(T) == 2>(a[j], P.alpha, f, slope);
        if (P.y) static_cast<T*>(P.y)[row * P.ys + c0 + k] = from_f32<T>(f * b[j]);
        if (P.dgate) static_cast<T*>(P.dgate)[row * P.dgs + c0 + k] = from_f32<T>(d[j] * slope * b[j]);
        if (P.dup) static_cast<T*>(P.dup)[row * P.dus + c0 + k] = from_f32<T>(d[j] * f);
    }
}

bool rows16(const void* p, int64_t stride, size_t eb, int64_t rows) {
    return !p || ((uintptr_t)p % 16 == 0 && (rows <= 1 || (stride * (int64_t)eb) % 16 == 0));
}

// Rows per launch so that its pieces stay below 2^31.
int64_t slab_rows(int per_row) { return std::max<int64_t>(1, ((1ll << 31) - 1 - kThreads * kUnroll) / per_row); }

template <typename T, int Q, int A>
cudaError_t launch_fwd_a(ActFwd P, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = P.cols % V == 0 && rows16(P.gate, P.gs, sizeof(T), P.rows) && rows16(P.up, P.us, sizeof(T), P.rows) &&
                     rows16(P.y, P.ys, sizeof(T), P.rows) && rows16(P.gc, 0, 1, 1) && rows16(P.uc, 0, 1, 1);
    const int per_row = vec ? P.n_groups * (P.group / V) : (P.cols + 127) / 128;
    const int64_t slab = slab_rows(per_row), rows = P.rows;
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t here = std::min(slab, rows - r);
        const Pieces W{divider((unsigned)per_row), (unsigned)(here * per_row)};
        if (vec) act_fwd_vec<T, V, Q, A, kUnroll><<<(W.n + kThreads * kUnroll - 1) / (kThreads * kUnroll), kThreads, 0, s>>>(P, W);
        else act_fwd_any<T, Q, A><<<(W.n + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, s>>>(P, W);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        P.gate = static_cast<const T*>(P.gate) + here * P.gs;
        if (P.up) P.up = static_cast<const T*>(P.up) + here * P.us;
        if (P.y) P.y = static_cast<T*>(P.y) + here * P.ys;
        P.gc += here * P.cols;
        P.gsc += here * P.n_groups;
        if (P.up) P.uc += here * P.cols, P.usc += here * P.n_groups;
    }
    return cudaSuccess;
}

template <typename T, int Q, int A>
cudaError_t launch_bwd_a(ActBwd P, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = P.cols % V == 0 && rows16(P.dy, P.dys, sizeof(T), P.rows) && rows16(P.dgate, P.dgs, sizeof(T), P.rows) &&
                     rows16(P.dup, P.dus, sizeof(T), P.rows) && rows16(P.y, P.ys, sizeof(T), P.rows) && rows16(P.gc, 0, 1, 1) &&
                     rows16(P.uc, 0, 1, 1);
    const int per_row = vec ? P.cols / V : (P.cols + 127) / 128;
    const int64_t slab = slab_rows(per_row), rows = P.rows;
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t here = std::min(slab, rows - r);
        const Pieces W{divider((unsigned)per_row), (unsigned)(here * per_row)};
        if (vec) act_bwd_vec<T, V, Q, A, kUnroll><<<(W.n + kThreads * kUnroll - 1) / (kThreads * kUnroll), kThreads, 0, s>>>(P, W);
        else act_bwd_any<T, Q, A><<<(W.n + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, s>>>(P, W);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (P.dy) P.dy = static_cast<const T*>(P.dy) + here * P.dys;
        if (P.dgate) P.dgate = static_cast<T*>(P.dgate) + here * P.dgs;
        if (P.dup) P.dup = static_cast<T*>(P.dup) + here * P.dus;
        if (P.y) P.y = static_cast<T*>(P.y) + here * P.ys;
        P.gc += here * P.cols;
        P.gsc += here * P.n_groups;
        if (P.uc) P.uc += here * P.cols, P.usc += here * P.n_groups;
    }
    return cudaSuccess;
}

template <typename T, int Q>
cudaError_t launch_fwd(const ActFwd& P, int act, cudaStream_t s) {
    switch (act) {
        case 1: return launch_fwd_a<T, Q, 1>(P, s);
        case 2: return launch_fwd_a<T, Q, 2>(P, s);
        case 3: return launch_fwd_a<T, Q, 3>(P, s);
        case 4: return launch_fwd_a<T, Q, 4>(P, s);
        case 5: return launch_fwd_a<T, Q, 5>(P, s);
        case 6: return launch_fwd_a<T, Q, 6>(P, s);
        default: return launch_fwd_a<T, Q, 0>(P, s);
    }
}

template <typename T, int Q>
cudaError_t launch_bwd(const ActBwd& P, int act, cudaStream_t s) {
    switch (act) {
        case 1: return launch_bwd_a<T, Q, 1>(P, s);
        case 2: return launch_bwd_a<T, Q, 2>(P, s);
        case 3: return launch_bwd_a<T, Q, 3>(P, s);
        case 4: return launch_bwd_a<T, Q, 4>(P, s);
        case 5: return launch_bwd_a<T, Q, 5>(P, s);
        case 6: return launch_bwd_a<T, Q, 6>(P, s);
        default: return launch_bwd_a<T, Q, 0>(P, s);
    }
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

int shift_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

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
             gate_stride, up_stride, y_stride, rows, (int)cols, group, shift_of(group), (int)((cols + group - 1) / group), alpha};
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
             shift_of(group), (int)((cols + group - 1) / group), alpha};
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
