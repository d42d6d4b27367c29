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

constexpr int kThreads = 256, kLongThreads = 1024;

struct NormFwd {
    const void *x, *res, *w;
    void *y, *h;
    float* rstd;
    uint8_t* codes;
    float* scales;
    int64_t xs, rs, ys, hs;  // row strides, elements
    int64_t rows;
    int cols, group, group_shift, quant;
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

// Rows too long for registers, or long and off 16-byte boundaries: a block per
// row, two passes over it, the second from L1.  2^25 bf16 elements with
// residual, h and int8 codes in rows of 4096: 97 us, bound by the instructions
// of single elements.
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
        const int n_groups = (A.cols + A.group - 1) >> A.group_shift;
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

// A row in registers: TPR threads hold it as NV pieces each of VEC elements,
// so x and the residual are read once and every output is written from
// registers.  Bound by memory: 2 x 2 bytes read and 3 to 5 written for an
// element of a 16-bit tensor, about ten instructions.  VEC is 16 bytes where
// rows are aligned to that; otherwise single elements, which a warp takes in
// runs of 32 consecutive ones so that accesses stay dense and a group of 32,
// 64 or 128 still lies in one warp.  Measured: 16384 x 2048 bf16 with residual,
// h and e4m3 codes 41 us, 5760 GB/s, 86% of the copy rate; issue is active 60%
// of the cycles, the rest waits for loads.
template <typename T, int VEC, int TPR, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_fwd_regs(NormFwd A) {
    __shared__ float part[32];
    constexpr int kRows = THREADS / TPR;  // rows a block handles (TPR = 32: one a warp)
    const int tid = threadIdx.x % TPR, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (TPR == 32 && row >= A.rows) return;  // whole warps
    const T* x = static_cast<const T*>(A.x) + row * A.xs;
    const T* r = A.res ? static_cast<const T*>(A.res) + row * A.rs : nullptr;
    const T* w = static_cast<const T*>(A.w);
    int col[NV];
    Vec<T, VEC> xv[NV], rv[NV], wv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        col[v] = VEC > 1 ? (v * TPR + tid) * VEC : ((tid >> 5) * NV + v) * 32 + lane;
        xv[v].zero();
        rv[v].zero();
        wv[v].zero();
        if (col[v] < A.cols) {
            xv[v].load(x + col[v]);
            if (r) rv[v].load(r + col[v]);
            if (w) wv[v].load(w + col[v]);
        }
    }
    float s[NV][VEC], ss = 0.f;
    if constexpr (VEC > 1) {
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                // + 0 without a residual: only a zero's sign can change
                const float2 p = __fadd2_rn(make_float2(xv[v].get(i), xv[v].get(i + 1)), make_float2(rv[v].get(i), rv[v].get(i + 1)));
                put(s[v] + i, p);
                sq = __ffma2_rn(p, p, sq);
            }
        ss = sq.x + sq.y;
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            s[v][0] = xv[v].get(0) + rv[v].get(0);
            ss = fmaf(s[v][0], s[v][0], ss);
        }
    }
    if constexpr (TPR == 32) ss = warp_sum(ss);
    else ss = block_sum<THREADS>(ss, part);
    const float rstd = 1.f / sqrtf(ss / (float)A.cols + A.eps);
    if (tid == 0 && A.rstd) A.rstd[row] = rstd;
    const int n_groups = (A.cols + A.group - 1) >> A.group_shift;
    [[maybe_unused]] unsigned amax1[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const bool in = col[v] < A.cols;
        float y[VEC], top = 0.f;
        if (in) {
            if (A.h) {
                Vec<T, VEC> o;
                o.set(s[v]);
                o.store(static_cast<T*>(A.h) + row * A.hs + col[v]);
            }
            if constexpr (VEC > 1) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    float2 p = __fmul2_rn(pair(s[v] + i), twice(rstd));
                    if (w) p = __fmul2_rn(p, make_float2(wv[v].get(i), wv[v].get(i + 1)));
                    put(y + i, p);
                    top = abs_max(top, p.x, p.y);
                }
            } else {
                y[0] = s[v][0] * rstd * (w ? wv[v].get(0) : 1.f);
                top = fabsf(y[0]);
            }
            if (A.y) {
                Vec<T, VEC> o;
                o.set(y);
                o.store(static_cast<T*>(A.y) + row * A.ys + col[v]);
            }
        }
        if (A.quant == CT_Q_NONE) continue;
        unsigned amax = abs_bits(top);
        if constexpr (VEC > 1) {
            const int lanes = A.group / VEC;  // VEC is a power of two
            amax = lanes_max(amax, lanes);
            float scale, inv;
            if (A.quant == CT_Q_INT8) group_scale<CT_Q_INT8>(amax, scale, inv);
            else group_scale<CT_Q_E4M3>(amax, scale, inv);
            if (in) {
                uint8_t* c = A.codes + row * A.cols + col[v];
                if (A.quant == CT_Q_INT8) store_codes<CT_Q_INT8, VEC>(c, y, inv);
                else store_codes<CT_Q_E4M3, VEC>(c, y, inv);
                if ((lane & (lanes - 1)) == 0) A.scales[row * n_groups + (col[v] >> A.group_shift)] = scale;
            }
        } else {
            amax1[v] = __reduce_max_sync(0xffffffffu, amax);
            s[v][0] = in ? y[0] : 0.f;
        }
    }
    if constexpr (VEC == 1) {
        if (A.quant != CT_Q_NONE) {
            const int m = A.group / 32;  // runs of 32 in a group: 1, 2 or 4
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (col[v] >= A.cols) continue;
                unsigned amax = amax1[v];
                if (m >= 2) amax = max(amax, amax1[v ^ 1]);
                if (m == 4) amax = max(amax, max(amax1[v ^ 2], amax1[v ^ 3]));
                float scale, inv;
                if (A.quant == CT_Q_INT8) group_scale<CT_Q_INT8>(amax, scale, inv);
                else group_scale<CT_Q_E4M3>(amax, scale, inv);
                A.codes[row * A.cols + col[v]] = A.quant == CT_Q_INT8 ? encode<CT_Q_INT8>(s[v][0], inv) : encode<CT_Q_E4M3>(s[v][0], inv);
                if ((col[v] & (A.group - 1)) == 0) A.scales[row * n_groups + (col[v] >> A.group_shift)] = scale;
            }
        }
    }
}

// Gradient of rows too long for registers: a block takes a contiguous run of
// rows and keeps its share of dw in its own row of the workspace, which it
// reads and writes again with each row.  Bound by the latency of those, so
// 1024 threads: 2^25 bf16 elements in rows of 16392, 264 us against 479 with
// 256.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_rows(NormBwd A) {
    __shared__ float part[32];
    const T* w = static_cast<const T*>(A.w);
    const int64_t r0 = A.rows * blockIdx.x / A.blocks, r1 = A.rows * (blockIdx.x + 1) / A.blocks;
    float* mine = A.part + (int64_t)blockIdx.x * A.cols;
    if (A.dw)
        for (int i = threadIdx.x; i < A.cols; i += kLongThreads) mine[i] = 0.f;
    for (int64_t row = r0; row < r1; ++row) {
        const T* dy = static_cast<const T*>(A.dy) + row * A.dys;
        const T* h = static_cast<const T*>(A.h) + row * A.hs;
        const T* dres = A.dres ? static_cast<const T*>(A.dres) + row * A.drs : nullptr;
        const float rstd = A.rstd[row];
        float c = 0.f;
        for (int i = threadIdx.x; i < A.cols; i += kLongThreads) {
            const float u = to_f32(h[i]) * rstd, d = to_f32(dy[i]);
            c = fmaf(d * (w ? to_f32(w[i]) : 1.f), u, c);
            if (A.dw) mine[i] = fmaf(d, u, mine[i]);
        }
        c = block_sum<kLongThreads>(c, part) / (float)A.cols;
        if (A.dx) {
            T* dx = static_cast<T*>(A.dx) + row * A.dxs;
            for (int i = threadIdx.x; i < A.cols; i += kLongThreads) {
                const float u = to_f32(h[i]) * rstd, d = to_f32(dy[i]) * (w ? to_f32(w[i]) : 1.f);
                dx[i] = from_f32<T>(rstd * (d - u * c) + (dres ? to_f32(dres[i]) : 0.f));
            }
        }
    }
}

// Barrier of the TPR threads that share a row (one of the block's groups).
template <int TPR, int THREADS>
__device__ __forceinline__ void row_barrier(int group) {
    if constexpr (TPR == THREADS) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

// One thread's 16 bytes of global memory into its own 16 bytes of shared
// memory, asynchronously; nothing is copied (zeros) where `in` is false.
__device__ __forceinline__ void copy16(void* to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Gradient with rows in flight: groups of TPR threads take rows in turn, each
// thread 16 bytes of a row.  Bound by memory: dy, h and dresidual read, dx
// written, each once.  The rows come through a ring of STAGES slots that
// belong to single threads (asynchronous copies that only their own thread
// reads), so no barrier guards them, and STAGES - 1 rows of three tensors are
// on their way while one is summed.  A thread keeps its columns' share of dw
// in fp32 registers; at the end the groups of a block add theirs in a fixed
// order and write one row of partial sums.  Measured: 32768 x 2048 bf16 with
// dresidual and dw 88 us with the sum of the parts, 6110 GB/s, 91% of the copy
// rate; two blocks an SM hold 192 KB of rows in flight.
template <typename T, int TPR, int THREADS, int STAGES>
__global__ void __launch_bounds__(THREADS, 2) norm_bwd_ring(NormBwd A) {
    constexpr int VEC = 16 / (int)sizeof(T), kGroups = THREADS / TPR, kWarpsPerRow = TPR / 32;
    extern __shared__ __align__(16) uint4 ring[];  // [STAGES][3][THREADS]
    __shared__ float part[kGroups][2][kWarpsPerRow];
    const int tid = threadIdx.x % TPR, lane = threadIdx.x & 31, group = threadIdx.x / TPR, wr = tid >> 5;
    const int col = tid * VEC;
    const bool in = col < A.cols;
    const T* w = static_cast<const T*>(A.w);
    Vec<T, VEC> wv;
    wv.zero();
    if (w && in) wv.load(w + col);
    float dw[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[i] = 0.f;
    const int64_t step = (int64_t)gridDim.x * kGroups, first = (int64_t)blockIdx.x * kGroups + group;
    auto fetch = [&](int64_t row, int slot) {
        if (row < A.rows) {
            uint4* to = ring + slot * 3 * THREADS + threadIdx.x;
            const int64_t c = in ? col : 0;
            copy16(to, static_cast<const T*>(A.dy) + row * A.dys + c, in);
            copy16(to + THREADS, static_cast<const T*>(A.h) + row * A.hs + c, in);
            if (A.dres) copy16(to + 2 * THREADS, static_cast<const T*>(A.dres) + row * A.drs + c, in);
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(first + k * step, k);
    const float inv_cols = 1.f / (float)A.cols;
    int turn = 0, slot = 0;
    float rstd = first < A.rows ? A.rstd[first] : 0.f;
    for (int64_t row = first; row < A.rows; row += step, turn ^= 1) {
        copies_wait<STAGES - 2>();
        const uint4* at = ring + slot * 3 * THREADS + threadIdx.x;
        Vec<T, VEC> dv, hv, rv;
        dv.load(reinterpret_cast<const T*>(at));
        hv.load(reinterpret_cast<const T*>(at + THREADS));
        rv.zero();
        if (A.dres) rv.load(reinterpret_cast<const T*>(at + 2 * THREADS));
        // the slot emptied in the round before takes the row STAGES - 1 ahead
        fetch(row + (STAGES - 1) * step, slot == 0 ? STAGES - 1 : slot - 1);
        const float next = row + step < A.rows ? A.rstd[row + step] : 0.f;
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float u = hv.get(i) * rstd, d = dv.get(i);
            dw[i] = fmaf(d, u, dw[i]);
            c = fmaf(w ? d * wv.get(i) : d, u, c);
        }
        c = warp_sum(c);
        if constexpr (kWarpsPerRow > 1) {
            // two buffers in turn: the barrier of the next row separates the
            // reads of one from its next writes
            if (lane == 0) part[group][turn][wr] = c;
            row_barrier<TPR, THREADS>(group);
            c = 0.f;
#pragma unroll
            for (int k = 0; k < kWarpsPerRow; ++k) c += part[group][turn][k];
        }
        c *= inv_cols;
        if (A.dx && in) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = hv.get(i) * rstd, d = w ? dv.get(i) * wv.get(i) : dv.get(i);
                o[i] = fmaf(rstd, fmaf(-u, c, d), rv.get(i));
            }
            Vec<T, VEC> ov;
            ov.set(o);
            ov.store(static_cast<T*>(A.dx) + row * A.dxs + col);
        }
        rstd = next;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    if (!A.dw) return;
    if constexpr (kGroups > 1) {
        // every copy has landed (the last ones are empty), so the ring is free
        copies_wait<0>();
        float* acc = reinterpret_cast<float*>(ring);
        for (int g = 0; g < kGroups; ++g) {
            __syncthreads();
            if (group == g)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float& a = acc[i * TPR + tid];
                    a = g == 0 ? dw[i] : a + dw[i];
                }
        }
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[i] = acc[i * TPR + tid];
    }
    if (!in) return;
    float* to = A.part + (int64_t)blockIdx.x * A.cols + col;
#pragma unroll
    for (int i = 0; i < VEC; ++i) to[i] = dw[i];
}

// Gradient with rows in registers: groups of TPR threads take rows in turn
// and keep their columns' share of dw in fp32 registers; at the end the
// groups of a block add theirs in a fixed order and write one row of partial
// sums.  Bound by memory: dy, h and dresidual read, dx written, each once.
template <typename T, int VEC, int TPR, int NV, int THREADS, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) norm_bwd_regs(NormBwd A) {
    constexpr int kGroups = THREADS / TPR, kWarpsPerRow = TPR / 32;
    __shared__ float part[kGroups][2][kWarpsPerRow];
    __shared__ float acc[kGroups > 1 ? TPR * NV * VEC : 1];
    const int tid = threadIdx.x % TPR, lane = threadIdx.x & 31, group = threadIdx.x / TPR, wr = tid >> 5;
    const T* w = static_cast<const T*>(A.w);
    int col[NV];
    Vec<T, VEC> wv[NV];
    float dw[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        col[v] = VEC > 1 ? (v * TPR + tid) * VEC : (wr * NV + v) * 32 + lane;
        wv[v].zero();
        if (w && col[v] < A.cols) wv[v].load(w + col[v]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[v][i] = 0.f;
    }
    const float inv_cols = 1.f / (float)A.cols;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kGroups + group; row < A.rows; row += (int64_t)gridDim.x * kGroups, turn ^= 1) {
        Vec<T, VEC> dv[NV], hv[NV], rv[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            dv[v].zero();
            hv[v].zero();
            rv[v].zero();
            if (col[v] < A.cols) {
                dv[v].load(static_cast<const T*>(A.dy) + row * A.dys + col[v]);
                hv[v].load(static_cast<const T*>(A.h) + row * A.hs + col[v]);
                if (A.dres) rv[v].load(static_cast<const T*>(A.dres) + row * A.drs + col[v]);
            }
        }
        const float rstd = A.rstd[row];
        float c = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = hv[v].get(i) * rstd, d = dv[v].get(i);
                dw[v][i] = fmaf(d, u, dw[v][i]);
                c = fmaf(w ? d * wv[v].get(i) : d, u, c);
            }
        c = warp_sum(c);
        if constexpr (kWarpsPerRow > 1) {
            // two buffers in turn: the barrier of the next row separates the
            // reads of one from its next writes
            if (lane == 0) part[group][turn][wr] = c;
            row_barrier<TPR, THREADS>(group);
            c = 0.f;
#pragma unroll
            for (int k = 0; k < kWarpsPerRow; ++k) c += part[group][turn][k];
        }
        c *= inv_cols;
        if (A.dx)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (col[v] >= A.cols) continue;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = hv[v].get(i) * rstd, d = w ? dv[v].get(i) * wv[v].get(i) : dv[v].get(i);
                    o[i] = fmaf(rstd, fmaf(-u, c, d), rv[v].get(i));
                }
                Vec<T, VEC> ov;
                ov.set(o);
                ov.store(static_cast<T*>(A.dx) + row * A.dxs + col[v]);
            }
    }
    if (!A.dw) return;
    if constexpr (kGroups > 1) {
        for (int g = 0; g < kGroups; ++g) {
            __syncthreads();
            if (group == g)
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float& a = acc[(v * VEC + i) * TPR + tid];
                        a = g == 0 ? dw[v][i] : a + dw[v][i];
                    }
        }
        __syncthreads();
        if (group != 0) return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (col[v] >= A.cols) continue;
        float* to = A.part + (int64_t)blockIdx.x * A.cols + col[v];
#pragma unroll
        for (int i = 0; i < VEC; ++i) to[i] = kGroups > 1 ? acc[(v * VEC + i) * TPR + tid] : dw[v][i];
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

// Rows of partial sums of dw, the same for every kernel below: enough blocks
// to fill the GPU twice over, never more than rows.
int bwd_blocks(int64_t rows, int sm_count) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)sm_count * 2));
}

template <typename T, int VEC, int TPR, int NV>
cudaError_t launch_regs(const NormFwd& A, cudaStream_t s) {
    constexpr int threads = TPR == 32 ? 128 : TPR, per = threads / TPR;
    const int64_t grid = (A.rows + per - 1) / per;
    norm_fwd_regs<T, VEC, TPR, NV, threads><<<(unsigned)grid, threads, 0, s>>>(A);
    return cudaGetLastError();
}

// Whether every row of a matrix starts on a 16-byte boundary.
bool rows16(const void* p, int64_t stride, size_t eb, int64_t rows) {
    return !p || ((uintptr_t)p % 16 == 0 && (rows <= 1 || (stride * (int64_t)eb) % 16 == 0));
}

// Threads and pieces of a row by its width: the fewest threads whose registers
// hold it, so that blocks stay small and rows many.  Measured on 2^25 bf16
// elements with residual, h and int8 codes (us, this / the next wider): 512
// columns in one warp of two vectors a thread 49 / 62 in four; 2048 in 128
// threads 48.  Rows off 16-byte boundaries go element by element (1024 columns
// 122 us; 512 in 64 threads 122, in 128 171), and beyond 1024 columns through
// norm_fwd_rows, whose second pass finds the row in L1: 1032 columns 138 us
// against 179 in registers, 2048 101 against 122, 4096 97 against 355, 8192 101
// against 196.
template <typename T>
cudaError_t launch_fwd(const NormFwd& A, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool fits = A.rows < (1ll << 31);
    if (fits && A.cols % V == 0 && rows16(A.x, A.xs, sizeof(T), A.rows) && rows16(A.res, A.rs, sizeof(T), A.rows) &&
        rows16(A.y, A.ys, sizeof(T), A.rows) && rows16(A.h, A.hs, sizeof(T), A.rows) && rows16(A.w, 0, sizeof(T), 1) &&
        rows16(A.codes, 0, 1, 1)) {
        const int n = A.cols / V;
        if (n <= 32) return launch_regs<T, V, 32, 1>(A, s);
        if (n <= 64) return launch_regs<T, V, 32, 2>(A, s);
        if (n <= 128) return launch_regs<T, V, 32, 4>(A, s);
        if (n <= 256) return launch_regs<T, V, 128, 2>(A, s);
        if (n <= 512) return launch_regs<T, V, 256, 2>(A, s);
        if (n <= 1024) return launch_regs<T, V, 512, 2>(A, s);
        if (n <= 2048) return launch_regs<T, V, 512, 4>(A, s);
        if (n <= 4096) return launch_regs<T, V, 1024, 4>(A, s);
    } else if (fits) {
        if (A.cols <= 256) return launch_regs<T, 1, 32, 8>(A, s);
        if (A.cols <= 512) return launch_regs<T, 1, 64, 8>(A, s);
        if (A.cols <= 1024) return launch_regs<T, 1, 128, 8>(A, s);
    }
    const unsigned grid = (unsigned)std::min<int64_t>(A.rows, 1 << 20);
    if (A.quant == CT_Q_INT8) norm_fwd_rows<T, CT_Q_INT8><<<grid, kThreads, 0, s>>>(A);
    else if (A.quant == CT_Q_E4M3) norm_fwd_rows<T, CT_Q_E4M3><<<grid, kThreads, 0, s>>>(A);
    else norm_fwd_rows<T, CT_Q_NONE><<<grid, kThreads, 0, s>>>(A);
    return cudaGetLastError();
}

template <typename T, int VEC, int TPR, int NV, int THREADS, int MINB>
cudaError_t launch_bwd_regs(const NormBwd& A, cudaStream_t s) {
    norm_bwd_regs<T, VEC, TPR, NV, THREADS, MINB><<<A.blocks, THREADS, 0, s>>>(A);
    return cudaGetLastError();
}

template <typename T, int TPR>
cudaError_t launch_bwd_ring(const NormBwd& A, cudaStream_t s) {
    constexpr int threads = 512, stages = 4, bytes = stages * 3 * threads * 16;
    auto k = norm_bwd_ring<T, TPR, threads, stages>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<A.blocks, threads, bytes, s>>>(A);
    return cudaGetLastError();
}

// The ring up to 512 vectors (2^25 bf16 elements with dresidual and dw: 2048
// columns 52 us, 4096 64), registers to 2048 (8192: 75, 16384: 88), two passes
// beyond (16392: 264).  Off 16-byte boundaries single elements, the narrowest
// group of threads that holds the row (2048 columns: 256 threads 88 us, 512 125;
// 512 columns: 64 threads 82, 128 120).
template <typename T>
cudaError_t launch_bwd_dx(const NormBwd& A, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (A.cols % V == 0 && rows16(A.dy, A.dys, sizeof(T), A.rows) && rows16(A.h, A.hs, sizeof(T), A.rows) &&
        rows16(A.dres, A.drs, sizeof(T), A.rows) && rows16(A.dx, A.dxs, sizeof(T), A.rows) && rows16(A.w, 0, sizeof(T), 1)) {
        const int n = A.cols / V;
        if (n <= 32) return launch_bwd_ring<T, 32>(A, s);
        if (n <= 64) return launch_bwd_ring<T, 64>(A, s);
        if (n <= 128) return launch_bwd_ring<T, 128>(A, s);
        if (n <= 256) return launch_bwd_ring<T, 256>(A, s);
        if (n <= 512) return launch_bwd_ring<T, 512>(A, s);
        if (n <= 1024) return launch_bwd_regs<T, V, 512, 2, 512, 1>(A, s);
        if (n <= 2048) return launch_bwd_regs<T, V, 512, 4, 512, 1>(A, s);
    } else {
        if (A.cols <= 256) return launch_bwd_regs<T, 1, 32, 8, 512, 2>(A, s);
        if (A.cols <= 512) return launch_bwd_regs<T, 1, 64, 8, 512, 2>(A, s);
        if (A.cols <= 1024) return launch_bwd_regs<T, 1, 128, 8, 512, 2>(A, s);
        if (A.cols <= 2048) return launch_bwd_regs<T, 1, 256, 8, 512, 2>(A, s);
        if (A.cols <= 4096) return launch_bwd_regs<T, 1, 512, 8, 512, 2>(A, s);
        if (A.cols <= 8192) return launch_bwd_regs<T, 1, 512, 16, 512, 1>(A, s);
    }
    norm_bwd_rows<T><<<A.blocks, kLongThreads, 0, s>>>(A);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd(const NormBwd& A, cudaStream_t s) {
    if (A.rows > 0) {
        cudaError_t e = launch_bwd_dx<T>(A, s);
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
              y_stride, h_stride, rows, (int)cols, quant != CT_Q_NONE ? group : 128, group == 32 ? 5 : group == 64 ? 6 : 7, quant, eps};
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
