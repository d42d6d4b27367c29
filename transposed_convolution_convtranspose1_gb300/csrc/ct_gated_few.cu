// ct_gated_few.cu -- the gated projection of a few rows (streaming steps).
//
// With a few rows the weights are nearly all there is to read, and each is
// used that often: plain fp32 multiply-adds keep up with memory (at 6.7 TB/s an SM
// gets about 12 16-bit weights a cycle; four rows make 46 multiply-adds of them).  No
// tiles, no copies: weights go from global memory to registers, 16 bytes an access,
// fp32 ones as they are.  Each result is summed in a fixed order.
//
// F dense: a block takes 128 or 256 columns; its warps take every eighth row of W in
// its share of C, blocks of a cluster share C and add up through distributed
// shared memory.  C dense: a warp takes two or four columns, its lanes share C;
// the sums (two for each column and row of x) are added over the lanes by halving
// what a lane keeps in each step.
//
// Measured (graph of calls, weights from HBM, F dense): one row of 2048 channels,
// F = 8192, bf16 14.4 us (4660 GB/s, 70% of the copy rate), fp32 25.5 us (79%); one row
// of 512, F = 2048, bf16 4.5 us.  Bound by the rows of W in flight; with five and
// more rows in 16 bits by the multiply-adds and their conversions (8 rows of 2048,
// F = 8192: 31 us, 44 with C dense; on the tensor cores 20), so those go there.
// fp32 stays up to 16 rows, eight at a time (33 us for eight; as bf16 parts on the
// tensor cores 112).
#include <algorithm>

#include "ct_gated.h"
#include "ct_internal.h"
#include "ct_rows.cuh"

namespace ct {
namespace {

using namespace rows;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSlice = 512;     // of C in shared memory at a time

// F dense: columns of a thread (R pairs of sums for each stay in registers), rows of
// W on their way, and the shared memory of a block.
template <typename T>
constexpr int few_columns() { return 16 / (int)sizeof(T); }
constexpr int kDepth = 6;
template <typename T, int R>
constexpr int few_bytes() {
    constexpr int own = 2 * R * 32 * few_columns<T>() * 4;
    constexpr int a = kSlice * R * 4 + kDepth * 2 * kThreads * 16, b = kWarps * own;
    return (a > b ? a : b) + own;
}

struct Few {
    const void *x, *wg, *wu;
    void* y;
    int64_t xs, gs, us, ys;  // row strides: x, the weights (dense axis last), y
    int rows, C, F, act;
    float alpha;
};

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float of_block(const float* p, unsigned rank) {
    unsigned a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((unsigned)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <bool FAST>
__device__ __forceinline__ float gated(float g, float u, int act, float alpha) {
    float v[1] = {g};
    act_all<1, FAST>(v, act, alpha);
    return v[0] * u;
}

// x[c0 .. c0 + n) of R rows as [c][R] fp32, zeros for rows that there are not.
template <typename T, int R>
__device__ __forceinline__ void stage_x(const Few& A, float* xs, int c0, int n) {
    for (int i = threadIdx.x; i < n * R; i += kThreads) {
        const int r = i / n, c = i - r * n;
        xs[c * R + r] = r < A.rows ? to_f32(static_cast<const T*>(A.x)[r * A.xs + c0 + c]) : 0.f;
    }
}

// F dense.  grid (ranks, strips of columns), clusters of the ranks.
template <typename T, int R>
__global__ void __launch_bounds__(kThreads) gated_few_f(Few A) {
    extern __shared__ __align__(16) float shared[];
    constexpr int V = few_columns<T>(), kColumns = 32 * V, kOwn = 2 * R * kColumns;
    // x [slice][R] and the slots; afterwards the warps' sums [warps][2][R][columns]
    float* const xs = shared;
    char* const slots = reinterpret_cast<char*>(shared + kSlice * R);
    float* const part = shared;
    float* const mine = shared + few_bytes<T, R>() / 4 - kOwn;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ranks = gridDim.x;
    const unsigned rank = ranks > 1 ? cluster_rank() : 0;
    const int col = (int)blockIdx.y * kColumns + lane * V;
    const bool in = col < A.F;
    const int c_begin = (int)((int64_t)A.C * rank / ranks), c_end = (int)((int64_t)A.C * (rank + 1) / ranks);
    const T* wg = static_cast<const T*>(A.wg) + (in ? col : 0);
    const T* wu = static_cast<const T*>(A.wu) + (in ? col : 0);
    float2 g[R][V / 2], u[R][V / 2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) g[r][j] = u[r][j] = make_float2(0.f, 0.f);
    for (int c0 = c_begin; c0 < c_end; c0 += kSlice) {
        const int n = min(kSlice, c_end - c0);
        __syncthreads();
        stage_x<T, R>(A, xs, c0, n);
        __syncthreads();
        // this warp's rows of the slice; kDepth of them are on their way, each thread's
        // pieces in slots of its own
        const int mine_n = warp < n ? (n - warp + kWarps - 1) / kWarps : 0;
        const T* pg = wg + (int64_t)(c0 + warp) * A.gs;
        const T* pu = wu + (int64_t)(c0 + warp) * A.us;
        const int64_t dg = (int64_t)kWarps * A.gs, du = (int64_t)kWarps * A.us;
        int asked = 0;
        const auto ask = [&](int slot) {
            if (asked < mine_n) {
                copy16(slots + (2 * slot * kThreads + threadIdx.x) * 16, pg, true);
                copy16(slots + ((2 * slot + 1) * kThreads + threadIdx.x) * 16, pu, true);
                pg += dg;
                pu += du;
            }
            ++asked;
            copies_commit();
        };
#pragma unroll
        for (int k = 0; k < kDepth; ++k) ask(k);
        const float* xc = xs + warp * R;
        for (int i = 0; i < mine_n; i += kDepth)
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
                copies_wait<kDepth - 1>();
                if (i + k < mine_n) {
                    Vec<T, V> a, b;
                    a.load(reinterpret_cast<const T*>(slots + (2 * k * kThreads + threadIdx.x) * 16));
                    b.load(reinterpret_cast<const T*>(slots + ((2 * k + 1) * kThreads + threadIdx.x) * 16));
                    float p[V], q[V], x[R];
                    a.values(p);
                    b.values(q);
                    if constexpr (R >= 4) {
#pragma unroll
                        for (int r = 0; r < R; r += 4) *reinterpret_cast<float4*>(x + r) = *reinterpret_cast<const float4*>(xc + r);
                    } else {
#pragma unroll
                        for (int r = 0; r < R; ++r) x[r] = xc[r];
                    }
                    xc += kWarps * R;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float2 x2 = twice(x[r]);
#pragma unroll
                        for (int j = 0; j < V / 2; ++j) {
                            g[r][j] = __ffma2_rn(pair(p + 2 * j), x2, g[r][j]);
                            u[r][j] = __ffma2_rn(pair(q + 2 * j), x2, u[r][j]);
                        }
                    }
                }
                ask(k);  // into the slot that has just been read
            }
        copies_wait<0>();
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            *reinterpret_cast<float2*>(part + warp * kOwn + r * kColumns + lane * V + 2 * j) = g[r][j];
            *reinterpret_cast<float2*>(part + warp * kOwn + (R + r) * kColumns + lane * V + 2 * j) = u[r][j];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < kOwn; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[w * kOwn + i];
        mine[i] = s;
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    for (int i = threadIdx.x + (int)rank * kThreads; i < R * kColumns; i += kThreads * ranks) {
        const int r = i / kColumns, c = (int)blockIdx.y * kColumns + i % kColumns;
        float sg = 0.f, su = 0.f;
        for (int k = 0; k < ranks; ++k) {
            sg += ranks > 1 ? of_block(mine + i, k) : mine[i];
            su += ranks > 1 ? of_block(mine + R * kColumns + i, k) : mine[R * kColumns + i];
        }
        if (r < A.rows && c < A.F) static_cast<T*>(A.y)[r * A.ys + c] = from_f32<T>(gated<sizeof(T) == 2>(sg, su, A.act, A.alpha));
    }
    if (ranks > 1) cluster_sync();  // the others have read this block's sums
}

// Sums of N values over the lanes: in each step a lane keeps the half of its
// values that belongs to its bit, until it has one; then the lanes that share
// that one add up.  Returns it; the lane's upper bits say which it is.
template <int N, int BIT = 16>
__device__ __forceinline__ float lanes_sum(float* v, int lane) {
    if constexpr (N > 1) {
        const bool high = lane & BIT;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float give = high ? v[i] : v[i + N / 2], keep = high ? v[i + N / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, BIT);
        }
        return lanes_sum<N / 2, BIT / 2>(v, lane);
    } else {
        float s = v[0];
#pragma unroll
        for (int b = BIT; b; b /= 2) s += __shfl_xor_sync(0xffffffffu, s, b);
        return s;
    }
}

// C dense.  A warp for two or four columns, the whole of C.
constexpr int few_at_once(int R) { return R <= 2 ? 2 : 4; }
template <typename T, int R>
__global__ void __launch_bounds__(kThreads) gated_few_c(Few A) {
    extern __shared__ __align__(16) float shared[];
    constexpr int V = 16 / (int)sizeof(T), kN = few_at_once(R);
    float* const xs = shared;  // [R][slice]
    const int lane = threadIdx.x & 31;
    const int f0 = ((int)blockIdx.x * kWarps + (int)(threadIdx.x >> 5)) * kN;
    // sums of (row, column) pairs; g in the lower half, u in the upper
    float v[2][kN * R];
#pragma unroll
    for (int i = 0; i < kN * R; ++i) v[0][i] = v[1][i] = 0.f;
    for (int c0 = 0; c0 < A.C; c0 += kSlice) {
        const int n = min(kSlice, A.C - c0);
        __syncthreads();
        for (int i = threadIdx.x; i < n * R; i += kThreads) {
            const int r = i / n, c = i - r * n;
            xs[r * kSlice + c] = r < A.rows ? to_f32(static_cast<const T*>(A.x)[r * A.xs + c0 + c]) : 0.f;
        }
        __syncthreads();
        if (f0 < A.F)
#pragma unroll(R <= 2 ? 2 : 1)
            for (int c = lane * V; c < n; c += 32 * V) {
                Vec<T, V> a[kN], b[kN];
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    const int64_t f = min(f0 + k, A.F - 1);  // columns behind the last: read again, not stored
                    a[k].load(static_cast<const T*>(A.wg) + f * A.gs + c0 + c);
                    b[k].load(static_cast<const T*>(A.wu) + f * A.us + c0 + c);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float x[V];
#pragma unroll
                    for (int j = 0; j < V; j += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(xs + r * kSlice + c + j);
                        x[j] = t.x;
                        x[j + 1] = t.y;
                        x[j + 2] = t.z;
                        x[j + 3] = t.w;
                    }
#pragma unroll
                    for (int k = 0; k < kN; ++k)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            v[0][k * R + r] = fmaf(a[k].get(j), x[j], v[0][k * R + r]);
                            v[1][k * R + r] = fmaf(b[k].get(j), x[j], v[1][k * R + r]);
                        }
                }
            }
    }
    constexpr int kShare = 32 / (kN * R);  // lanes that end up with the same pair
    const float g = lanes_sum<kN * R>(v[0], lane), u = lanes_sum<kN * R>(v[1], lane);
    const int f = f0 + lane / kShare / R, r = lane / kShare % R;
    if (lane % kShare == 0 && f < A.F && r < A.rows)
        static_cast<T*>(A.y)[r * A.ys + f] = from_f32<T>(gated<sizeof(T) == 2>(g, u, A.act, A.alpha));
}

template <typename T, int R>
cudaError_t launch_r(const Few& A, bool f_dense, int sm_count, cudaStream_t s) {
    if (!f_dense) {
        constexpr int n = kWarps * few_at_once(R);
        gated_few_c<T, R><<<(unsigned)((A.F + n - 1) / n), kThreads, R * kSlice * 4, s>>>(A);
        return cudaGetLastError();
    }
    constexpr int columns = 32 * few_columns<T>();
    const int strips = (A.F + columns - 1) / columns;
    // two blocks an SM, 16 rows of W a block at least
    int ranks = 1;
    while (ranks < 8 && strips * ranks < 2 * sm_count && A.C >= 32 * ranks) ranks *= 2;
    constexpr int bytes = few_bytes<T, R>();
    auto k = gated_few_f<T, R>;
    if (bytes > 48 << 10) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ranks, (unsigned)strips);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, A);
}

template <typename T>
cudaError_t launch_t(const Few& A, bool f_dense, int sm_count, cudaStream_t s) {
    if (A.rows <= 1) return launch_r<T, 1>(A, f_dense, sm_count, s);
    if (A.rows <= 2) return launch_r<T, 2>(A, f_dense, sm_count, s);
    if constexpr (sizeof(T) == 4)
        if (A.rows > 4) return launch_r<T, 8>(A, f_dense, sm_count, s);
    return launch_r<T, 4>(A, f_dense, sm_count, s);
}

}  // namespace

bool gated_few_fits(int64_t rows, int64_t C, int64_t F, bool f_dense, int dtype) {
    // vectors end with the rows of W: of 8 columns, or 16 bytes of C
    return rows <= (dtype == CT_F32 ? 16 : 4) && (f_dense ? F % 8 == 0 && F <= 65535 * 128 : C % (dtype == CT_F32 ? 4 : 8) == 0);
}

cudaError_t launch_gated_few(const GemmOperand& x, const GemmOperand& wg, const GemmOperand& wu, bool f_dense, void* y, int64_t y_stride,
                             int act, float alpha, int dtype, int sm_count, cudaStream_t s) {
    Few A{};
    A.x = x.p; A.wg = wg.p; A.wu = wu.p; A.y = y;
    A.xs = x.stride; A.gs = wg.stride; A.us = wu.stride; A.ys = y_stride;
    A.rows = (int)x.outer; A.C = (int)x.inner; A.F = (int)(f_dense ? wg.inner : wg.outer);
    A.act = act; A.alpha = alpha;
    if (dtype == CT_F32) {
        // eight rows at a time
        for (int64_t r = 0; r < x.outer; r += 8) {
            A.x = static_cast<const float*>(x.p) + r * x.stride;
            A.y = static_cast<float*>(y) + r * y_stride;
            A.rows = (int)std::min<int64_t>(8, x.outer - r);
            const cudaError_t e = launch_t<float>(A, f_dense, sm_count, s);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    return dtype == CT_F16 ? launch_t<__half>(A, f_dense, sm_count, s) : launch_t<__nv_bfloat16>(A, f_dense, sm_count, s);
}

}  // namespace ct
