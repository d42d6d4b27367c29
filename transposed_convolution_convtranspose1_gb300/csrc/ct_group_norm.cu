// ct_group_norm.cu -- group norm with an activation over channels-last tokens,
// and its gradient.
//
//   x [B, S, C]; a group is Cg = C / groups channels of one of the B
//   m = mean, v = variance over the group's S * Cg values, rstd = (v + eps)^-1/2
//   n = (x - m) * rstd,  u = n * weight + bias,  y = act(u)
//
// Gradient from x, m and rstd, with du = dy * act'(u):
//   s1 = sum of weight * du, s2 = sum of weight * du * n over the group
//   dx = rstd * (weight * du - (s1 + n * s2) / (S * Cg))
//   dweight = sum over b, s of du * n,  dbias = sum over b, s of du
//
// Two passes, statistics and application, with a join between: a block sums a
// chunk of positions for each channel and its channels for each group, small
// blocks join the chunks of a group in a fixed order, and a second pass over x
// writes the result.  Calls larger than
// the L2 keeps go over samples in ranges, so that the second pass reads what
// the first one left in L2.
//
// The statistics are those of differences: a thread takes the mean of its first
// positions and sums what the others differ from it, and the squares of that;
// threads, blocks and channels are joined by the rule for two sets (counts n,
// means m, squares q about the means): q = qa + qb + (mb - ma)^2 na nb / (na + nb).
// Squares of x itself are never summed: they would lose a spread that is small
// next to the mean.
#include <algorithm>

#include "ct_internal.h"
#include "ct_rows.cuh"

namespace ct {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kBlocks = 2;  // resident on an SM
constexpr int kBwdBlocks = 2;
constexpr int kTile = 256;  // vectors of channels a block spans at most
constexpr int kRows = 4, kBwdRows = 2;  // positions of a batch
constexpr int kDepth = 4;               // batches of a ring

struct GroupNorm {
    const void *x, *dy, *w, *b;
    void* y;                      // or dx
    void *dw, *db;
    const float *mean, *rstd;     // [B][groups]
    float *mean_out, *rstd_out;
    float2* part;                 // [B][chunks][C]: (mean, squares about it), or (sum of du, sum of du * n)
    float2* sums;                 // [B][C]: (sum of du, sum of du * n)
    float2* coef;                 // [B][groups]: (s1, s2) / (S * Cg)
    int64_t xb, xr, yb, yr, db_, dr;  // strides of batch and position: x, y or dx, dy
    int64_t b0;                   // first sample of this launch
    int64_t B, S;
    int C, G, Cg, chunks, act;
    int early;                    // gn_bwd_channels beside gn_bwd_apply
    int grouped;                  // the first pass joins its channels to groups itself
    float2* gpart;                // [B][chunks][groups]: (mean, squares about it), or the chunk's part of (s1, s2)
    int set, slot_bytes;          // one pass: channels of a cluster, bytes of a block's slots
    int64_t chunk_rows;
    Divider by_cg;
    float eps, alpha;
};

// The join and the second pass are launched while the kernel before them still
// runs; what it wrote is there after this.
__device__ __forceinline__ void after_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Where a thread works: `lanes` threads share a vector of channels and take
// every lanes-th position of the chunk [r0, r1).
struct Place {
    int lane, lanes, vec, vecs, c, n;  // n: positions of this thread
    int64_t b, first;                  // the first of them
    bool on;
};
template <int V>
__device__ __forceinline__ Place place(const GroupNorm& A, int64_t chunk) {
    Place p;
    const int all = A.C / V, first = (int)blockIdx.y * kTile;
    p.vecs = min(kTile, all - first);
    p.lanes = kThreads / p.vecs;
    p.lane = (int)threadIdx.x / p.vecs;
    p.vec = (int)threadIdx.x - p.lane * p.vecs;
    p.on = p.lane < p.lanes;
    p.c = (first + p.vec) * V;
    const int64_t r0 = chunk * A.chunk_rows;
    const int rows = (int)min(A.S - r0, A.chunk_rows);
    p.first = r0 + p.lane;
    p.n = p.on && p.lane < rows ? (rows - p.lane + p.lanes - 1) / p.lanes : 0;
    return p;
}

// A vector of a thread's own, asynchronously.
template <int BYTES>
__device__ __forceinline__ void copy_bytes(void* to, const void* from) {
    if constexpr (BYTES == 16) copy16(to, from, true);
    else if constexpr (BYTES == 2) *static_cast<unsigned short*>(to) = *static_cast<const unsigned short*>(from);  // no asynchronous copy is that small
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from), "n"(BYTES) : "memory");
}

// A thread's positions, `BATCH` at a time, of STREAMS tensors.  Vectors of 4 bytes
// or more come through a ring in shared memory whose slots belong to single
// threads (asynchronous copies that only their own thread reads: no barriers),
// DEPTH - 1 batches on their way while one is worked on; single 16-bit values are
// loaded as they are needed.
template <typename T, int V, int STREAMS, int BATCH, int DEPTH>
struct Stream {
    static constexpr int kVec = V * (int)sizeof(T);
    static constexpr bool kRing = kVec >= 4;
    static constexpr int kSlot = BATCH * STREAMS * kThreads * kVec;  // of a batch
    static constexpr int kBytes = kRing ? DEPTH * kSlot : 0;
    const T* p[STREAMS];      // of the batch to fetch next
    int64_t step[STREAMS];    // from a position of this thread to its next
    int left, ahead;          // positions to come, to fetch
    char *ring, *at, *end;

    // p and step are set; `n` positions
    __device__ __forceinline__ void begin(int n, uint4* smem) {
        left = ahead = n;
        ring = at = reinterpret_cast<char*>(smem) + threadIdx.x * kVec;
        end = ring + DEPTH * kSlot;
        if constexpr (kRing)
#pragma unroll
            for (int k = 0; k < DEPTH - 1; ++k) fetch(ring + k * kSlot);
    }
    __device__ __forceinline__ void fetch(char* to) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (j < ahead)
#pragma unroll
                for (int i = 0; i < STREAMS; ++i) copy_bytes<kVec>(to + (j * STREAMS + i) * kThreads * kVec, p[i] + j * step[i]);
#pragma unroll
        for (int i = 0; i < STREAMS; ++i) p[i] += BATCH * step[i];
        ahead -= BATCH;
        copies_commit();
    }
    // The next batch; how many of its positions there are (0: the end).
    __device__ __forceinline__ int next(Vec<T, V> (&v)[STREAMS][BATCH]) {
        if (left <= 0) return 0;
        if constexpr (kRing) {
            copies_wait<DEPTH - 2>();
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
#pragma unroll
                for (int i = 0; i < STREAMS; ++i) v[i][j].load(reinterpret_cast<const T*>(at + (j * STREAMS + i) * kThreads * kVec));
            // into the slot that the round before emptied
            fetch(at == ring ? end - kSlot : at - kSlot);
            at += kSlot;
            if (at == end) at = ring;
        } else {
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (j < left)
#pragma unroll
                    for (int i = 0; i < STREAMS; ++i) v[i][j].load(p[i] + j * step[i]);
#pragma unroll
            for (int i = 0; i < STREAMS; ++i) p[i] += BATCH * step[i];
        }
        const int got = min(left, BATCH);
        left -= BATCH;
        return got;
    }
    __device__ __forceinline__ void finish() const {
        if constexpr (kRing) copies_wait<0>();
    }
};

// A thread's statistics: sums of x less the mean of its first batch.
template <typename T, int V>
struct Sums {
    float sum[V], sqr[V], minus[V];
    __device__ __forceinline__ void begin(const Vec<T, V> (&v)[kRows], int got) {
        const float few = 1.f / (float)got;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (j < got) s += v[j].get(i);
            minus[i] = -s * few;
            sum[i] = sqr[i] = 0.f;
        }
    }
    __device__ __forceinline__ void add(const Vec<T, V> (&v)[kRows], int got) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (j >= got) break;
            float d[V];
            v[j].values(d);
            add_all(d, minus);
            add_all(sum, d);
            fma_all(sqr, d, d, sqr);
        }
    }
    __device__ __forceinline__ void end(int n, float (&mean)[V], float (&squares)[V]) const {
        const float inv = 1.f / (float)n;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float m = sum[i] * inv;
            mean[i] = m - minus[i];
            squares[i] = fmaf(-m, sum[i], sqr[i]);
        }
    }
};

// The lanes of a vector joined in a tree; lane 0 has the result.
template <int V>
__device__ __forceinline__ void join_lanes(const Place& p, int n, float (&mean)[V], float (&sqr)[V], int* sn, float* sm, float* sq) {
    __syncthreads();
    sn[threadIdx.x] = n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sm[i * kThreads + threadIdx.x] = mean[i];
        sq[i * kThreads + threadIdx.x] = sqr[i];
    }
    int half = 1;
    while (half < p.lanes) half *= 2;
    for (half /= 2; half; half /= 2) {
        __syncthreads();
        if (p.lane < half && p.lane + half < p.lanes) {
            const int o = threadIdx.x + half * p.vecs, m = sn[o];
            if (m) {
                const float scale = (float)m / (float)(n + m), weight = (float)n * scale;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = sm[i * kThreads + o] - mean[i];
                    mean[i] = fmaf(d, scale, mean[i]);
                    sqr[i] += fmaf(d * weight, d, sq[i * kThreads + o]);
                    sm[i * kThreads + threadIdx.x] = mean[i];
                    sq[i * kThreads + threadIdx.x] = sqr[i];
                }
                sn[threadIdx.x] = n += m;
            }
        }
    }
    __syncthreads();
}
// Positions of a chunk (one pass: of a block of the cluster).
__device__ __forceinline__ float rows_of(const GroupNorm& A, int chunk) {
    return (float)max((int64_t)0, min(A.S - chunk * A.chunk_rows, A.chunk_rows));
}
// Channels' (mean, squares) of `rows` positions each to groups', a warp for each.
__device__ __forceinline__ void join_channels(const GroupNorm& A, const float* sm, const float* sq, float rows, int groups, float2* out) {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
        float s = 0.f, q = 0.f;
        for (int c = lane; c < A.Cg; c += 32) s += sm[g * A.Cg + c];
        s = warp_sum(s) / (float)A.Cg;
        for (int c = lane; c < A.Cg; c += 32) {
            const float d = sm[g * A.Cg + c] - s;
            q += fmaf(d * d, rows, sq[g * A.Cg + c]);
        }
        q = warp_sum(q);
        if (lane == 0) out[g] = make_float2(s, q);
    }
}
// The same for plain sums.
template <int V>
__device__ __forceinline__ void join_lanes_sums(const Place& p, float (&a)[V], float (&q)[V], float* sa, float* sb) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sa[i * kThreads + threadIdx.x] = a[i];
        sb[i * kThreads + threadIdx.x] = q[i];
    }
    int half = 1;
    while (half < p.lanes) half *= 2;
    for (half /= 2; half; half /= 2) {
        __syncthreads();
        if (p.lane < half && p.lane + half < p.lanes) {
            const int o = threadIdx.x + half * p.vecs;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sa[i * kThreads + threadIdx.x] = a[i] += sa[i * kThreads + o];
                sb[i * kThreads + threadIdx.x] = q[i] += sb[i * kThreads + o];
            }
        }
    }
}

// First pass.  Bound by memory: 2 x 262144 positions of 64 channels, bf16, 67 MB in
// about 15 us from a cold start (the launch included); two blocks an SM have up to
// 96 KB of positions on their way.  Three blocks with 80 registers a thread took 38
// us for the whole call, two with room for all of it 36.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, kBlocks) gn_stats(GroupNorm A) {
    extern __shared__ uint4 smem[];
    float *const sm = reinterpret_cast<float*>(smem), *const sq = sm + kThreads * V;  // after the loop
    __shared__ int sn[kThreads];
    let_next_kernel_start();
    Place p = place<V>(A, blockIdx.x);
    p.b = A.b0 + blockIdx.z;
    float mean[V], sqr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] = sqr[i] = 0.f;
    if (p.n) {
        Stream<T, V, 1, kRows, kDepth> in;
        in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
        in.step[0] = p.lanes * A.xr;
        in.begin(p.n, smem);
        Vec<T, V> v[1][kRows];
        Sums<T, V> sums;
        int got = in.next(v);
        sums.begin(v[0], got);
        do {
            sums.add(v[0], got);
            got = in.next(v);
        } while (got);
        in.finish();
        sums.end(p.n, mean, sqr);
    }
    join_lanes<V>(p, p.n, mean, sqr, sn, sm, sq);
    if (A.grouped) {
        if (p.lane == 0)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sm[p.c + i] = mean[i];
                sq[p.c + i] = sqr[i];
            }
        __syncthreads();
        join_channels(A, sm, sq, rows_of(A, blockIdx.x), A.G, A.gpart + (p.b * A.chunks + blockIdx.x) * A.G);
        return;
    }
    if (p.lane == 0) {
        float2* out = A.part + (p.b * A.chunks + blockIdx.x) * A.C + p.c;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = make_float2(mean[i], sqr[i]);
    }
}

// Where a block has not all channels: a block for each group, the chunks and
// channels joined, mean first and then the squares about it.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) gn_join(GroupNorm A) {
    __shared__ float red[32];
    const int64_t b = A.b0 + blockIdx.x / A.G;
    const int g = (int)(blockIdx.x % A.G), items = A.chunks * A.Cg;
    const float2* part = A.part + b * A.chunks * A.C + g * A.Cg;
    let_next_kernel_start();
    after_previous_kernel();
    const float count = (float)A.S * (float)A.Cg;
    // item i: channel i mod Cg of chunk i / Cg
    const auto at = [&](int i, float* rows) {
        unsigned c;
        const unsigned k = divide((unsigned)i, A.by_cg, &c);
        *rows = (float)min(A.chunk_rows, A.S - k * A.chunk_rows);
        return part[(int64_t)k * A.C + c];
    };
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += THREADS) {
        float rows;
        const float2 v = at(i, &rows);
        s = fmaf(v.x, rows, s);
    }
    const float mean = block_sum<THREADS>(s, red) / count;
    float q = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += THREADS) {
        float rows;
        const float2 v = at(i, &rows);
        const float d = v.x - mean;
        q += fmaf(d * d, rows, v.y);
    }
    q = block_sum<THREADS>(q, red);
    if (threadIdx.x == 0) {
        A.mean_out[b * A.G + g] = mean;
        A.rstd_out[b * A.G + g] = 1.f / sqrtf(q / count + A.eps);
    }
}

// The same from what the first pass's blocks left of each group: a warp for each.
__global__ void __launch_bounds__(kThreads) gn_join_groups(GroupNorm A, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    let_next_kernel_start();
    after_previous_kernel();
    if (i >= n) return;
    const int64_t b = A.b0 + i / A.G;
    const int g = (int)(i % A.G);
    const float2* part = A.gpart + b * A.chunks * A.G + g;
    float s = 0.f, q = 0.f;
#pragma unroll 4
    for (int k = lane; k < A.chunks; k += 32) s = fmaf(part[(int64_t)k * A.G].x, rows_of(A, k) / (float)A.S, s);
    s = warp_sum(s);
#pragma unroll 4
    for (int k = lane; k < A.chunks; k += 32) {
        const float2 v = part[(int64_t)k * A.G];
        const float d = v.x - s;
        q += fmaf(d * d, rows_of(A, k) * (float)A.Cg, v.y);
    }
    q = warp_sum(q);
    if (lane == 0) {
        A.mean_out[b * A.G + g] = s;
        A.rstd_out[b * A.G + g] = 1.f / sqrtf(q / ((float)A.S * (float)A.Cg) + A.eps);
    }
}

// A vector's mean, weight * rstd and bias.
template <typename T, int V>
struct Channels {
    float mean[V], scale[V], bias[V];
    __device__ __forceinline__ void load(const GroupNorm& A, int64_t b, int c) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t g = b * A.G + (c + i) / A.Cg;
            mean[i] = A.mean[g];
            scale[i] = A.rstd[g] * (A.w ? to_f32(static_cast<const T*>(A.w)[c + i]) : 1.f);
            bias[i] = A.b ? to_f32(static_cast<const T*>(A.b)[c + i]) : 0.f;
        }
    }
};

// Second pass.  Bound by memory and, with silu, by the special-function unit (an
// exponential and a reciprocal an element): the same tensor 20 us cold; after the
// first pass x comes from L2.  All three kernels: 36 us in a graph, 39 in a program
// (67 MB read and written: 3410 GB/s, 51% of the copy rate).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, kBlocks) gn_apply(GroupNorm A) {
    // the last positions first: they are the ones most likely still in L2
    Place p = place<V>(A, gridDim.x - 1 - blockIdx.x);
    p.b = A.b0 + gridDim.z - 1 - blockIdx.z;
    if (!p.on) return;
    extern __shared__ uint4 smem[];
    constexpr bool kFast = sizeof(T) == 2;
    Stream<T, V, 1, kRows, kDepth> in;
    in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
    in.step[0] = p.lanes * A.xr;
    in.begin(p.n, smem);
    after_previous_kernel();
    Channels<T, V> ch;
    ch.load(A, p.b, p.c);
    T* y = static_cast<T*>(A.y) + p.b * A.yb + p.first * A.yr + p.c;
    const int64_t step = p.lanes * A.yr;
    Vec<T, V> x[1][kRows];
    while (const int got = in.next(x)) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (j >= got) break;
            float v[V];
            x[0][j].values(v);
            sub_all(v, ch.mean);
            fma_all(v, v, ch.scale, ch.bias);
            act_all<V, kFast>(v, A.act, A.alpha);
            Vec<T, V> out;
            out.set(v);
            out.stream(y);
            y += step;
        }
    }
}

// x - mean and du of V values.
template <typename T, int V>
__device__ __forceinline__ void centred_and_du(const GroupNorm& A, const Channels<T, V>& ch, const Vec<T, V>& x, const Vec<T, V>& dy,
                                               float (&d)[V], float (&du)[V]) {
    float u[V];
    x.values(d);
    dy.values(du);
    sub_all(d, ch.mean);
    fma_all(u, d, ch.scale, ch.bias);
    times_slope<V, sizeof(T) == 2>(du, u, A.act, A.alpha);
}

// First pass of the gradient: sums of du and du * n for each channel.  Bound by
// memory, the slope's exponential and reciprocal close behind: 16 x 4096 positions
// of 256 channels, bf16, 67 MB in 18 us cold.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) gn_bwd_sums(GroupNorm A) {
    extern __shared__ uint4 smem[];
    float *const sa = reinterpret_cast<float*>(smem), *const sb = sa + kThreads * V;  // after the loop
    let_next_kernel_start();
    Place p = place<V>(A, blockIdx.x);
    p.b = A.b0 + blockIdx.z;
    float a[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = q[i] = 0.f;
    if (p.on) {
        Stream<T, V, 2, kBwdRows, kDepth> in;
        in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
        in.p[1] = static_cast<const T*>(A.dy) + p.b * A.db_ + p.first * A.dr + p.c;
        in.step[0] = p.lanes * A.xr;
        in.step[1] = p.lanes * A.dr;
        in.begin(p.n, smem);
        Channels<T, V> ch;
        ch.load(A, p.b, p.c);
        Vec<T, V> v[2][kBwdRows];
        while (const int got = in.next(v)) {
#pragma unroll
            for (int j = 0; j < kBwdRows; ++j) {
                if (j >= got) break;
                float d[V], du[V];
                centred_and_du<T, V>(A, ch, v[0][j], v[1][j], d, du);
                add_all(a, du);
                fma_all(q, du, d, q);
            }
        }
        in.finish();
    }
    join_lanes_sums<V>(p, a, q, sa, sb);
    if (p.lane == 0) {
        float2* out = A.part + (p.b * A.chunks + blockIdx.x) * A.C + p.c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            q[i] *= A.rstd[p.b * A.G + (p.c + i) / A.Cg];
            out[i] = make_float2(a[i], q[i]);
        }
    }
    if (A.grouped) {
        __syncthreads();
        if (p.lane == 0)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = A.w ? to_f32(static_cast<const T*>(A.w)[p.c + i]) : 1.f;
                sa[p.c + i] = a[i] * w;
                sb[p.c + i] = q[i] * w;
            }
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int g = threadIdx.x >> 5; g < A.G; g += kThreads / 32) {
            float s1 = 0.f, s2 = 0.f;
            for (int c = lane; c < A.Cg; c += 32) {
                s1 += sa[g * A.Cg + c];
                s2 += sb[g * A.Cg + c];
            }
            s1 = warp_sum(s1);
            s2 = warp_sum(s2);
            if (lane == 0) A.gpart[(p.b * A.chunks + blockIdx.x) * A.G + g] = make_float2(s1, s2);
        }
    }
}

// A block for each group of a sample: its channels' sums over the chunks, and
// s1 and s2 from those.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) gn_bwd_join(GroupNorm A) {
    __shared__ float red[32];
    __shared__ float2 lanes_sum[THREADS];
    const int64_t b = A.b0 + blockIdx.x / A.G;
    const int g = (int)(blockIdx.x % A.G);
    const float2* part = A.part + b * A.chunks * A.C + g * A.Cg;
    float2* sums = A.sums + b * A.C + g * A.Cg;
    const T* w = A.w ? static_cast<const T*>(A.w) + g * A.Cg : nullptr;
    float s1 = 0.f, s2 = 0.f;
    let_next_kernel_start();
    after_previous_kernel();
    for (int c0 = 0; c0 < A.Cg; c0 += THREADS) {
        // `width` channels at a time, `n` threads share the chunks of each
        const int width = min(THREADS, A.Cg - c0), n = THREADS / width, lane = threadIdx.x / width, c = threadIdx.x - lane * width;
        float2 v = make_float2(0.f, 0.f);
        if (lane < n)
#pragma unroll 4
            for (int k = lane; k < A.chunks; k += n) {
                const float2 u = part[(int64_t)k * A.C + c0 + c];
                v.x += u.x;
                v.y += u.y;
            }
        __syncthreads();
        lanes_sum[threadIdx.x] = v;
        __syncthreads();
        if (lane == 0) {
            for (int k = 1; k < n; ++k) {
                const float2 u = lanes_sum[k * width + c];
                v.x += u.x;
                v.y += u.y;
            }
            sums[c0 + c] = v;
            const float f = w ? to_f32(w[c0 + c]) : 1.f;
            s1 = fmaf(v.x, f, s1);
            s2 = fmaf(v.y, f, s2);
        }
    }
    s1 = block_sum<THREADS>(s1, red);
    s2 = block_sum<THREADS>(s2, red);
    if (threadIdx.x == 0) {
        const float inv = 1.f / ((float)A.S * (float)A.Cg);
        A.coef[b * A.G + g] = make_float2(s1 * inv, s2 * inv);
    }
}

// s1 and s2 from the chunks' parts of each group: a warp for each.
__global__ void __launch_bounds__(kThreads) gn_bwd_join_groups(GroupNorm A, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    let_next_kernel_start();
    after_previous_kernel();
    if (i >= n) return;
    const int64_t b = A.b0 + i / A.G;
    const int g = (int)(i % A.G);
    const float2* part = A.gpart + b * A.chunks * A.G + g;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int k = lane; k < A.chunks; k += 32) {
        const float2 v = part[(int64_t)k * A.G];
        s1 += v.x;
        s2 += v.y;
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    const float inv = 1.f / ((float)A.S * (float)A.Cg);
    if (lane == 0) A.coef[b * A.G + g] = make_float2(s1 * inv, s2 * inv);
}

// dweight and dbias: 32 channels a block, 32 warps share the samples (and
// their chunks, where no join has added those up).
template <typename T>
__global__ void __launch_bounds__(1024) gn_bwd_channels(GroupNorm A) {
    __shared__ float sa[32][33], sb[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float a = 0.f, q = 0.f;
    const int64_t n = A.S ? (A.grouped ? A.B * A.chunks : A.B) : 0;
    const float2* from = A.grouped ? A.part : A.sums;
    // beside the second pass: the sums were there before that let this kernel start; who
    // waits for this kernel has then waited for both
    if (!A.early) after_previous_kernel();
    if (c < A.C)
#pragma unroll 8
        for (int64_t k = warp; k < n; k += 32) {
            const float2 v = from[k * A.C + c];
            a += v.x;
            q += v.y;
        }
    sa[warp][lane] = a;
    sb[warp][lane] = q;
    __syncthreads();
    a = warp_sum(sa[lane][warp]);
    q = warp_sum(sb[lane][warp]);
    const int d = blockIdx.x * 32 + warp;
    if (lane == 0 && d < A.C) {
        if (A.db) static_cast<T*>(A.db)[d] = from_f32<T>(a);
        if (A.dw) static_cast<T*>(A.dw)[d] = from_f32<T>(q);
    }
    if (A.early) after_previous_kernel();
}

// Second pass of the gradient: x and dy from L2, dx written.  18 us cold for the
// same tensors; all four kernels 33 us in a graph, 35 to 36 in a program (101 MB:
// 2800 GB/s, 42% of the copy rate).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) gn_bwd_apply(GroupNorm A) {
    Place p = place<V>(A, gridDim.x - 1 - blockIdx.x);
    p.b = A.b0 + gridDim.z - 1 - blockIdx.z;
    if (!p.on) return;
    extern __shared__ uint4 smem[];
    Stream<T, V, 2, kBwdRows, kDepth> in;
    in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
    in.p[1] = static_cast<const T*>(A.dy) + p.b * A.db_ + p.first * A.dr + p.c;
    in.step[0] = p.lanes * A.xr;
    in.step[1] = p.lanes * A.dr;
    in.begin(p.n, smem);
    Channels<T, V> ch;
    ch.load(A, p.b, p.c);
    after_previous_kernel();
    let_next_kernel_start();
    float m1[V], m2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t g = p.b * A.G + (p.c + i) / A.Cg;
        const float rstd = A.rstd[g];
        const float2 s = A.coef[g];
        m1[i] = -s.x * rstd;
        m2[i] = -s.y * rstd * rstd;  // of x - mean
    }
    T* dx = static_cast<T*>(A.y) + p.b * A.yb + p.first * A.yr + p.c;
    const int64_t step = p.lanes * A.yr;
    Vec<T, V> v[2][kBwdRows];
    while (const int got = in.next(v)) {
#pragma unroll
        for (int j = 0; j < kBwdRows; ++j) {
            if (j >= got) break;
            float d[V], du[V];
            centred_and_du<T, V>(A, ch, v[0][j], v[1][j], d, du);
            fma_all(d, d, m2, m1);
            fma_all(du, du, ch.scale, d);
            Vec<T, V> out;
            out.set(du);
            out.stream(dx);
            dx += step;
        }
    }
}

// ---- one pass -----------------------------------------------------------------
//
// A sample's channels are cut into sets of whole groups, and a cluster of up to
// eight blocks keeps all positions of a set in shared memory: x is read once,
// the blocks exchange a few numbers for each group (distributed shared memory),
// and the result is written from what they hold.  A thread's slots are its own,
// as in Stream, but none is used twice.

constexpr int kHeldBytes = 224 << 10;  // shared memory of a block at most
constexpr int kHeldDepth = 6;  // batches on their way

template <typename T, int V, int STREAMS, int BATCH>
struct Held {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kSlot = BATCH * STREAMS * kThreads * kBytes;  // of a batch
    const T* p[STREAMS];
    int64_t step[STREAMS];
    int left, ahead;
    char *at, *to;

    __device__ __forceinline__ void begin(int n, char* smem) {
        left = ahead = n;
        at = to = smem + threadIdx.x * kBytes;
#pragma unroll
        for (int k = 0; k < kHeldDepth; ++k) fetch();
    }
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (j < ahead)
#pragma unroll
                for (int i = 0; i < STREAMS; ++i) copy_bytes<kBytes>(to + (j * STREAMS + i) * kThreads * kBytes, p[i] + j * step[i]);
#pragma unroll
        for (int i = 0; i < STREAMS; ++i) p[i] += BATCH * step[i];
        ahead -= BATCH;
        to += kSlot;
        copies_commit();
    }
    __device__ __forceinline__ int take(Vec<T, V> (&v)[STREAMS][BATCH]) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int i = 0; i < STREAMS; ++i) v[i][j].load(reinterpret_cast<const T*>(at + (j * STREAMS + i) * kThreads * kBytes));
        at += kSlot;
        const int got = min(left, BATCH);
        left -= BATCH;
        return got;
    }
    __device__ __forceinline__ int next(Vec<T, V> (&v)[STREAMS][BATCH]) {
        if (left <= 0) return 0;
        copies_wait<kHeldDepth - 1>();
        const int got = take(v);
        fetch();
        return got;
    }
    // once more from the first position
    __device__ __forceinline__ void rewind(int n, char* smem) {
        left = n;
        at = smem + threadIdx.x * kBytes;
    }
    __device__ __forceinline__ int again(Vec<T, V> (&v)[STREAMS][BATCH]) { return left <= 0 ? 0 : take(v); }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Another block's copy of a shared variable.
__device__ __forceinline__ float2 of_block(const float2* p, unsigned rank) {
    unsigned a;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((unsigned)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// Blocks of a launch: x the cluster's blocks (ranks), y the sets, z the samples.
template <int V>
__device__ __forceinline__ Place held_place(const GroupNorm& A) {
    Place p;
    p.vecs = A.set / V;
    p.lanes = kThreads / p.vecs;
    p.lane = (int)threadIdx.x / p.vecs;
    p.vec = (int)threadIdx.x - p.lane * p.vecs;
    p.on = p.lane < p.lanes;
    p.c = (int)blockIdx.y * A.set + p.vec * V;
    p.b = A.b0 + blockIdx.z;
    const int64_t r0 = (int64_t)blockIdx.x * A.chunk_rows;
    const int rows = (int)max((int64_t)0, min(A.S - r0, A.chunk_rows));
    p.first = r0 + p.lane;
    p.n = p.on && p.lane < rows ? (rows - p.lane + p.lanes - 1) / p.lanes : 0;
    return p;
}

// Bound by latency: 256 positions of 512 channels, bf16, 6.5 us in a graph.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_held(GroupNorm A) {
    extern __shared__ uint4 smem[];
    constexpr bool kFast = sizeof(T) == 2;
    // behind the slots: the lanes' numbers, the channels', the groups'
    char* const slots = reinterpret_cast<char*>(smem);
    float *const sm = reinterpret_cast<float*>(slots + A.slot_bytes), *const sq = sm + kThreads * V;
    float2 *const mine = reinterpret_cast<float2*>(sq + kThreads * V), *const stat = mine + A.set / A.Cg;
    __shared__ int sn[kThreads];
    const Place p = held_place<V>(A);
    const int groups = A.set / A.Cg, ranks = gridDim.x;
    float mean[V], sqr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] = sqr[i] = 0.f;
    int n = p.n;
    Held<T, V, 1, kRows> in;
    Vec<T, V> v[1][kRows];
    if (n) {
        in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
        in.step[0] = p.lanes * A.xr;
        in.begin(n, slots);
        Sums<T, V> sums;
        int got = in.next(v);
        sums.begin(v[0], got);
        do {
            sums.add(v[0], got);
            got = in.next(v);
        } while (got);
        sums.end(n, mean, sqr);
    }
    join_lanes<V>(p, n, mean, sqr, sn, sm, sq);
    // channels of this block, then its groups: a warp for each
    if (p.lane == 0)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm[p.vec * V + i] = mean[i];
            sq[p.vec * V + i] = sqr[i];
        }
    __syncthreads();
    join_channels(A, sm, sq, rows_of(A, blockIdx.x), groups, mine);
    if (ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int g = threadIdx.x; g < groups; g += kThreads) {
        const float count = (float)A.S * (float)A.Cg;
        float s = 0.f, q = 0.f;
        for (int k = 0; k < ranks; ++k) s = fmaf(ranks > 1 ? of_block(mine + g, k).x : mine[g].x, rows_of(A, k) / (float)A.S, s);
        for (int k = 0; k < ranks; ++k) {
            const float2 o = ranks > 1 ? of_block(mine + g, k) : mine[g];
            const float d = o.x - s;
            if (rows_of(A, k) > 0.f) q += fmaf(d * d, rows_of(A, k) * (float)A.Cg, o.y);
        }
        const float rstd = 1.f / sqrtf(q / count + A.eps);
        stat[g] = make_float2(s, rstd);
        if (blockIdx.x == 0) {
            const int64_t at = p.b * A.G + (int64_t)blockIdx.y * groups + g;
            if (A.mean_out) A.mean_out[at] = s;
            if (A.rstd_out) A.rstd_out[at] = rstd;
        }
    }
    __syncthreads();
    if (ranks > 1) cluster_arrive();  // this block has read the others' numbers
    if (n && A.y) {
        float scale[V], bias[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 o = stat[(p.vec * V + i) / A.Cg];
            mean[i] = o.x;
            scale[i] = o.y * (A.w ? to_f32(static_cast<const T*>(A.w)[p.c + i]) : 1.f);
            bias[i] = A.b ? to_f32(static_cast<const T*>(A.b)[p.c + i]) : 0.f;
        }
        T* y = static_cast<T*>(A.y) + p.b * A.yb + p.first * A.yr + p.c;
        const int64_t step = p.lanes * A.yr;
        copies_wait<0>();
        in.rewind(n, slots);
        while (const int got = in.again(v)) {
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                if (j >= got) break;
                float u[V];
                v[0][j].values(u);
                sub_all(u, mean);
                fma_all(u, u, scale, bias);
                act_all<V, kFast>(u, A.act, A.alpha);
                Vec<T, V> out;
                out.set(u);
                out.store(y);
                y += step;
            }
        }
    }
    copies_wait<0>();
    if (ranks > 1) cluster_wait();  // the others have read this block's
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 2) gn_bwd_held(GroupNorm A) {
    extern __shared__ uint4 smem[];
    let_next_kernel_start();
    char* const slots = reinterpret_cast<char*>(smem);
    float *const sa = reinterpret_cast<float*>(slots + A.slot_bytes), *const sb = sa + kThreads * V;
    float2 *const mine = reinterpret_cast<float2*>(sb + kThreads * V), *const coef = mine + A.set;
    const Place p = held_place<V>(A);
    const int lane = threadIdx.x & 31, groups = A.set / A.Cg, ranks = gridDim.x, n = p.n;
    float a[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = q[i] = 0.f;
    Held<T, V, 2, kBwdRows> in;
    Vec<T, V> v[2][kBwdRows];
    Channels<T, V> ch;
    if (n) {
        in.p[0] = static_cast<const T*>(A.x) + p.b * A.xb + p.first * A.xr + p.c;
        in.p[1] = static_cast<const T*>(A.dy) + p.b * A.db_ + p.first * A.dr + p.c;
        in.step[0] = p.lanes * A.xr;
        in.step[1] = p.lanes * A.dr;
        in.begin(n, slots);
        ch.load(A, p.b, p.c);
        while (const int got = in.next(v)) {
#pragma unroll
            for (int j = 0; j < kBwdRows; ++j) {
                if (j >= got) break;
                float d[V], du[V];
                centred_and_du<T, V>(A, ch, v[0][j], v[1][j], d, du);
                add_all(a, du);
                fma_all(q, du, d, q);
            }
        }
    }
    join_lanes_sums<V>(p, a, q, sa, sb);
    if (p.lane == 0)
#pragma unroll
        for (int i = 0; i < V; ++i) mine[p.vec * V + i] = make_float2(a[i], q[i]);
    if (ranks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // a warp for each group: its channels' sums over the blocks, in order
    for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
        const int64_t at = p.b * A.G + (int64_t)blockIdx.y * groups + g;
        const float rstd = A.rstd[at];
        float s1 = 0.f, s2 = 0.f;
        for (int c = lane; c < A.Cg; c += 32) {
            float2 t = make_float2(0.f, 0.f);
            for (int k = 0; k < ranks; ++k) {
                const float2 o = ranks > 1 ? of_block(mine + g * A.Cg + c, k) : mine[g * A.Cg + c];
                t.x += o.x;
                t.y += o.y;
            }
            t.y *= rstd;
            const int channel = (int)blockIdx.y * A.set + g * A.Cg + c;
            if (blockIdx.x == 0) A.sums[p.b * A.C + channel] = t;
            const float w = A.w ? to_f32(static_cast<const T*>(A.w)[channel]) : 1.f;
            s1 = fmaf(t.x, w, s1);
            s2 = fmaf(t.y, w, s2);
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        const float inv = 1.f / ((float)A.S * (float)A.Cg);
        if (lane == 0) coef[g] = make_float2(-s1 * inv * rstd, -s2 * inv * rstd * rstd);
    }
    __syncthreads();
    if (ranks > 1) cluster_arrive();
    if (n && A.y) {
        float m1[V], m2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 o = coef[(p.vec * V + i) / A.Cg];
            m1[i] = o.x;
            m2[i] = o.y;
        }
        T* dx = static_cast<T*>(A.y) + p.b * A.yb + p.first * A.yr + p.c;
        const int64_t step = p.lanes * A.yr;
        copies_wait<0>();
        in.rewind(n, slots);
        while (const int got = in.again(v)) {
#pragma unroll
            for (int j = 0; j < kBwdRows; ++j) {
                if (j >= got) break;
                float d[V], du[V];
                centred_and_du<T, V>(A, ch, v[0][j], v[1][j], d, du);
                fma_all(d, d, m2, m1);
                fma_all(du, du, ch.scale, d);
                Vec<T, V> out;
                out.set(du);
                out.store(dx);
                dx += step;
            }
        }
    }
    copies_wait<0>();
    if (ranks > 1) cluster_wait();
}

// ---- host -------------------------------------------------------------------

// Samples whose statistics and application run one after the other: what two
// passes read of them should stay in the 129 MB of L2.
constexpr int64_t kRangeBytes = 64ll << 20;

// One pass: channels of a set, blocks of a cluster, positions of a block.  Taken
// where all blocks are resident at once: with more of them the phases of a block
// (load, join, write) leave memory idle, and two passes are faster.  Graphs of
// calls, cold, us, one pass / two: 256 positions of 512 channels bf16 6.5 / 7.2, 4
// x 1024 of 512 8.6 / 10.5, 3 x 3363 of 210 fp32 15 / 19; not taken: 16 x 1024 of
// 512 20 / 17, 16 x 4096 of 256 30 / 22, its gradient 56 / 34.  One launch, too,
// instead of three, which a host feels first.
struct HeldPlan {
    int set = 0, ranks = 0, bytes = 0, slot_bytes = 0;
    int64_t rows = 0;
};
HeldPlan held_plan(int64_t B, int64_t S, int64_t C, int64_t Cg, int V, int eb, bool backward, int sm) {
    HeldPlan best;
    if (S == 0 || C % V) return best;
    // whole groups and whole vectors
    int64_t unit = Cg;
    while (unit % V) unit += Cg;
    if (C % unit || unit / V > kThreads || C / unit > 65535) return best;
    int64_t set = unit;
    // 64 bytes of a row where there are blocks enough: whole sectors, two of them
    while (set * eb < 64 && C % (2 * set) == 0 && 2 * set / V <= kThreads && B * (C / (2 * set)) >= sm) set *= 2;
    const int streams = backward ? 2 : 1, batch = backward ? kBwdRows : kRows;
    const int64_t lanes = kThreads / (set / V), clusters = B * (C / set);
    const int64_t extra = 2 * kThreads * V * 4 + (backward ? set : set / Cg) * 8 + set / Cg * 8;
    for (int ranks = 1; ranks <= 8; ranks *= 2) {
        const int64_t rows = (S + ranks - 1) / ranks, each = (rows + lanes - 1) / lanes;
        const int64_t slots = (each + batch - 1) / batch * batch * streams * kThreads * V * eb, bytes = slots + extra;
        if (bytes > kHeldBytes || clusters * ranks > (bytes > kHeldBytes / 2 ? sm : 2 * sm)) continue;
        best.set = (int)set;
        best.ranks = ranks;
        best.rows = rows;
        best.slot_bytes = (int)slots;
        best.bytes = (int)bytes;
        if (clusters * ranks >= sm || each <= 2 * batch) break;  // as few positions as are worth a block
    }
    return best;
}
// Vectors that a tensor of these channels may have: 16 bytes, two elements, one.
bool held_always(int64_t B, int64_t S, int64_t C, int64_t G, int dtype, bool backward, int sm) {
    const int eb = dtype == CT_F32 ? 4 : 2;
    for (const int V : {16 / eb, 2, 1})
        if (C % V == 0 && !held_plan(B, S, C, C / G, V, eb, backward, sm).ranks) return false;
    return true;
}

struct Plan {
    int64_t range;  // samples of a launch
    int chunks;
    int64_t chunk_rows;
    size_t part, stats, gpart, bytes;
};

Plan plan(int64_t B, int64_t S, int64_t C, int64_t G, int dtype, int backward, int sm) {
    Plan p;
    const int64_t sample = std::max<int64_t>(1, S * C * (dtype == CT_F32 ? 4 : 2) * (backward ? 2 : 1));
    // a grid's z has 65535 at most, the join's x (a block for each group) 2^31 - 1
    p.range = std::min<int64_t>({std::max<int64_t>(1, kRangeBytes / sample), std::max<int64_t>(B, 1), 32768, 2147483647 / G});
    // what is resident at once, at least 16 positions a chunk
    const int64_t want = std::max<int64_t>(1, (backward ? kBwdBlocks : kBlocks) * sm / p.range);
    const int64_t most = (S + 15) / 16;
    int64_t chunks = std::max<int64_t>(1, std::min(want, most));
    p.chunk_rows = std::max<int64_t>(1, (S + chunks - 1) / chunks);
    p.chunks = (int)((S + p.chunk_rows - 1) / p.chunk_rows);
    p.part = ((size_t)B * p.chunks * C * sizeof(float2) + 255) / 256 * 256;
    p.stats = ((size_t)B * G * sizeof(float2) + 255) / 256 * 256;
    // one pass needs room for the channels' sums alone
    if (held_always(B, S, C, G, dtype, backward != 0, sm)) p.part = p.stats = 0;
    p.gpart = p.part ? ((size_t)B * p.chunks * G * sizeof(float2) + 255) / 256 * 256 : 0;
    p.bytes = p.part + p.stats + p.gpart + (backward ? ((size_t)B * C * sizeof(float2) + 255) / 256 * 256 : 0);
    return p;
}

template <typename T, int V>
bool fits(const void* p, int64_t batch, int64_t row) {
    return !p || ((uintptr_t)p % (V * sizeof(T)) == 0 && batch % V == 0 && row % V == 0);
}

// Dynamic shared memory that needs no attribute: 48 KB with the kernels' own variables.
constexpr int kPlainBytes = 40 << 10;

template <typename K, typename... More>
cudaError_t launch(K k, dim3 grid, int threads, int bytes, bool follows, const GroupNorm& A, cudaStream_t s, More... more) {
    if (bytes > kPlainBytes) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, A, more...);
}

template <typename T>
cudaError_t join(const GroupNorm& A, int64_t samples, bool backward, cudaStream_t s) {
    const dim3 blocks((unsigned)(samples * A.G));
    if (A.grouped) {
        const dim3 warps((unsigned)((samples * A.G + kThreads / 32 - 1) / (kThreads / 32)));
        return launch(backward ? gn_bwd_join_groups : gn_join_groups, warps, kThreads, 0, true, A, s, (int64_t)(samples * A.G));
    }
    // a warp for up to four numbers a lane, a large block for a thousand and more
    const int64_t items = (int64_t)A.chunks * A.Cg;
    if (backward)
        return items <= 128    ? launch(gn_bwd_join<T, 32>, blocks, 32, 0, true, A, s)
               : items <= 1024 ? launch(gn_bwd_join<T, 256>, blocks, 256, 0, true, A, s)
                               : launch(gn_bwd_join<T, 1024>, blocks, 1024, 0, true, A, s);
    return items <= 128    ? launch(gn_join<32>, blocks, 32, 0, true, A, s)
           : items <= 1024 ? launch(gn_join<256>, blocks, 256, 0, true, A, s)
                           : launch(gn_join<1024>, blocks, 1024, 0, true, A, s);
}

template <typename K>
cudaError_t launch_held(K k, const HeldPlan& h, GroupNorm A, cudaStream_t s) {
    if (h.bytes > kPlainBytes) {
        // the same for every size: the attribute is the kernel's, and another thread's smaller call
        // may set it between this one's two steps
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldBytes);
        if (e != cudaSuccess) return e;
    }
    A.set = h.set;
    A.slot_bytes = h.slot_bytes;
    A.chunk_rows = h.rows;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)h.bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)h.ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = h.ranks > 1 ? 1 : 0;
    for (A.b0 = 0; A.b0 < A.B; A.b0 += 32768) {
        cfg.gridDim = dim3((unsigned)h.ranks, (unsigned)(A.C / h.set), (unsigned)std::min<int64_t>(32768, A.B - A.b0));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, k, A);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Whether the first pass's blocks join their channels: those of a group that has
// thousands of numbers from them otherwise.  Cold, us, joined there / between the
// passes: 40000 positions of 512 channels in one group 25 / 100, 2 x 30000 of 320 in
// 8 groups 24 / 26, the gradient 50 / 53; not so joined: 2 x 262144 of 64 in 32 groups
// 39 / 36, the gradient 77 / 68.
bool joins_itself(const GroupNorm& A, int tiles) { return tiles == 1 && (int64_t)A.chunks * A.Cg > 2048; }

template <typename T, int V>
cudaError_t forward_v(GroupNorm A, int64_t range, int sm, cudaStream_t s) {
    const int tiles = (A.C / V + kTile - 1) / kTile;
    constexpr int ring = Stream<T, V, 1, kRows, kDepth>::kBytes, tree = 2 * kThreads * V * 4;
    const HeldPlan h = held_plan(A.B, A.S, A.C, A.Cg, V, sizeof(T), false, sm);
    if (h.ranks) return launch_held(gn_held<T, V>, h, A, s);
    A.grouped = A.S && joins_itself(A, tiles);
    for (A.b0 = 0; A.b0 < A.B; A.b0 += range) {
        const int64_t n = std::min(range, A.B - A.b0);
        const dim3 grid(A.chunks, tiles, (unsigned)n);
        cudaError_t e = cudaSuccess;
        if (A.S) e = launch(gn_stats<T, V>, grid, kThreads, std::max(ring, tree), false, A, s);
        if (e == cudaSuccess) e = join<T>(A, n, false, s);
        if (e == cudaSuccess && A.S && A.y) e = launch(gn_apply<T, V>, grid, kThreads, ring, true, A, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t forward(const GroupNorm& A, int64_t range, int sm, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T), N = 2;
    if (A.C % W == 0 && fits<T, W>(A.x, A.xb, A.xr) && fits<T, W>(A.y, A.yb, A.yr)) return forward_v<T, W>(A, range, sm, s);
    if (A.C % N == 0 && fits<T, N>(A.x, A.xb, A.xr) && fits<T, N>(A.y, A.yb, A.yr)) return forward_v<T, N>(A, range, sm, s);
    return forward_v<T, 1>(A, range, sm, s);
}

template <typename T, int V>
cudaError_t backward_v(GroupNorm A, int64_t range, int sm, cudaStream_t s) {
    const int tiles = (A.C / V + kTile - 1) / kTile;
    constexpr int ring = Stream<T, V, 2, kBwdRows, kDepth>::kBytes, tree = 2 * kThreads * V * 4;
    cudaError_t e = cudaSuccess;
    const HeldPlan h = held_plan(A.B, A.S, A.C, A.Cg, V, sizeof(T), true, sm);
    if (h.ranks) e = launch_held(gn_bwd_held<T, V>, h, A, s);
    A.grouped = A.S && !h.ranks && joins_itself(A, tiles);
    if (A.S && !h.ranks)
        for (A.b0 = 0; A.b0 < A.B && e == cudaSuccess; A.b0 += range) {
            const int64_t n = std::min(range, A.B - A.b0);
            const dim3 grid(A.chunks, tiles, (unsigned)n);
            e = launch(gn_bwd_sums<T, V>, grid, kThreads, std::max(ring, tree), false, A, s);
            if (e == cudaSuccess) e = join<T>(A, n, true, s);
            if (e == cudaSuccess && A.y) e = launch(gn_bwd_apply<T, V>, grid, kThreads, ring, true, A, s);
        }
    A.early = A.S && A.B && !h.ranks && A.y;
    if (e == cudaSuccess && (A.dw || A.db)) e = launch(gn_bwd_channels<T>, dim3((A.C + 31) / 32), 1024, 0, A.S && A.B, A, s);
    return e;
}

template <typename T>
cudaError_t backward(const GroupNorm& A, int64_t range, int sm, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T), N = 2;
    if (A.C % W == 0 && fits<T, W>(A.x, A.xb, A.xr) && fits<T, W>(A.y, A.yb, A.yr) && fits<T, W>(A.dy, A.db_, A.dr))
        return backward_v<T, W>(A, range, sm, s);
    if (A.C % N == 0 && fits<T, N>(A.x, A.xb, A.xr) && fits<T, N>(A.y, A.yb, A.yr) && fits<T, N>(A.dy, A.db_, A.dr))
        return backward_v<T, N>(A, range, sm, s);
    return backward_v<T, 1>(A, range, sm, s);
}

bool bad_ptr(const void* p, size_t a) { return p && (uintptr_t)p % a != 0; }

int check_problem(int64_t B, int64_t S, int64_t C, int64_t G, int dtype) {
    if (dtype != CT_F32 && dtype != CT_F16 && dtype != CT_BF16)
        return report_error(CT_ERR_DTYPE, "dtype %d is not a supported floating type (CT_F32, CT_F16, CT_BF16)", dtype);
    if (B < 0 || S < 0 || C < 1)
        return report_error(CT_ERR_SHAPE, "B and S must be >= 0 and C >= 1 (got %lld, %lld, %lld)", (long long)B, (long long)S, (long long)C);
    if (C > 65536 || S > 2147483647ll || B > 65535) return report_error(CT_ERR_TOO_LARGE, "C <= 65536, S < 2^31 and B <= 65535 supported");
    if (G < 1 || C % G) return report_error(CT_ERR_GROUPS, "groups must divide the %lld channels (got %lld)", (long long)C, (long long)G);
    return CT_OK;
}

int check_activation(int activation) {
    if (activation < CT_ACT_NONE || activation > CT_ACT_SIGMOID)
        return report_error(CT_ERR_PARAM, "activation %d is not a ct_activation", activation);
    return CT_OK;
}

// The call's workspace: the caller's, or one allocated on the stream.
struct Workspace {
    void* p = nullptr;
    bool owned = false;
    int take(void* given, size_t bytes, size_t need, cudaStream_t s) {
        if (need == 0) return CT_OK;
        if (given) {
            if (bytes < need) return report_error(CT_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", bytes, need);
            if (bad_ptr(given, 256)) return report_error(CT_ERR_ALIGN, "workspace must be 256-byte aligned");
            p = given;
        } else {
            const cudaError_t e = cudaMallocAsync(&p, need, s);
            if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "cudaMallocAsync(workspace): %s", cudaGetErrorString(e));
            owned = true;
        }
        return CT_OK;
    }
    cudaError_t give(cudaError_t e, cudaStream_t s) {
        if (!owned) return e;
        const cudaError_t f = cudaFreeAsync(p, s);
        return e == cudaSuccess ? f : e;
    }
};

int sm_count() {
    DeviceInfo d;
    return device_info(&d) == cudaSuccess ? d.sm_count : 152;
}

}  // namespace
}  // namespace ct

using namespace ct;

extern "C" int ct_group_norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t groups, int dtype, int backward, size_t* bytes) {
    if (!bytes) return report_error(CT_ERR_NULL, "bytes is NULL");
    const int rc = check_problem(B, S, C, groups, dtype);
    if (rc != CT_OK) return rc;
    *bytes = plan(B, S, C, groups, dtype, backward, sm_count()).bytes;
    return CT_OK;
}

extern "C" int ct_group_norm_forward(const void* x, const int64_t* x_strides, const void* weight, const void* bias, void* y,
                                     const int64_t* y_strides, float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                                     int64_t B, int64_t S, int64_t C, int64_t groups, float eps, int activation, float alpha,
                                     int dtype, void* stream) {
    int rc = check_problem(B, S, C, groups, dtype);
    if (rc == CT_OK) rc = check_activation(activation);
    if (rc != CT_OK) return rc;
    if (!(eps >= 0.f)) return report_error(CT_ERR_PARAM, "eps must be >= 0");
    if (B == 0 || (!y && !mean && !rstd)) return CT_OK;
    if (S > 0 && (!x || !x_strides || (y && !y_strides))) return report_error(CT_ERR_NULL, "x and the strides must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(x, eb) || bad_ptr(weight, eb) || bad_ptr(bias, eb) || bad_ptr(y, eb) || bad_ptr(mean, 4) || bad_ptr(rstd, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    const int sm = sm_count();
    const Plan p = plan(B, S, C, groups, dtype, 0, sm);
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    if ((rc = ws.take(workspace, workspace_bytes, p.bytes, s)) != CT_OK) return rc;
    float* stats = p.stats ? reinterpret_cast<float*>(static_cast<char*>(ws.p) + p.part) : nullptr;
    GroupNorm A{};
    A.x = x; A.w = weight; A.b = bias; A.y = y;
    A.mean_out = mean ? mean : stats;
    A.rstd_out = rstd ? rstd : stats ? stats + B * groups : nullptr;
    A.mean = A.mean_out; A.rstd = A.rstd_out;
    A.part = static_cast<float2*>(ws.p);
    A.gpart = reinterpret_cast<float2*>(static_cast<char*>(ws.p) + p.part + p.stats);
    if (S > 0) { A.xb = x_strides[0]; A.xr = x_strides[1]; }
    if (S > 0 && y) { A.yb = y_strides[0]; A.yr = y_strides[1]; }
    A.B = B; A.S = S; A.C = (int)C; A.G = (int)groups; A.Cg = (int)(C / groups); A.by_cg = divider((unsigned)A.Cg);
    A.chunks = p.chunks; A.chunk_rows = p.chunk_rows; A.act = activation; A.eps = eps; A.alpha = alpha;
    cudaError_t e = dtype == CT_F32 ? forward<float>(A, p.range, sm, s) : dtype == CT_F16 ? forward<__half>(A, p.range, sm, s)
                                                                                      : forward<__nv_bfloat16>(A, p.range, sm, s);
    e = ws.give(e, s);
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "group norm: %s", cudaGetErrorString(e));
    return CT_OK;
}

extern "C" int ct_group_norm_backward(const void* dy, const int64_t* dy_strides, const void* x, const int64_t* x_strides,
                                      const float* mean, const float* rstd, const void* weight, const void* bias, void* dx,
                                      const int64_t* dx_strides, void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                      int64_t B, int64_t S, int64_t C, int64_t groups, int activation, float alpha, int dtype,
                                      void* stream) {
    int rc = check_problem(B, S, C, groups, dtype);
    if (rc == CT_OK) rc = check_activation(activation);
    if (rc != CT_OK) return rc;
    const bool any = B > 0 && S > 0;
    if ((!dx || !any) && !dweight && !dbias) return CT_OK;
    if (any && (!dy || !dy_strides || !x || !x_strides || !mean || !rstd || (dx && !dx_strides)))
        return report_error(CT_ERR_NULL, "dy, x, mean, rstd and the strides must not be NULL");
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(dy, eb) || bad_ptr(x, eb) || bad_ptr(weight, eb) || bad_ptr(bias, eb) || bad_ptr(dx, eb) || bad_ptr(dweight, eb) ||
        bad_ptr(dbias, eb) || bad_ptr(mean, 4) || bad_ptr(rstd, 4))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    const int sm = sm_count();
    const Plan p = plan(B, S, C, groups, dtype, 1, sm);
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    if (any && (rc = ws.take(workspace, workspace_bytes, p.bytes, s)) != CT_OK) return rc;
    GroupNorm A{};
    A.x = x; A.dy = dy; A.w = weight; A.b = bias; A.y = dx; A.dw = dweight; A.db = dbias;
    A.mean = mean; A.rstd = rstd;
    A.part = static_cast<float2*>(ws.p);
    A.coef = any ? reinterpret_cast<float2*>(static_cast<char*>(ws.p) + p.part) : nullptr;
    A.gpart = any ? reinterpret_cast<float2*>(static_cast<char*>(ws.p) + p.part + p.stats) : nullptr;
    A.sums = any ? reinterpret_cast<float2*>(static_cast<char*>(ws.p) + p.part + p.stats + p.gpart) : nullptr;
    if (any) {
        A.xb = x_strides[0]; A.xr = x_strides[1];
        A.db_ = dy_strides[0]; A.dr = dy_strides[1];
        if (dx) { A.yb = dx_strides[0]; A.yr = dx_strides[1]; }
    }
    A.B = B; A.S = S; A.C = (int)C; A.G = (int)groups; A.Cg = (int)(C / groups); A.by_cg = divider((unsigned)A.Cg);
    A.chunks = p.chunks; A.chunk_rows = p.chunk_rows; A.act = activation; A.alpha = alpha;
    cudaError_t e = dtype == CT_F32 ? backward<float>(A, p.range, sm, s) : dtype == CT_F16 ? backward<__half>(A, p.range, sm, s)
                                                                                       : backward<__nv_bfloat16>(A, p.range, sm, s);
    e = ws.give(e, s);
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "group norm backward: %s", cudaGetErrorString(e));
    return CT_OK;
}
