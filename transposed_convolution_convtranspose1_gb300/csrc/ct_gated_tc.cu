// ct_gated_tc.cu -- the products of the gated projection and its gradients on
// the tensor cores (tcgen05, TMEM, TMA).
//
//   forward        g = x Wg, u = x Wu side by side in TMEM; y = act(g) * u
//   gradients, 1   g and u again; dg = dy * u * act'(g), du = dy * act(g)
//   gradients, 2   dx = dg Wg^T + du Wu^T; dWg = x^T dg, dWu = x^T du
//
// One persistent kernel for all of them: a producer warp for each operand (TMA
// into a ring of stages), a warp that issues the MMAs, eight warps that take the
// results out of TMEM.  Two accumulators of 256 columns each fill TMEM: while the
// eight warps work on one tile the MMAs of the next run.
//
// A tile is 128 x 256 accumulator columns on one SM, or 256 x 256 on a pair of
// SMs (cta_group::2: each SM keeps its own 128 rows of A and half of B, which
// halves what B costs in shared memory).  For g and u the 256 columns are 128
// of each, so that a thread of the epilogue has both in its row; on a pair one
// SM holds the gate's half of B and the other the up's.
//
// Where there are fewer tiles than SMs K is split too: each piece writes its fp32
// sums, and gated_join adds them in order and finishes the work.
//
// Operands are read as they lie: K-major (K dense) or MN-major (rows or columns
// dense), both with a 128-byte swizzle, so that x, the weights and the
// transposed products need no transposed copies.  An fp32 result is a sum over
// six products of bf16 parts (ct_gated.cu), taken out of TMEM every other block of
// K and added up in registers.
//
// Bound by shared-memory bandwidth: a block of K (64) writes 32 KB into an SM's
// shared memory and its MMAs read about 48 KB of it, some 640 cycles at 128 bytes
// a cycle, where the MMAs themselves take 512; the tensor pipe is active 81% of
// the cycles.  16384 x 1024 x 4096 bf16 with silu, back to back for a second, where the
// power limit lowers the clock: 174 us, 1580 TFLOP/s, 82% of the measured product rate
// (91% of the sustained one); the first calls after a pause: 151 us, 94%.  Its
// gradients: 555 us, 77% (85%); 475 us after a pause.  A wait on a
// barrier takes an issuing warp 100 cycles, a copy 110, an expected count 65: one
// producer warp for both operands was slower than the MMAs (650 cycles a block,
// 190 us), one for each is not.
#include <algorithm>

#include "ct_gated.h"
#include "ct_internal.h"
#include "ct_rows.cuh"
#include "ct_settle.h"
#include "ct_tcgen05.cuh"

namespace ct {
namespace {

using namespace rows;
using namespace tcg;

constexpr int kEpiWarps = 8;
constexpr int kThreads = 96 + 32 * kEpiWarps;
constexpr uint32_t kBlock = 128 * 128;                       // 128 rows of 128 bytes
constexpr uint32_t kSlab = 32 * 128;                         // 32 rows of 128 bytes: a warp's piece of dy, or of a result off 16-byte boundaries
constexpr uint32_t kSlabs = kEpiWarps * kSlab;
constexpr int kMaxStages = 6;

struct GemmParams {
    CUtensorMap a[6], b[6], dy;
    int a_part[12], b_part[12];
    int parts, b_block, a_z, b_z;
    int a_mn, b_mn;
    int a_whole, b_whole;      // MN-major, a multiple of 64 wide: maps of [n / 64][k][64]
    int nk, chunk;             // blocks of 64 along K of a part; of them in a sum that leaves TMEM
    int m_tiles, n_tiles, tiles, strip;
    int splits;                // pieces of K
    float* part;               // [z][piece][sum][M][pitch], pieces > 1
    int64_t pitch;
    int M, N;
    int act;
    float alpha;
    void* out[2];
    int64_t out_stride[2];
    int aligned;               // of the results: 32, 16 or 0 bytes
    int early;                 // starts beside the kernel before it
    int head_groups, head_tiles;  // the first SMs (pairs) have this many tiles to themselves
    uint32_t idesc;
    uint64_t wait_ns;
};

// Shared-memory matrix descriptor: MN-major, 128-byte swizzle: rows of 64
// MN elements (128 bytes) per K index, 8-row groups 1024 bytes apart along K
// (SBO), 64-element MN blocks 8192 bytes apart (LBO), descriptor version 1.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);       // start address
    d |= (uint64_t)(8192u >> 4) << 16;             // leading byte offset: next 64 MN elements
    d |= (uint64_t)(1024u >> 4) << 32;             // stride byte offset: next 8 K rows
    d |= (uint64_t)1 << 46;                        // version
    d |= (uint64_t)2 << 61;                        // SWIZZLE_128B
    return d;
}

template <int CG>
struct Layout {
    static constexpr uint32_t kStage = CG == 2 ? 2 * kBlock : 3 * kBlock;  // A, B (half of it on each SM of a pair)
    static constexpr int kStages = CG == 2 ? 6 : 4;
    static constexpr uint32_t kBytes = kStages * kStage + kSlabs + 1024;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of the first SM's copy of a shared variable.
__device__ __forceinline__ uint32_t at_first(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Into the other SM's copy of a shared variable.
__device__ __forceinline__ void put_other(uint32_t addr, uint32_t other, uint32_t v) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(addr), "r"(other), "r"(v) : "memory");
}
// Bytes that were announced and will not land.
__device__ __forceinline__ void complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Copies, MMAs and commits are issued by one elected lane of a converged warp.
#define CT_ELECTED "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q "
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
    if constexpr (CG == 2)
        asm volatile(CT_ELECTED
                     "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
                     : "memory");
    else
        asm volatile(CT_ELECTED
                     "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
                     : "memory");
}
// Both 64-wide halves of an MN-major block at once: coordinates (0, k, n / 64).
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c1, int c2) {
    if constexpr (CG == 2)
        asm volatile(CT_ELECTED
                     "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(bar)
                     : "memory");
    else
        asm volatile(CT_ELECTED
                     "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(bar)
                     : "memory");
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile(CT_ELECTED "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes) : "memory");
}
// The four MMAs of a block of K (64: 16 each) and the commit that frees its stage
// on both SMs of a pair; one elected lane for all of them.  A and B advance by
// `as` and `bs` (in descriptor units) an MMA.
template <int CG>
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint64_t as, uint64_t bs, uint32_t idesc, uint32_t accumulate,
                                          uint32_t bar) {
#define CT_MMA(GROUP, P) "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], a, b, %5, " P ";\n\t"
#define CT_NEXT "add.s64 a, a, %3;\n\tadd.s64 b, b, %4;\n\t"
#define CT_BLOCK(GROUP, COMMIT)                                                                                            \
    asm volatile(                                                                                                          \
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t.reg .b16 m;\n\t"                                                 \
        "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\tmov.b16 m, 3;\n\tmov.b64 a, %1;\n\tmov.b64 b, %2;\n\t"           \
        "elect.sync _|q, 0xffffffff;\n\t" CT_MMA(GROUP, "p") CT_NEXT CT_MMA(GROUP, "t") CT_NEXT CT_MMA(GROUP, "t") CT_NEXT \
            CT_MMA(GROUP, "t") "@q tcgen05.commit.cta_group::" GROUP ".mbarrier::arrive::one.shared::cluster" COMMIT        \
        ";\n\t}" ::"r"(d),                                                                                                 \
        "l"(a), "l"(b), "l"(as), "l"(bs), "r"(idesc), "r"(accumulate), "r"(bar)                                            \
        : "memory")
    if constexpr (CG == 2) CT_BLOCK("2", ".multicast::cluster.b64 [%7], m");
    else CT_BLOCK("1", ".b64 [%7]");
#undef CT_BLOCK
#undef CT_NEXT
#undef CT_MMA
}
// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Arrives on `bar` when every MMA issued so far is done; on both SMs of a pair.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\t"
            "mov.b16 m, 3;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "elect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void arrive_first(uint32_t bar) {
    if constexpr (CG == 2)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_first(bar)) : "memory");
    else
        mbar_arrive(bar);
}

struct Tile {
    int m, n, z;       // rows from m, columns from n (in 128s: g and u; in 256s: a product)
    int piece, k0, k1; // blocks of K
};
// The i-th tile of a group of SMs (one, or a pair): tiles go round, but the first
// head_groups start head_tiles rounds before the others.
__device__ __forceinline__ int tile_number(const GemmParams& P, int group, int groups, int i) {
    const int head = P.head_tiles;
    if (group < P.head_groups) return i < head ? i * P.head_groups + group : head * P.head_groups + (i - head) * groups + group;
    return head * P.head_groups + i * groups + group;
}
template <int CG, int KIND>
__device__ __forceinline__ Tile tile_at(const GemmParams& P, int t) {
    Tile r;
    const int zp = t / (P.m_tiles * P.n_tiles);
    t -= zp * P.m_tiles * P.n_tiles;
    r.z = zp / P.splits;
    r.piece = zp - r.z * P.splits;
    r.k0 = (int)((int64_t)r.piece * P.nk / P.splits);
    r.k1 = (int)((int64_t)(r.piece + 1) * P.nk / P.splits);
    const int strip = t / (P.strip * P.n_tiles), m0 = strip * P.strip, height = min(P.strip, P.m_tiles - m0);
    t -= strip * P.strip * P.n_tiles;
    r.n = t / height;
    r.m = (m0 + t - r.n * height) * (128 * CG);
    r.n *= KIND == kProduct ? 256 : 128;
    return r;
}

// 32 values of a row (16 bits: half of a slab's row, `part` 0 or 1; fp32: the
// whole row) into the swizzled slab.
template <typename T>
__device__ __forceinline__ void put_row(uint32_t slab, int lane, int part, const float (&v)[32]) {
    constexpr int V = 16 / (int)sizeof(T), N = 32 / V;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Vec<T, V> w;
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = v[i * V + j];
        w.set(e);
        const uint32_t at = slab + lane * 128 + (((sizeof(T) == 2 ? part * 4 : 0) + i) ^ (lane & 7)) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.w[0]), "r"(w.w[1]), "r"(w.w[2]), "r"(w.w[3]) : "memory");
    }
}
template <typename T>
__device__ __forceinline__ void get_row(uint32_t slab, int lane, int part, float (&v)[32]) {
    constexpr int V = 16 / (int)sizeof(T), N = 32 / V;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Vec<T, V> w;
        const uint32_t at = slab + lane * 128 + (((sizeof(T) == 2 ? part * 4 : 0) + i) ^ (lane & 7)) * 16;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.w[0]), "=r"(w.w[1]), "=r"(w.w[2]), "=r"(w.w[3]) : "r"(at) : "memory");
#pragma unroll
        for (int j = 0; j < V; ++j) v[i * V + j] = w.get(j);
    }
}

// 32 columns of a row straight from registers, 32 or 16 bytes a store (shared
// memory, which the MMAs' operands nearly fill the bandwidth of, is left alone);
// `n` of them exist.
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[32], int n, bool by32) {
    constexpr int V = 16 / (int)sizeof(T), N = 32 / V;
    Vec<T, V> w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = v[i * V + j];
        w[i].set(e);
    }
    if (n >= 32 && by32) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i * V), "r"(w[i].w[0]), "r"(w[i].w[1]),
                         "r"(w[i].w[2]), "r"(w[i].w[3]), "r"(w[i + 1].w[0]), "r"(w[i + 1].w[1]), "r"(w[i + 1].w[2]), "r"(w[i + 1].w[3])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (n >= (i + 1) * V) w[i].store(p + i * V);
            else
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (i * V + j < n) p[i * V + j] = from_f32<T>(v[i * V + j]);
        }
    }
}

// A slab to a result off 16-byte boundaries, row by row.
template <typename T>
__device__ __forceinline__ void send(const GemmParams& P, int which, const uint8_t* slab, int row, int col, int lane) {
    constexpr int kCols = 128 / (int)sizeof(T);
    __syncwarp();
    T* out = static_cast<T*>(P.out[which]);
    for (int r = 0; r < 32 && row + r < P.M; ++r)
#pragma unroll
        for (int c = lane; c < kCols; c += 32)
            if (col + c < P.N) {
                const uint32_t b = c * (uint32_t)sizeof(T);
                out[(int64_t)(row + r) * P.out_stride[which] + col + c] = *reinterpret_cast<const T*>(slab + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15));
            }
    __syncwarp();
}

// act(g) * u, or (dg, du) from dy, 32 values.
template <bool FAST>
__device__ __forceinline__ void gate(float (&g)[32], const float (&u)[32], int act, float alpha) {
    act_all<32, FAST>(g, act, alpha);
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] *= u[i];
}
template <bool FAST, int N>
__device__ __forceinline__ void gate_back(float (&g)[N], float (&u)[N], const float (&dy)[N], int act, float alpha) {
#define CT_ACT_CASE(A)                                        \
    case A:                                                   \
        _Pragma("unroll") for (int i = 0; i < N; ++i) {       \
            float f, slope;                                   \
            act_both<A, FAST>(g[i], alpha, f, slope);         \
            g[i] = dy[i] * u[i] * slope;                      \
            u[i] = dy[i] * f;                                 \
        }                                                     \
        break;
    switch (act) {
        CT_ACT_CASE(1) CT_ACT_CASE(2) CT_ACT_CASE(3) CT_ACT_CASE(4) CT_ACT_CASE(5) CT_ACT_CASE(6)
        default: CT_ACT_CASE(0)
    }
#undef CT_ACT_CASE
}

template <typename T, int CG, int KIND>
__global__ void __launch_bounds__(kThreads, 1) gated_gemm(const __grid_constant__ GemmParams P) {
    using L = Layout<CG>;
    constexpr bool kWide = sizeof(T) == 4, kFast = !kWide;
    constexpr int kK = 64;                       // elements of a block of K
    constexpr int kCols = 128 / (int)sizeof(T);  // columns of a slab
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], acc_full[2], acc_empty[2], dy_bar[kEpiWarps], done_bar;
    __shared__ uint32_t tmem_base_slot;
    __shared__ volatile int abort_flag;
    // uses of the ring that the producers of A and B issued; the other SM's, and whether it gave up
    __shared__ uint32_t sent[2], other_sent[2], other_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int group = (int)blockIdx.x / CG, groups = (int)gridDim.x / CG;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        other_abort = 0;
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 2);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), kEpiWarps * CG);
        }
        for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(&dy_bar[i]), 1);
        mbar_init(smem_u32(&done_bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_slot)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base_slot)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    // What the kernel before this one wrote (operands, parts that it still read) is there
    // from here on, and the next kernel of the call may take this one's place SM by SM.  An
    // early kernel reads nothing of the one before it, and what that one waited for has been
    // there since it let this one start: it waits at its end, so that whoever waits for this
    // kernel has waited for both.
    if (!P.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers: A, B
        const bool is_b = warp == 2;
        // on a pair both SMs' copies count on the first one's barriers
        const uint32_t full = smem_u32(&full_bar[0]), to = CG == 2 ? at_first(full) : full;
        const uint32_t at = ring + (is_b ? kBlock : 0);
        const bool mn = is_b ? P.b_mn : P.a_mn, whole = is_b ? P.b_whole : P.a_whole;
        const uint32_t bytes = CG * (is_b ? L::kStage - kBlock : kBlock);
        const uint32_t empty = smem_u32(&empty_bar[0]);
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true, ready = false;
        for (int i = 0, t; ok && (t = tile_number(P, group, groups, i)) < P.tiles; ++i) {
            const Tile tile = tile_at<CG, KIND>(P, t);
            for (int k0 = tile.k0, part = 0; k0 < tile.k1 && ok; part = part + 1 < P.parts ? part + 1 : (k0 += P.chunk, 0)) {
                // the 128 rows of A; of B 128 columns of 256, on one SM both
                const CUtensorMap* map[2];
                int x[2];
                if (is_b) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int j = CG == 2 ? (int)rank : i;
                        map[i] = &P.b[P.b_part[part] + tile.z * P.b_z + (KIND == kProduct ? 0 : j * P.b_block)];
                        x[i] = tile.n + (KIND == kProduct ? j * 128 : 0);
                    }
                } else {
                    map[0] = &P.a[P.a_part[part] + tile.z * P.a_z];
                    x[0] = tile.m + (int)rank * 128;
                    map[1] = map[0];
                    x[1] = x[0];
                }
                const int loads = is_b && CG == 1 ? 2 : 1;
                const int k1 = min(tile.k1, k0 + P.chunk) * kK;
                for (int k = k0 * kK; k < k1; k += kK) {
                    ok = issued < (uint32_t)L::kStages || (ready && P.wait_ns) ||
                         __all_sync(0xffffffffu, mbar_wait(empty + stage * 8, phase ^ 1, kErrProducer, &abort_flag, P.wait_ns));
                    if (!ok) break;
                    const uint32_t nxt = stage + 1 == L::kStages ? 0 : stage + 1;
                    const bool seen = mbar_test(empty + nxt * 8, nxt ? phase ^ 1 : phase);
                    const uint32_t bar = to + stage * 8, dst = at + stage * L::kStage;
                    if (rank == 0) expect(full + stage * 8, bytes);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == loads) break;
                        const uint32_t d = dst + i * kBlock;
                        if (!mn) {
                            load_2d<CG>(d, map[i], bar, k, x[i]);
                        } else if (whole) {
                            load_3d<CG>(d, map[i], bar, k, x[i] / kK);
                        } else {
                            load_2d<CG>(d, map[i], bar, x[i], k);
                            load_2d<CG>(d + kBlock / 2, map[i], bar, x[i] + kK, k);
                        }
                    }
                    ready = __all_sync(0xffffffffu, seen);
                    ++issued;
                    if (++stage == L::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        }
        if (lane == 0) sent[is_b] = issued;
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (rank == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, used = 0;
            bool ok = true, ready = false;
            const uint32_t full = smem_u32(&full_bar[0]), empty = smem_u32(&empty_bar[0]), idesc = P.idesc;
            const uint64_t a0 = P.a_mn ? smem_desc_mn_sw128(ring) : smem_desc_sw128(ring);
            const uint64_t b0 = P.b_mn ? smem_desc_mn_sw128(ring + kBlock) : smem_desc_sw128(ring + kBlock);
            // K = 16 an MMA: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major block
            const uint64_t as = P.a_mn ? 128 : 2, bs = P.b_mn ? 128 : 2;
            for (int i = 0, t; ok && (t = tile_number(P, group, groups, i)) < P.tiles; ++i) {
                const Tile tile = tile_at<CG, KIND>(P, t);
                for (int k0 = tile.k0; k0 < tile.k1 && ok; k0 += P.chunk) {
                    // the accumulator's last sum but one has been taken out
                    ok = used < 2 || __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_empty[buf]), ((used >> 1) & 1) ^ 1, kErrMma, &abort_flag, P.wait_ns));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * 256;
                    const int blocks = P.parts * min(P.chunk, tile.k1 - k0);
                    for (int k = 0; k < blocks; ++k) {
                        // a wait takes 100 cycles also where there is nothing to wait for: the next
                        // block's barrier is looked at while this one's MMAs are issued
                        ok = (ready && P.wait_ns) || __all_sync(0xffffffffu, mbar_wait(full + stage * 8, phase, kErrMma, &abort_flag, P.wait_ns));
                        if (!ok) break;
                        tc_fence_after();
                        const int now = stage;
                        if (++stage == L::kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                        const bool seen = mbar_test(full + stage * 8, phase);
                        const uint64_t at = (uint64_t)(now * (L::kStage >> 4));
                        mma_block<CG>(d, a0 + at, b0 + at, as, bs, idesc, k != 0, empty + now * 8);
                        ready = __all_sync(0xffffffffu, seen);
                    }
                    if (!ok) break;
                    commit<CG>(smem_u32(&acc_full[buf]));
                    ++used;
                    buf ^= 1;
                }
            }
            // none may be in flight when TMEM is released or a CTA of the pair exits
            if constexpr (CG == 2)
                asm volatile(
                    "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                    "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(&done_bar))
                    : "memory");
            else
                commit<1>(smem_u32(&done_bar));
            mbar_drain(smem_u32(&done_bar), 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        // a warp has the 32 rows of its quarter of TMEM's lanes and half of the columns
        const int e = warp - 3, q = warp & 3, half = e >> 2;
        const uint32_t slab = ring + L::kStages * L::kStage + e * kSlab;
        const uint8_t* slab_p = smem_raw + (slab - raw);
        constexpr int kSteps = (KIND == kProduct ? 128 : 64) / kCols;  // slabs of a warp's columns
        constexpr int kChunks = kCols / 32;                            // of 32 columns in a slab
        uint32_t used = 0, dy_phase = 0;
        int buf = 0;
        bool ok = true;
        // columns of this warp: of the product, or of g (those of u are 128 further)
        constexpr int kOwn = KIND == kProduct ? 128 : 64;
        const auto taken = [&] {  // the accumulator may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first<CG>(smem_u32(&acc_empty[buf]));
            ++used;
            buf ^= 1;
        };
        const auto wait_sum = [&] {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&acc_full[buf]), (used >> 1) & 1, kErrEpilogue, &abort_flag, P.wait_ns));
            tc_fence_after();
        };
        for (int i = 0, t; ok && (t = tile_number(P, group, groups, i)) < P.tiles; ++i) {
            const Tile tile = tile_at<CG, KIND>(P, t);
            const int row = tile.m + (int)rank * 128 + q * 32;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
            // fp32: the sums of a chunk of K are added up here, rounded to nearest.  The tensor core
            // drops what it shifts out of its sums; over all of K that would add up.  128 sums a
            // thread leave few registers: 168 and about 1 KB of spills where dg and du follow, 40
            // bytes in the forward product, none in the others.
            float sum[kWide ? 128 : 1];
            if constexpr (kWide) {
#pragma unroll
                for (int i = 0; i < 128; ++i) sum[i] = 0.f;
                for (int k0 = tile.k0; k0 < tile.k1; k0 += P.chunk) {
                    wait_sum();
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 128; i += 16) {
                        float v[16];
                        tmem_ld16(lanes + buf * 256 + half * kOwn + (KIND == kProduct ? i : (i / 64) * 128 + i % 64), v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i + j] += v[j];
                    }
                    taken();
                }
                if (!ok) break;
            }
            if (P.splits > 1) {
                // a piece's sums as they are: columns [0, kOwn) of this warp, for g and u of each
                if constexpr (!kWide) {
                    wait_sum();
                    if (!ok) break;
                }
                float* const to = P.part + ((int64_t)(tile.z * P.splits + tile.piece) * (KIND == kProduct ? 1 : 2) * P.M + row + lane) * P.pitch;
#pragma unroll
                for (int i = 0; i < 128; i += 32) {
                    const int which = KIND == kProduct ? 0 : i / 64, c = half * kOwn + (KIND == kProduct ? i : i % 64);
                    float v[32];
                    if constexpr (kWide) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = sum[i + j];
                    } else {
                        tmem_ld32(lanes + buf * 256 + which * 128 + c, v);
                        tmem_ld_wait();
                    }
                    if (row + lane < P.M) {
                        float* const q = to + which * P.M * P.pitch + tile.n + c;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (tile.n + c + j < P.N) *reinterpret_cast<float4*>(q + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
                if constexpr (!kWide) taken();
                continue;
            }
#pragma unroll(kWide ? kSteps : 1)
            for (int i = 0; i < kSteps; ++i) {
                const int c0 = half * kOwn + i * kCols;  // of the tile
                const int col = tile.n + c0;
                if constexpr (KIND == kGatedBackward) {
                    // dy's piece comes while the MMAs run
                    __syncwarp();
                    expect(smem_u32(&dy_bar[e]), kSlab);
                    load_2d<1>(slab, &P.dy, smem_u32(&dy_bar[e]), col, row);
                }
                if constexpr (!kWide)
                    if (i == 0) wait_sum();
                if constexpr (KIND == kGatedBackward) {
                    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&dy_bar[e]), dy_phase, kErrEpilogue, &abort_flag, P.wait_ns));
                    if (!ok) {
                        if (lane == 0) mbar_drain(smem_u32(&dy_bar[e]), dy_phase);
                        __syncwarp();
                        break;
                    }
                    dy_phase ^= 1;
                } else {
                    if (!ok) break;
                }
                const int which = KIND == kProduct ? tile.z : 0;
                T* const to = static_cast<T*>(P.out[which]) + (int64_t)(row + lane) * P.out_stride[which] + col;
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    float g[32], u[32];
                    if constexpr (kWide) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            g[j] = sum[i * 32 + j];
                            if constexpr (KIND != kProduct) u[j] = sum[64 + i * 32 + j];
                        }
                    } else {
                        tmem_ld32(lanes + buf * 256 + c0 + c * 32, g);
                        if constexpr (KIND != kProduct) tmem_ld32(lanes + buf * 256 + 128 + c0 + c * 32, u);
                        tmem_ld_wait();
                        if (i == kSteps - 1 && c == kChunks - 1) taken();
                    }
                    if constexpr (KIND == kGatedForward) {
                        gate<kFast>(g, u, P.act, P.alpha);
                    } else if constexpr (KIND == kGatedBackward) {
                        float dy[32];
                        get_row<T>(slab, lane, c, dy);
                        gate_back<kFast>(g, u, dy, P.act, P.alpha);
                    }
                    if (P.aligned) {
                        if (row + lane < P.M) {
                            store_row<T>(to + c * 32, g, P.N - col - c * 32, P.aligned == 32);
                            if constexpr (KIND == kGatedBackward)
                                store_row<T>(static_cast<T*>(P.out[1]) + (int64_t)(row + lane) * P.out_stride[1] + col + c * 32, u,
                                             P.N - col - c * 32, P.aligned == 32);
                        }
                    } else {
                        put_row<T>(slab, lane, c, g);  // dg and du are always aligned
                    }
                }
                if constexpr (KIND != kGatedBackward)
                    if (!P.aligned) send<T>(P, which, slab_p, row, col, lane);
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {
        if (threadIdx.x == 0) {
            if (rank == 1) {
                put_other(smem_u32(&other_sent[0]), 0, sent[0]);
                put_other(smem_u32(&other_sent[1]), 0, sent[1]);
            }
            if (abort_flag) put_other(smem_u32(&other_abort), rank ^ 1, 1);
        }
        __syncwarp();
        cluster_sync();
    }
    if (abort_flag || (CG == 2 && other_abort)) {
        // every copy issued must land before an SM exits (without a give-up the MMAs have waited
        // for all); where the producers stopped at different uses, the barriers get what they lack
        if (rank == 0 && threadIdx.x == 0) {
            uint32_t n = max(sent[0], sent[1]);
            if constexpr (CG == 2) n = max(n, max(other_sent[0], other_sent[1]));
            for (uint32_t k = unsettled_from(n, L::kStages); k < n; ++k) {
                const uint32_t bar = smem_u32(&full_bar[k % L::kStages]);
                for (int i = 0; i < 2; ++i) {
                    const Owed o = owed(k, sent[i], CG == 2 ? other_sent[i] : 0, CG == 2, i ? L::kStage - kBlock : kBlock);
                    if (o.arrive) mbar_expect_tx(bar, o.announce);
                    if (o.absent) complete_tx(bar, o.absent);
                }
                mbar_drain(bar, (k / L::kStages) & 1);
            }
        }
        __syncthreads();
        if constexpr (CG == 2) cluster_sync();
    }
    tc_fence_after();
    if (warp == 1) {
        if constexpr (CG == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (P.early) asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct JoinParams {
    const float* part;  // [z][piece][sum][M][pitch]
    int64_t pitch;
    int splits, M, N, act;
    float alpha;
    void* out[2];
    int64_t out_stride[2];
    const void* dy;
    int64_t dy_stride;
};

// The pieces added in order, then what the epilogue does.  Four columns a
// thread; z is the y axis of the grid.
// Bound by latency where it is used: dg and du of 8 rows, F = 8192, two pieces, 5 us;
// dx of 8 rows, C = 2048, 19 pieces, 7 us.
template <typename T, int KIND>
__global__ void __launch_bounds__(256) gated_join(JoinParams J) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr bool kFast = sizeof(T) == 2;
    constexpr int kSums = KIND == kProduct ? 1 : 2;
    const int64_t groups = J.pitch / 4, n = groups * J.M, sum = J.M * J.pitch;
    const float* part = J.part + (int64_t)blockIdx.y * J.splits * kSums * sum;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / groups;
        const int c = (int)(i - r * groups) * 4;
        float v[kSums][4] = {};
#pragma unroll 4
        for (int k = 0; k < J.splits; ++k)
#pragma unroll
            for (int j = 0; j < kSums; ++j) {
                const float4 p = *reinterpret_cast<const float4*>(part + (k * kSums + j) * sum + r * J.pitch + c);
                v[j][0] += p.x;
                v[j][1] += p.y;
                v[j][2] += p.z;
                v[j][3] += p.w;
            }
        if constexpr (KIND == kGatedForward) {
            act_all<4, kFast>(v[0], J.act, J.alpha);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[0][j] *= v[1][j];
        } else if constexpr (KIND == kGatedBackward) {
            float dy[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dy[j] = c + j < J.N ? to_f32(static_cast<const T*>(J.dy)[r * J.dy_stride + c + j]) : 0.f;
            gate_back<kFast>(v[0], v[1], dy, J.act, J.alpha);
        }
#pragma unroll
        for (int k = 0; k < (KIND == kGatedBackward ? 2 : 1); ++k) {
            const int which = KIND == kProduct ? (int)blockIdx.y : k;
            T* out = static_cast<T*>(J.out[which]) + r * J.out_stride[which] + c;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < J.N) out[j] = from_f32<T>(v[k][j]);
        }
    }
}

// ---- host -------------------------------------------------------------------

bool encode(CUtensorMap* map, const GemmOperand& m, int dtype, int box_inner, int box_outer) {
    auto enc = encode_fn();
    if (!enc) return false;
    const CUtensorMapDataType dt = dtype == CT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : dtype == CT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int eb = dtype == CT_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)m.inner, (cuuint64_t)m.outer};
    const cuuint64_t strides[1] = {(cuuint64_t)(m.stride * eb)};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer}, es[2] = {1, 1};
    return enc(map, dt, 2, const_cast<void*>(m.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An MN-major matrix as [n / 64][k][64], loaded 2 x 64 x 64 at a time; its width
// is a multiple of 64.
bool encode_halves(CUtensorMap* map, const GemmOperand& m, int dtype) {
    auto enc = encode_fn();
    if (!enc) return false;
    const CUtensorMapDataType dt = dtype == CT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[3] = {64, (cuuint64_t)m.outer, (cuuint64_t)(m.inner / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)(m.stride * 2), 128};
    const cuuint32_t box[3] = {64, 64, 2}, es[3] = {1, 1, 1};
    return enc(map, dt, 3, const_cast<void*>(m.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int CG, int KIND>
cudaError_t launch_kind(const GemmParams& P, bool follows, int sm_count, cudaStream_t s) {
    auto k = gated_gemm<T, CG, KIND>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<CG>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    const int groups = std::min(P.tiles, std::max(1, sm_count / CG));
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<CG>::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = follows ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, P);
}

template <typename T, int CG>
cudaError_t launch_cg(const Gemm& g, const GemmParams& P, int sm_count, cudaStream_t s) {
    switch (g.kind) {
        case kGatedForward: return launch_kind<T, CG, kGatedForward>(P, g.follows, sm_count, s);
        case kGatedBackward: return launch_kind<T, CG, kGatedBackward>(P, g.follows, sm_count, s);
        default: return launch_kind<T, CG, kProduct>(P, g.follows, sm_count, s);
    }
}

template <typename T>
cudaError_t launch_t(const Gemm& g, GemmParams& P, int cg, int sm_count, cudaStream_t s) {
    return cg == 2 ? launch_cg<T, 2>(g, P, sm_count, s) : launch_cg<T, 1>(g, P, sm_count, s);
}

}  // namespace

namespace {
// How a product is cut: pairs of SMs share a tile where there are more than 128
// rows; K is split where tiles fill less than half of the SMs, into as many
// pieces as are worth it: a block (of 64) takes 0.3 us, the pieces' sums cost
// 8 bytes of L2 traffic each (about 5 TB/s) and their join 4 us.  8 rows of 2048
// channels, F = 8192, gradients in bf16: 161 us unsplit, about 60 split; 2048
// rows of 512, F = 2048: 54 unsplit, 59 with K always split.
struct Cut {
    int cg, m_tiles, n_tiles, splits;
    int64_t pitch;
};
Cut cut_of(GemmKind kind, int64_t M, int64_t N, int64_t K, int parts, int z, int sm_count) {
    Cut c;
    c.cg = M > 128 ? 2 : 1;
    const int n = kind == kProduct ? 256 : 128;
    c.m_tiles = (int)((M + 128 * c.cg - 1) / (128 * c.cg));
    c.n_tiles = (int)((N + n - 1) / n);
    c.pitch = (N + 3) / 4 * 4;
    const int64_t tiles = std::max<int64_t>(1, (int64_t)c.m_tiles * c.n_tiles * z), nk = (K + 63) / 64;
    const int64_t most = std::min<int64_t>(sm_count / c.cg / tiles, nk);
    const double sums = (double)M * c.pitch * z * (kind == kProduct ? 1 : 2);
    double best = 0.3 * nk * parts;
    c.splits = 1;
    for (int64_t k = 2; k <= most; ++k) {
        const double us = 0.3 * ((nk + k - 1) / k) * parts + 4.0 + 8.0 * k * sums / 5e6;
        if (us < best) {
            best = us;
            c.splits = (int)k;
        }
    }
    return c;
}

template <typename T>
cudaError_t launch_join(GemmKind kind, const JoinParams& J, int z, int sm_count, cudaStream_t s) {
    const int64_t n = J.pitch / 4 * J.M;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((n + 255) / 256, 8 * sm_count), (unsigned)(kind == kProduct ? z : 1));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return kind == kGatedForward    ? cudaLaunchKernelEx(&cfg, gated_join<T, kGatedForward>, J)
           : kind == kGatedBackward ? cudaLaunchKernelEx(&cfg, gated_join<T, kGatedBackward>, J)
                                    : cudaLaunchKernelEx(&cfg, gated_join<T, kProduct>, J);
}
}  // namespace

size_t gemm_part_bytes(GemmKind kind, int64_t M, int64_t N, int64_t K, int parts, int z, int sm_count) {
    const Cut c = cut_of(kind, M, N, K, parts, z, sm_count);
    if (c.splits == 1) return 0;
    return ((size_t)z * c.splits * (kind == kProduct ? 1 : 2) * M * c.pitch * 4 + 255) / 256 * 256;
}

cudaError_t launch_gemm(const Gemm& g, int sm_count, cudaStream_t s) {
    const bool wide = g.dtype == CT_F32;
    const int in = wide ? CT_BF16 : g.dtype;  // of the operands
    const int eb = wide ? 4 : 2, cols = 128 / eb;
    GemmParams P{};
    P.a_whole = g.a_mn && g.M % 64 == 0;
    P.b_whole = g.b_mn && g.N % 64 == 0;
    for (int i = 0; i < g.n_a; ++i)
        if (!(P.a_whole ? encode_halves(&P.a[i], g.a[i], in) : encode(&P.a[i], g.a[i], in, 64, g.a_mn ? 64 : 128))) return cudaErrorInvalidValue;
    for (int i = 0; i < g.n_b; ++i)
        if (!(P.b_whole ? encode_halves(&P.b[i], g.b[i], in) : encode(&P.b[i], g.b[i], in, 64, g.b_mn ? 64 : 128))) return cudaErrorInvalidValue;
    const int outs = g.kind == kGatedBackward ? 2 : g.z;
    P.aligned = 32;
    for (int i = 0; i < outs; ++i) {
        P.out[i] = g.out[i];
        P.out_stride[i] = g.out_stride[i];
        const int64_t step = g.M <= 1 ? 0 : g.out_stride[i] * eb;  // one row has no stride
        for (const int n : {32, 16})
            if (((uintptr_t)g.out[i] % n || step % n) && P.aligned >= n) P.aligned = n == 32 ? 16 : 0;
    }
    if (g.kind == kGatedBackward && !encode(&P.dy, g.dy, g.dtype, cols, 32)) return cudaErrorInvalidValue;
    for (int i = 0; i < g.parts; ++i) {
        P.a_part[i] = g.a_part[i];
        P.b_part[i] = g.b_part[i];
    }
    P.parts = g.parts;
    P.nk = (int)((g.K + 63) / 64);
    // fp32: two blocks a sum.  2048 x 512 x 2048: one 53.8 us, 1.6e-7 off; two 46.5 us, 2.4e-7; four 43.7 us,
    // 4.3e-7 (fp32 arithmetic 5.7e-7): the producers turn to another part's map less often
    P.chunk = wide ? 2 : P.nk;
    P.b_block = g.b_block;
    P.a_z = g.a_z;
    P.b_z = g.b_z;
    P.a_mn = g.a_mn;
    P.b_mn = g.b_mn;
    const Cut cut = cut_of(g.kind, g.M, g.N, g.K, g.parts, g.z, sm_count);
    const int cg = cut.cg;
    P.m_tiles = cut.m_tiles;
    P.n_tiles = cut.n_tiles;
    P.splits = cut.splits;
    P.part = g.part;
    P.pitch = cut.pitch;
    P.tiles = P.m_tiles * P.n_tiles * P.splits * g.z;
    // tiles go through strips of eight rows of tiles, so that those at work together share operands
    // in L2 (16384 x 4096 x 1024: 196 us by columns, 184 by strips)
    P.strip = 8;
    if (g.ahead) {
        // the kernel before leaves its last round's idle groups to this one for as long as one of its tiles takes
        const Gemm& h = *g.ahead;
        const Cut before = cut_of(h.kind, h.M, h.N, h.K, h.parts, h.z, sm_count);
        const int groups = std::max(1, sm_count / cg), tiles = before.m_tiles * before.n_tiles * h.z;
        P.early = before.splits == 1 && cut.splits == 1 && before.cg == cg;
        if (P.early && tiles % groups && P.tiles > groups) {
            P.head_groups = groups - tiles % groups;
            P.head_tiles = (int)std::min<int64_t>((h.K + 63) / 64 * h.parts / std::max<int64_t>(1, (int64_t)P.nk * P.parts), P.tiles / groups);
            if (tiles < groups) P.head_tiles = P.tiles / groups;  // they have nothing else to do
        }
    }
    P.M = (int)g.M;
    P.N = (int)g.N;
    P.act = g.act;
    P.alpha = g.alpha;
    const uint32_t type = in == CT_BF16 ? 1u : 0u;
    P.idesc = (1u << 4)                               // D = f32
              | (type << 7) | (type << 10)            // A, B
              | ((uint32_t)g.a_mn << 15) | ((uint32_t)g.b_mn << 16)
              | ((256u >> 3) << 17)                   // N = 256
              | ((128u * cg >> 4) << 24);             // M = 128 or 256
    P.wait_ns = wait_limit_ns();
    if (P.tiles == 0) return cudaSuccess;
    const cudaError_t e = g.dtype == CT_F32 ? launch_t<float>(g, P, cg, sm_count, s)
                        : g.dtype == CT_F16 ? launch_t<__half>(g, P, cg, sm_count, s) : launch_t<__nv_bfloat16>(g, P, cg, sm_count, s);
    if (e != cudaSuccess || P.splits == 1) return e;
    JoinParams J{};
    J.part = g.part;
    J.pitch = P.pitch;
    J.splits = P.splits;
    J.M = P.M;
    J.N = P.N;
    J.act = g.act;
    J.alpha = g.alpha;
    for (int i = 0; i < outs; ++i) {
        J.out[i] = g.out[i];
        J.out_stride[i] = g.out_stride[i];
    }
    J.dy = g.dy.p;
    J.dy_stride = g.dy.stride;
    return g.dtype == CT_F32 ? launch_join<float>(g.kind, J, g.z, sm_count, s)
         : g.dtype == CT_F16 ? launch_join<__half>(g.kind, J, g.z, sm_count, s) : launch_join<__nv_bfloat16>(g.kind, J, g.z, sm_count, s);
}

cudaError_t gated_error_word(unsigned int* v, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(v, g_device_error, sizeof(*v));
    if (e == cudaSuccess && clear && *v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace ct
