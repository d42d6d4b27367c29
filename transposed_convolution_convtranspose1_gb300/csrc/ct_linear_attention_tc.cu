// ct_linear_attention_tc.cu -- the recurrence of ct_linear_attention.h in
// chunks of 128 tokens on the tensor cores (16-bit inputs, head sizes up to
// 128), for prompts and gradients.
//
// With the chunk's rows Z, X (128 x Da), Y (128 x Db), a row i's distance
// d(i, j) >= 0 to the rows it sees, and M the matrix before the chunk:
//   S   = Z X^T                          128 x 128
//   P   = S * decay^d(i,j) * mscale, 0 where j is not seen by i
//   out = oscale * (P Y + decay^w(i) * (Z M))
//   M  <- decay^e M + (mscale * decay^f(j) x_j)^T Y
// forward in time (n rows in the chunk): d = i - j, w = i + 1, f = n - 1 - j,
// e = n; backward: d = j - i, w = n - i, f = j, e = n, one less in w and e for
// the chunk that holds the sequence's last token.
//
// All four products are tcgen05 MMAs with fp32 accumulators in TMEM, 16-bit
// operands.  S is exact in its operands.  P, M and the decayed x are fp32
// values, and each enters as hi + lo, two 16-bit numbers, in two MMAs: with
// one rounding each, out's error would be 1.4 to 1.7 times that of rounding
// out itself, and the fp32 state's 2^-9; with two, both to nearest, a bf16
// value keeps about 17 bits (an f16 one 22) and the state comes to about 3e-6
// of its norm.  f16's lo parts are kept 2^11 times their size, or they would
// lose their digits where values are small (gradients of 1e-5 came out 1e-3
// off, a state of 1e-6 under queries of 64 8e-3): their products are summed
// first, and the MMA that adds the first of the others scales the sum down.
// P and x enter from TMEM (P over S, in place), M from shared memory.
//
// One CTA per sequence, head and segment walks its chunks in order.  Sixteen
// warps do the same step of the work at the same time, each a lane quarter of
// TMEM and a quarter of the columns (or tokens):
//   A  M times decay^e in TMEM, decayed x; then M's hi, lo to shared memory
//   B  out of the chunk before: TMEM -> memory;  S -> P
//   C  the scaling of Z M
// while the tensor cores run P Y of the chunk before and S under A, the new M
// under M's split, Z M under B.  Warps with a role each (P, x, M at the same
// time) came first: their bodies evicted one another from the instruction
// caches and a warp issued once in 13 cycles (8 x 2048 x 16 heads of 128:
// 93 us; as it is, 67).
// One more warp loads tiles by TMA into a ring of five that Z, X and Y take in
// turn (X's place, once x is in TMEM, stages out for its TMA store), one issues
// the MMAs.
// What bounds it is the chain A, B, C of a chunk and the waits between its
// steps, about 7000 cycles at D = 128 and 4700 at 64, one CTA to an SM; memory
// would take 5650 (4 x 128 x D x 2 bytes at the SM's share of the copy rate)
// and 2820, the MMAs 3600 at D = 128.  Measured: 8 x 2048 x 16 heads of 128
// with the last state 67 us (61% of the copy rate), 32768 tokens of 8
// heads of 64 in 19 segments 91 us, the three gradients of 8 x 2048 x 8 heads
// of 64 in one launch 78 us.
//
// Few heads and long sequences: a sequence is cut into segments.  A first
// launch forms each segment's own sum (the last line above from M = 0), a
// small kernel chains them into the matrix before each segment, and the main
// launch runs all segments at once.
//
// More walks than SMs: the chunks of all walks, one after another, are cut into
// equal runs, one for each SM.  A walk cut by a run's end is begun by the one
// CTA as its first piece and ended by the next CTA as its last, which takes the
// matrix from memory; nothing is read twice (the gradients above: 192 walks of
// 16 chunks, 21 chunks an SM instead of 32; 96 us in two turns).  CTAs number
// themselves as they start, so the one that another waits for has started
// before it, and its first piece waits for nobody: the walks end however many
// of them the GPU, or the part of it that the stream has, runs at once.
#include <algorithm>
#include <cstring>

#include "ct_linear_attention.h"
#include "ct_tcgen05.cuh"
#include "ct_types.cuh"

namespace ct {
namespace {

using namespace tcg;

constexpr int kC = 128;            // tokens of a chunk
constexpr int kLaWorkers = 16;     // warps
constexpr int kLaThreads = (kLaWorkers + 2) * 32;
constexpr uint32_t kTmemP = 0, kTmemP2 = 256, kTmemX = 128;
constexpr float kF16Max = 65504.f;

struct LaTcParams {
    CUtensorMap tz, tx, ty;      // (D, T, H, B), boxes of 64 columns x 128 tokens
    CUtensorMap to;              // boxes of DB / 4 columns x 32 tokens
    void* out;
    int64_t os[3];
    const void *z, *x, *y;       // the same tensors, for la_token_by_token
    int64_t zs[3], xs[3], ys[3];
    const float* m_in;           // before segment 0 of the walk, or per segment
    int m_in_t, m_in_seg;        // transposed; one for each segment ([seg][bh][Da][Db])
    float* m_out;                // after the walk of a segment ([seg][bh])
    int final;                   // m_out is the walk's result, not a segment's own sum
    const float* log_decay;
    const int32_t* lengths;
    int* flags;                  // f16: [bh], set where a value left f16's range
    float mscale, oscale;
    int reverse, T, H, Da, Db, BH;
    int seg_tokens, segs;
    uint32_t idesc_s, idesc_n;   // N = 128, B K-major; N = DB, B MN-major
    uint64_t wait_ns;
};

// Up to three walks of one launch (the gradients of q, k and v).
struct LaTcBatch {
    LaTcParams core[3];
    int ctas;                    // of one core
    // shared walks (quota > 0): the chunks of all walks in a row, cut into runs
    // of `quota` chunks, one for each CTA
    int quota, chunks, walks;    // chunks: of one walk; quota >= chunks
    float* handed;               // [CTA][Da][Db]
    unsigned* done;              // [CTA]: its first piece's matrix is there
    unsigned* read;              // [CTA]: m_in is not read any more (la_token_by_token)
    unsigned* started;           // CTAs that have taken a number
};

// Tile n of the walk (Z, X, Y of chunk 0, Z, X, Y of chunk 1, ...) lies in
// place n % 5 of the ring; M's parts after it, and decayed x where it is an
// operand in shared memory.
//
// kStacked (64 x 64): x enters as its hi and lo parts one above the other, 128
// rows of one MMA, and so does M: its first 64 TMEM rows sum the hi products,
// the last 64 the lo products, and Z M takes hi and lo of the first and hi of
// the second.  Against x in TMEM, 64 of whose 128 rows are empty at this size,
// the new M takes half the MMAs, and all lanes and warps share the work.
template <int DA, int DB>
struct LaShape {
    static constexpr bool kStacked = DA == 64 && DB == 64;
    static constexpr uint32_t kTile = 256 * (DA > DB ? DA : DB), kM = 2 * DA * DB;
    static constexpr int kMParts = kStacked ? 3 : 2;
    static constexpr uint32_t oM = 5 * kTile, oX = oM + kMParts * kM, kX = kStacked ? 32768 : 0;
    static constexpr uint32_t kBytes = oX + 2 * kX;
    static __device__ __forceinline__ uint32_t z(int c) { return (uint32_t)(3 * c % 5) * kTile; }
    static __device__ __forceinline__ uint32_t x(int c) { return (uint32_t)((3 * c + 1) % 5) * kTile; }
    static __device__ __forceinline__ uint32_t y(int c) { return (uint32_t)((3 * c + 2) % 5) * kTile; }
};

// MN-major operand, 128-byte swizzle: rows of 64 MN elements per K index,
// 8-row groups 1024 bytes apart, `block` bytes between blocks of 64.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// MMAs issued by one lane of a converged warp: the branch is inside, so that
// descriptors and addresses stay in uniform registers (under `if (lane == 0)`
// each MMA cost its thread about 75 cycles of moves into them).
__device__ __forceinline__ void mma_ss_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with D scaled by 2^-DOWN before the product is added.
template <int DOWN>
__device__ __forceinline__ void mma_ss_down(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p, %4;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(DOWN)
        : "memory");
}
template <int DOWN>
__device__ __forceinline__ void mma_ts_down(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p, %4;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "n"(DOWN)
        : "memory");
}
// D += A B with A (16-bit, two consecutive K in a column) in TMEM.
__device__ __forceinline__ void mma_ts_one(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t& bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(&bar))
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 lanes x 32 columns: thread i holds lanes i / 4 (even registers) and
// i / 4 + 8 (odd ones), column i % 4 of every four: the layout of a transposed
// ldmatrix of 16-bit pairs.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, transposed.
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// One arrival for the warp, after what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t& bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
}

template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float* v) {
    if constexpr (N == 32) tmem_ld32(taddr, v);
    else tmem_ld16(taddr, v);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t* r) {
    if constexpr (N == 32) tmem_st32(taddr, r);
    else tmem_st16(taddr, r);
}
// N columns of TMEM <- v * f, 16 at a time (fewer registers at once).
template <int N>
__device__ __forceinline__ void tmem_st_scaled(uint32_t taddr, const float* v, float f) {
#pragma unroll
    for (int k = 0; k < N / 16; ++k) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 m = __fmul2_rn(make_float2(v[16 * k + 2 * i], v[16 * k + 2 * i + 1]), make_float2(f, f));
            u[2 * i] = __float_as_uint(m.x);
            u[2 * i + 1] = __float_as_uint(m.y);
        }
        tmem_st16(taddr + k * 16, u);
    }
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Eight consecutive floats (32 bytes, aligned to that) as one access.
__device__ __forceinline__ void load8(const float* p, float* v) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float2 lds64(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two fp32 values as one word of two T.
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// v = hi + lo / kLoUp to within U^2 |v|, each half a T.  f16 has five bits of
// exponent: lo is kept 2^11 times its size, as large as hi, so that it has all
// its digits wherever hi has (and the sum is good to 2^-36 below that, where hi
// is subnormal).
template <typename T>
constexpr int kLoBits = std::is_same<T, __half>::value ? 11 : 0;
template <typename T>
constexpr float kLoUp = (float)(1 << kLoBits<T>);
template <typename T>
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
    hi = pack2<T>(v.x, v.y);
    float2 r = __ffma2_rn(unpack2<T>(hi), make_float2(-1.f, -1.f), v);
    if constexpr (kLoBits<T> != 0) r = __fmul2_rn(r, make_float2(kLoUp<T>, kLoUp<T>));
    lo = pack2<T>(r.x, r.y);
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void mbar_inval(uint32_t bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Waits, for a limited time, until another CTA of the launch has set *done.
__device__ __forceinline__ bool wait_done(const unsigned* done, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
        if (v) return true;
        if (limit_ns == 0 || globaltimer_ns() - t0 > limit_ns) {
            atomicOr(&g_device_error, kErrEpilogue);
            return false;
        }
        __nanosleep(100);
    }
}

// Votes of the worker warps (a barrier of theirs).
__device__ __forceinline__ bool workers_any(bool v) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((unsigned)v), "n"(kLaWorkers * 32)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ bool not_finite(float v) { return !(fabsf(v) < __uint_as_float(0x7f800000u)); }
__device__ __forceinline__ void set_done(unsigned* done) {
    __threadfence();
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(done), "r"(1u) : "memory");
}

// Pieces of this CTA's run once more (bit i: of the i-th walk it meets), token
// by token, M in shared memory (`M`, 128 columns a row, then the token's
// values).  In a chunk's products a row meets every token's y with a factor of
// 0 where it does not see it, and 0 times an infinity or a NaN is NaN: outputs
// of tokens before such a value are lost with the others.  Here no token meets
// a later one.  For pieces that hold such values alone (2 us a token), and
// after everything else, so that nothing of it is alive in the walk's own loop
// (M in registers takes half the time here, but up to 2 us of the cases above,
// whose loop the compiler then schedules otherwise).
//
// A walk's last matrix may take the first one's place.  The CTA that ends such
// a walk leaves it to this function, and waits until the CTA that began the
// walk has read the first one again: pieces that begin a walk come first here
// and wait for nobody.
template <typename T>
__device__ __forceinline__ void la_token_by_token(const LaTcBatch& Q, unsigned me, unsigned pieces, float* M) {
    float *xs = M + 128 * 128, *zs = xs + 128, *ys = zs + 128, *part = ys + 128;
    const int tid = threadIdx.x, c = tid & 127, quarter = tid >> 7;
    const int run0 = (int)me * Q.quota, run1 = min(run0 + Q.quota, Q.walks * Q.chunks);
#pragma unroll 1
    while (pieces) {
        const int piece = 31 - __clz(pieces);
        pieces ^= 1u << piece;
        unsigned cta = me;
        int w0 = 0, w1 = Q.chunks;  // (no quota: 0 chunks)
        if (Q.quota) {
            cta = run0 / Q.chunks + piece;
            w0 = max(run0 - (int)cta * Q.chunks, 0);
            w1 = min(run1 - (int)cta * Q.chunks, Q.chunks);
        }
        const bool begun = w0 > 0, handed = w1 < Q.chunks;
        const LaTcParams& P = Q.core[cta / (unsigned)Q.ctas];
        cta %= (unsigned)Q.ctas;
        const int bh = (int)(cta % (unsigned)P.BH), seg = (int)(cta / (unsigned)P.BH), b = bh / P.H, h = bh % P.H;
        const int len = P.lengths ? max(0, min(P.T, P.lengths[b])) : P.T;
        const int s0 = Q.quota ? (P.reverse ? Q.chunks - w1 : w0) * kC : seg * P.seg_tokens;
        const int s1 = min(P.T, Q.quota ? s0 + (w1 - w0) * kC : s0 + P.seg_tokens);
        const int n = max(0, min(len, s1) - s0);
        const bool holds_end = P.reverse && s0 + n == len;
        const int64_t msize = (int64_t)P.Da * P.Db;
        const float* m_in = begun ? Q.handed + (me - 1) * msize : P.m_in ? P.m_in + ((P.m_in_seg ? (int64_t)seg * P.BH : 0) + bh) * msize : nullptr;
        const bool m_in_t = P.m_in_t && !begun;
        const float gamma = expf(la_log_decay(P.log_decay[h]));
        const int a0 = quarter * 32, a1 = min(a0 + 32, P.Da);
        bool odd = false;
        if (c < P.Db)
#pragma unroll 1
            for (int a = a0; a < a1; ++a) {
                const float m = m_in ? m_in[m_in_t ? (int64_t)c * P.Da + a : (int64_t)a * P.Db + c] : 0.f;
                M[a * 128 + c] = m;
                odd = odd || not_finite(m);
            }
        odd = workers_any(odd);
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const int64_t t = s0 + (P.reverse ? n - 1 - k : k);
            if (quarter == 0 && c < P.Da) xs[c] = to_f32(static_cast<const T*>(P.x)[b * P.xs[0] + t * P.xs[1] + h * P.xs[2] + c]) * P.mscale;
            if (quarter == 1 && c < P.Da) zs[c] = to_f32(static_cast<const T*>(P.z)[b * P.zs[0] + t * P.zs[1] + h * P.zs[2] + c]);
            if (quarter == 2 && c < P.Db) ys[c] = to_f32(static_cast<const T*>(P.y)[b * P.ys[0] + t * P.ys[1] + h * P.ys[2] + c]);
            workers_any(false);
            const float g = holds_end && k == 0 ? 1.f : gamma;
            float sum = 0.f;
            if (c < P.Db)
#pragma unroll 4
                for (int a = a0; a < a1; ++a) {
                    const float m = fmaf(xs[a], ys[c], g * M[a * 128 + c]);
                    M[a * 128 + c] = m;
                    sum = fmaf(m, zs[a], sum);
                }
            part[tid] = sum;
            workers_any(false);
            if (tid < P.Db)
                static_cast<T*>(P.out)[b * P.os[0] + t * P.os[1] + h * P.os[2] + tid] =
                    from_f32<T>((part[tid] + part[128 + tid] + part[256 + tid] + part[384 + tid]) * P.oscale);
        }
        if (handed) {  // its matrix is where the next CTA takes it
            if (tid == 0) set_done(Q.read + me);
        } else if (P.m_out && P.final) {
            // the matrix began so: the CTA before is at its piece once more
            if (begun && odd && P.m_out == P.m_in) {
                const bool late = tid == 0 && !wait_done(Q.read + me - 1, P.wait_ns);
                if (workers_any(late)) return;
            }
            const float last = P.reverse && n > 0 ? gamma : 1.f;
            if (c < P.Db)
#pragma unroll 1
                for (int a = a0; a < a1; ++a) P.m_out[bh * msize + (int64_t)a * P.Db + c] = M[a * 128 + c] * last;
        }
    }
}

template <typename T, int DA, int DB, bool STATE>
__global__ void __launch_bounds__(kLaThreads, 1) la_chunks(const __grid_constant__ LaTcBatch Q) {
    using Sh = LaShape<DA, DB>;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    // f16 scores and decayed x are kept 16 and 64 times their size: the ranges
    // then are 4094 and 1023 (beyond them the flag has the head done again),
    // and they are good to 2^-40 and 2^-42 where they are smallest, M to 2^-36
    constexpr float kUp = kHalf ? 16.f : 1.f, kUpX = kHalf ? 64.f : 1.f;
    constexpr int kN = DB / 4;  // columns of Y, M and out a warp has
    constexpr bool kStacked = Sh::kStacked;
    constexpr int kDown = kLoBits<T>;
    // 64 columns of out and M leave room for a second S: the next chunk's is
    // formed before P Y of this one
    constexpr bool kTwoS = DB == 64;
    constexpr uint32_t kTmemO = kTwoS ? 384 : 256, kTmemM = kTwoS ? 448 : 384;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t x_full[2], y_full[2], z_free[2], x_free[2], y_free[2];  // x_full: Z and X
    __shared__ uint64_t s_ready, m_ready, a_done, p_done, o_ready, o_free, sum_ready, drain_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned number;
    __shared__ volatile int abort_flag;
    __shared__ unsigned again;  // pieces for la_token_by_token
    // tab[0][kC - 1 + j - i]: factor of S[i][j], 0 where i does not see j; [1]:
    // one later, for aligned pairs, half the banks on (lanes take both in turn)
    __shared__ __align__(8) float tab[2][2 * kC + 16];
    __shared__ float pw[kC + 2];    // decay^k

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the tiles' swizzle needs 1024-byte alignment, which the declaration asks
    // for; there is no room to round up (227 KiB are used at 128 x 128)
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_device_error, kErrProducer);
        return;
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        again = 0;
        number = Q.quota ? atomicAdd(Q.started, 1u) : blockIdx.x;
    }
    if (warp == kLaWorkers + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // One piece, a whole walk or segment, without a quota.  With one, the run's
    // pieces from its end to its start: the first may be a walk's beginning,
    // handed to the next CTA, the last a walk's end, begun by the CTA before,
    // which had it done before this one's other pieces: quota >= chunks.
    const unsigned me = number;
    const int run0 = (int)me * Q.quota;
    int run = min(run0 + Q.quota, Q.walks * Q.chunks);
    do {
    unsigned cta = me;
    int w0 = 0, w1 = 0;  // the piece's chunks of its walk
    if (Q.quota) {
        cta = (unsigned)(run - 1) / (unsigned)Q.chunks;
        const int walk0 = (int)cta * Q.chunks, from = max(run0, walk0);
        w0 = from - walk0;
        w1 = run - walk0;
        run = from;
    }
    const LaTcParams& P = Q.core[cta / (unsigned)Q.ctas];
    cta %= (unsigned)Q.ctas;
    const int bh = (int)(cta % (unsigned)P.BH), seg = (int)(cta / (unsigned)P.BH);
    const int b = bh / P.H, h = bh % P.H;
    const int len = P.lengths ? max(0, min(P.T, P.lengths[b])) : P.T;
    const int s0 = Q.quota ? (P.reverse ? Q.chunks - w1 : w0) * kC : seg * P.seg_tokens;
    const int s1 = min(P.T, Q.quota ? s0 + (w1 - w0) * kC : s0 + P.seg_tokens);
    const int n_tok = max(0, min(len, s1) - s0);
    const int n_chunks = (n_tok + kC - 1) / kC;
    const int64_t msize = (int64_t)P.Da * P.Db;
    // the walk's first chunk holds the sequence's last token: its matrix is
    // that token's own gradient, undecayed
    const bool holds_end = P.reverse && n_tok > 0 && s0 + n_tok == len;

    // tokens after the sequence's length: out = 0 (whole chunks of them; the
    // last chunk's own are written with it)
    if (!STATE && P.out) {
        const int from = s0 + n_chunks * kC;
        const int64_t rows = s1 - from;
        T* out = static_cast<T*>(P.out) + b * P.os[0] + h * P.os[2];
        for (int64_t i = threadIdx.x; i < rows * P.Db; i += kLaThreads) out[(from + i / P.Db) * P.os[1] + i % P.Db] = from_f32<T>(0.f);
    }
    const bool begun = w0 > 0, handed = w1 < Q.chunks;  // the CTA before, the next one has the rest
    bool late = false;
    if (begun && threadIdx.x == 0) late = !wait_done(Q.done + me - 1, P.wait_ns);
    if (__syncthreads_or(late)) break;
    const float* m_in = begun ? Q.handed + (me - 1) * msize : P.m_in ? P.m_in + (P.m_in_seg ? ((int64_t)seg * P.BH + bh) * msize : bh * msize) : nullptr;
    const bool m_in_t = P.m_in_t && !begun, last_piece = P.final && !handed;
    float* m_out = handed ? Q.handed + me * msize : P.m_out ? P.m_out + ((int64_t)seg * P.BH + bh) * msize : nullptr;
    if (n_chunks == 0 && m_out)  // (the same for every thread)
        for (int64_t i = threadIdx.x; i < msize; i += kLaThreads)
            m_out[i] = m_in ? (m_in_t ? m_in[(i % P.Db) * P.Da + i / P.Db] : m_in[i]) : 0.f;
    if (n_chunks > 0) {

    const float g = la_log_decay(P.log_decay[h]);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&y_full[i]), 1);
            mbar_init(smem_u32(&y_free[i]), 1);
            mbar_init(smem_u32(&z_free[i]), 1);
            mbar_init(smem_u32(&x_full[i]), 1);
            mbar_init(smem_u32(&x_free[i]), kLaWorkers + (STATE ? 0 : 1));
        }
        mbar_init(smem_u32(&s_ready), 1);
        mbar_init(smem_u32(&a_done), kLaWorkers);
        mbar_init(smem_u32(&p_done), kLaWorkers);
        mbar_init(smem_u32(&o_ready), 1);
        mbar_init(smem_u32(&m_ready), 1);
        mbar_init(smem_u32(&o_free), kLaWorkers);
        mbar_init(smem_u32(&sum_ready), kLaWorkers / 2);
        mbar_init(smem_u32(&drain_bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (threadIdx.x < kC + 1) pw[threadIdx.x] = expf((float)threadIdx.x * g);
    for (int i = threadIdx.x; i < 2 * kC; i += kLaThreads) {
        const int d = P.reverse ? i - (kC - 1) : (kC - 1) - i;
        const float f = d < 0 ? 0.f : expf((float)d * g) * (P.mscale * kUp);
        tab[0][i] = f;
        if (i > 0) tab[1][i - 1] = f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // decayed x of chunk c; without S its place serves every second chunk, so
    // that x is made ready while the chunk before is multiplied
    auto x_at = [&](int c) { return STATE && (c & 1) ? kTmemP : kTmemX; };
    auto x_smem = [&](int c) { return base + Sh::oX + (STATE && (c & 1) ? Sh::kX : 0); };
    auto p_at = [&](int c) { return kTwoS && (c & 1) ? kTmemP2 : kTmemP; };
    auto chunk_at = [&](int c) { return P.reverse ? n_chunks - 1 - c : c; };
    auto rows_of = [&](int k) { return min(kC, n_tok - k * kC); };
    auto waits = [&](uint64_t& bar, int parity, unsigned code) {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), (uint32_t)parity & 1u, code, &abort_flag, P.wait_ns));
    };

    if (warp < kLaWorkers) {
        const int w4 = warp & 3, g4 = warp >> 2;
        const int row = w4 * 32 + lane, col0 = g4 * kN;
        const bool fed = DA == 128 || kStacked || w4 * 32 < DA;  // columns of X feed this lane quarter of the decayed x and of M
        [[maybe_unused]] float top = 0.f;
        // TMEM's M times its true size: stacked, the sums of lo products keep
        // lo's scale; otherwise M starts a chunk in it, as lo products come
        // first, and ends in hi's
        const bool lo_rows = kStacked && w4 >= 2;
        const float m_start = !kStacked || lo_rows ? kUpX * kLoUp<T> : kUpX, m_end = lo_rows ? 1.f / (kUpX * kLoUp<T>) : 1.f / kUpX;
        bool ok = true;
        if (!fed) {
            uint32_t zero[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) zero[i] = 0;
            tmem_st32(lane_base + kTmemX + g4 * 32, zero);
            if (STATE) tmem_st32(lane_base + kTmemP + g4 * 32, zero);
            tmem_stn<kN>(lane_base + kTmemM + col0, zero);
            tmem_st_wait();
        }
        // ldmatrix: lanes 0-7, 8-15, 16-23, 24-31 point at the rows of the
        // matrices (x columns 0-7 | 8-15) x (tokens 0-7), then tokens 8-15
        const uint32_t xs = base + (uint32_t)(w4 >> 1) * 16384u + (g4 * 32 + (lane & 7) + (lane >> 4) * 8) * 128u;
        const uint32_t ch = (uint32_t)(w4 & 1) * 4 + ((lane >> 3) & 1);
        const int j0 = g4 * 32 + 2 * (lane & 3);  // this lane's tokens of x: j0 + 8 m, + 1

        // out of chunk c (v: its sums, read from TMEM), staged in the place of a
        // tile that nothing reads any more, this warp's 32 rows x kN columns.
        // o_free then lets Z M of the chunk after begin: out's place is free
        // and this warp's part of M is in shared memory.
        auto write_out = [&](int c, uint32_t place, const float (&v)[kN]) {
            const int n = rows_of(chunk_at(c));
            tc_fence_before();
            warp_arrive(o_free, lane);
            const float2 os = make_float2(P.oscale / kUp, P.oscale / kUp);
            const uint32_t tile = base + place + (uint32_t)warp * (32 * kN * 2);
            // rows of 64 (32) bytes, swizzled as the tensor map says
            const uint32_t at = tile + lane * (kN * 2), sw = kN == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
            for (int k = 0; k < kN / 8; ++k) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 m = __fmul2_rn(make_float2(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]), os);
                    u[i] = row < n ? pack2<T>(m.x, m.y) : 0u;
                }
                sts128(at + (k ^ sw) * 16u, u[0], u[1], u[2], u[3]);
            }
            fence_async_smem();
            __syncwarp();
            const int t = s0 + chunk_at(c) * kC + w4 * 32;
            if (lane == 0 && t < P.T && col0 < P.Db) tma_store_4d(&P.to, tile, col0, t, h, b);
        };

        // P of chunk c with n tokens, from S in its place
        auto make_p = [&](int c, int n) {
            tc_fence_after();
            const int p0 = g4 * 32;  // columns of S
            uint32_t u[32];          // hi, then lo
            // whether any of the 32 columns is seen by any of the 32 rows
            const bool seen = P.reverse ? g4 >= w4 : g4 <= w4;
            if (!seen) {
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = 0;
            } else {
                float v[32];
                tmem_ld32(lane_base + p_at(c) + p0, v);
                // the factors are on their way while S is (the MMAs' own reads
                // of shared memory make theirs slow)
                const int at = (kC - 1) + p0 - row;
                const uint32_t ft = smem_u32(tab[at & 1] + (at & ~1));
                float2 f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = lds64(ft + 8 * i);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 m = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), f[i]);
                    v[2 * i] = m.x;
                    v[2 * i + 1] = m.y;
                }
                if (n < kC)  // rows after the end hold anything, NaN included
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (row >= n || p0 + i >= n || (P.reverse ? p0 + i < row : p0 + i > row)) v[i] = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    split2<T>(make_float2(v[2 * i], v[2 * i + 1]), u[i], u[16 + i]);
                    if constexpr (kHalf) top = fmaxf(top, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
                }
            }
            tmem_st32(lane_base + p_at(c) + p0, u);
        };

        // this warp's part of M before the chunk at hand: a thread has kN
        // columns of a row, eight to an access where rows lie on 32 bytes
        // (single ones touch a sector each: the segments' matrices of 128 x 128
        // then cost more than their chunks)
        float mv[kN];
        const bool wide = P.Db % 8 == 0 && ((uintptr_t)m_in | (uintptr_t)m_out) % 32 == 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) mv[i] = 0.f;
        if (m_in && row < P.Da) {
            if (wide && !m_in_t) {
#pragma unroll
                for (int i = 0; i < kN; i += 8)
                    if (col0 + i < P.Db) load8(m_in + (int64_t)row * P.Db + col0 + i, mv + i);
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (col0 + i < P.Db) mv[i] = m_in[m_in_t ? (int64_t)(col0 + i) * P.Da + row : (int64_t)row * P.Db + col0 + i];
            }
        }
        auto rescale = [&] {  // what TMEM holds to M
            if constexpr (kHalf)
#pragma unroll
                for (int i = 0; i < kN; ++i) mv[i] *= m_end;
        };
        for (int c = 0; c < n_chunks; ++c) {
            const int n = rows_of(chunk_at(c));
            const int first = holds_end && c == 0 ? 1 : 0;
            // ------------------------------------------------- A: M, and x
            // (the chunk before's M has been read in its step C)
            // (with two places for S it was formed long ago, of the loaded X)
            ok = !STATE && kTwoS ? waits(s_ready, c, kErrEpilogue) : waits(x_full[c & 1], c >> 1, kErrEpilogue);
            if (!ok) break;
            if constexpr (kStacked) {
                if (!STATE) tmem_st_scaled<kN>(lane_base + kTmemM + col0, mv, pw[n - first] * m_start);
                // 8 columns of a token at a time, in the tile's own places, the
                // second ones loaded before the first are split
                const int j0 = threadIdx.x >> 3;
                const uint32_t at0 = (uint32_t)j0 * 128u + (uint32_t)((threadIdx.x ^ j0) & 7) * 16u;
                // the factor of the last row forward in time (0 for tokens
                // after it), of the first one backward
                const float* ft = tab[0] + (P.reverse ? kC - 1 : kC - n) + j0;
                uint32_t x[2][4];
                float fx[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds128(base + Sh::x(c) + at0 + i * 8192u, x[i]);
                    fx[i] = ft[i * 64] * (kUpX / kUp);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + i * 64;
                    const uint32_t at = at0 + i * 8192u;
                    uint32_t hi[4], lo[4];
                    const float f = fx[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float2 v = __fmul2_rn(unpack2<T>(x[i][k]), make_float2(f, f));
                        if (n < kC && j >= n) v = make_float2(0.f, 0.f);  // what lies after the end may be NaN
                        split2<T>(v, hi[k], lo[k]);
                        if constexpr (kHalf) top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                    sts128(x_smem(c) + at, hi[0], hi[1], hi[2], hi[3]);
                    sts128(x_smem(c) + 16384u + at, lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                if (!STATE) tmem_st_wait();
            } else if (fed) {
                // the factors of the last row forward in time (0 for tokens
                // after it), of the first one backward
                const int at = (P.reverse ? kC - 1 : kC - n) + j0;
                const float2* ft = reinterpret_cast<const float2*>(tab[at & 1] + (at & ~1));
                float2 f[4];
                uint32_t x[2][8];  // 32 tokens x 16 columns of x
#pragma unroll
                for (int ah = 0; ah < 2; ++ah)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        ldsm4_trans(xs + Sh::x(c) + k * 2048u + (((ch + ah * 2) ^ (lane & 7)) << 4), x[ah] + 4 * k);
#pragma unroll
                for (int m = 0; m < 4; ++m) f[m] = ft[4 * m];
                if (!STATE) tmem_st_scaled<kN>(lane_base + kTmemM + col0, mv, pw[n - first] * m_start);
                if constexpr (kUpX != kUp)
#pragma unroll
                    for (int m = 0; m < 4; ++m) f[m] = __fmul2_rn(f[m], make_float2(kUpX / kUp, kUpX / kUp));
#pragma unroll
                for (int ah = 0; ah < 2; ++ah) {
                    uint32_t u[16];  // hi, then lo
#pragma unroll
                    for (int r = 0; r < 8; ++r) {  // r % 2: 8 columns; r / 2: 8 tokens
                        float2 v = __fmul2_rn(unpack2<T>(x[ah][r]), f[r >> 1]);
                        if (n < kC) {  // what lies after the end may be NaN
                            if (j0 + 8 * (r >> 1) >= n) v.x = 0.f;
                            if (j0 + 8 * (r >> 1) + 1 >= n) v.y = 0.f;
                        }
                        split2<T>(v, u[r], u[8 + r]);
                        if constexpr (kHalf) top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                    tmem_st_16x32(lane_base + ((uint32_t)(ah * 16) << 16) + x_at(c) + g4 * 32, u);
                }
                if (!STATE) tmem_st_wait();
            }
            if (STATE) {
                warp_arrive(x_free[c & 1], lane);
                if (c > 0) {
                    ok = waits(m_ready, c - 1, kErrEpilogue);
                    if (!ok) break;
                    tc_fence_after();
                    tmem_ldn<kN>(lane_base + kTmemM + col0, mv);
                    tmem_ld_wait();
                    rescale();
                }
                tmem_st_scaled<kN>(lane_base + kTmemM + col0, mv, pw[n - first] * m_start);
                tmem_st_wait();
            }
            if (n < kC) {  // rows of Y after the end meet factors of 0: they must be finite
                ok = waits(y_full[c & 1], c >> 1, kErrEpilogue);
                if (!ok) break;
                const uint32_t ys = base + Sh::y(c);
                for (int i = threadIdx.x; i < (kC - n) * 8 * (DB / 64); i += kLaWorkers * 32) {
                    const int blk = i / ((kC - n) * 8), r = i % ((kC - n) * 8);
                    sts128(ys + blk * 16384u + (uint32_t)(n + r / 8) * 128u + (uint32_t)(r % 8) * 16u, 0, 0, 0, 0);
                }
                fence_async_smem();
            }
            tc_fence_before();
            warp_arrive(a_done, lane);
            if constexpr (!STATE) {
                // ------------------------------------------- A: M's parts
                if (fed) {
                    const uint32_t at = base + Sh::oM + (uint32_t)(col0 >> 6) * (DA * 128u) + (uint32_t)(row & (DA - 1)) * 128u;
#pragma unroll
                    for (int k = 0; k < kN / 8; ++k) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float2 m = make_float2(mv[8 * k + 2 * i], mv[8 * k + 2 * i + 1]);
                            if constexpr (kStacked && kHalf)
                                if (lo_rows) m = __fmul2_rn(m, make_float2(kLoUp<T>, kLoUp<T>));
                            split2<T>(m, hi[i], lo[i]);
                            if constexpr (kHalf) top = fmaxf(top, fmaxf(fabsf(m.x), fabsf(m.y)));
                        }
                        const uint32_t o = ((uint32_t)(((col0 & 63) >> 3) + k) ^ (uint32_t)(row & 7)) * 16u;
                        if (lo_rows) {  // 2^-9 (2^-12) of M: their hi part is enough
                            sts128(at + 2 * Sh::kM + o, hi[0], hi[1], hi[2], hi[3]);
                            continue;
                        }
                        sts128(at + o, hi[0], hi[1], hi[2], hi[3]);
                        sts128(at + Sh::kM + o, lo[0], lo[1], lo[2], lo[3]);
                    }
                    fence_async_smem();
                }
                // ---------------------------------------------- B: out, P
                // With S formed and every warp's step A done nothing reads X
                // any more.  Warps that had nothing to do in A take P first,
                // the others out.
                if (!kTwoS) {
                    ok = waits(s_ready, c, kErrEpilogue);
                    if (!ok) break;
                }
                if (!fed) make_p(c, n);
                ok = waits(a_done, c, kErrEpilogue);
                if (!ok) break;
                if (c > 0) {
                    if (kTwoS) {  // (one place for S: it is free, so P Y is done)
                        ok = waits(o_ready, c - 1, kErrEpilogue);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    float v[kN];
                    tmem_ldn<kN>(lane_base + kTmemO + col0, v);
                    tmem_ld_wait();
                    write_out(c - 1, Sh::x(c), v);
                } else {
                    warp_arrive(o_free, lane);
                }
                if (fed) make_p(c, n);
                // --------------------------------------------- C: Z M
                ok = waits(m_ready, c, kErrEpilogue);
                if (!ok) break;
                tc_fence_after();
                {
                    const int w = P.reverse ? n - row - first : row + 1;
                    float v[kN];
                    tmem_ldn<kN>(lane_base + kTmemO + col0, v);
                    tmem_ldn<kN>(lane_base + kTmemM + col0, mv);
                    tmem_ld_wait();
                    // rows after the end may hold NaN; they are not stored
                    tmem_st_scaled<kN>(lane_base + kTmemO + col0, v, row < n ? pw[w] * (kUp * kLoUp<T>) : 0.f);
                    tmem_st_wait();
                }
                tc_fence_before();
                warp_arrive(p_done, lane);
                rescale();
                if (lane == 0) {
                    bulk_wait_read_all();  // X's place is free when out has left it
                    mbar_arrive(smem_u32(&x_free[c & 1]));
                }
                __syncwarp();
            }
        }
        if (STATE && ok) {
            ok = waits(m_ready, n_chunks - 1, kErrEpilogue);
            if (ok) {
                tc_fence_after();
                tmem_ldn<kN>(lane_base + kTmemM + col0, mv);
                tmem_ld_wait();
                rescale();
            }
        }
        if constexpr (kStacked) {
            if (ok && m_out) {  // the two sums joined; M's parts are not read any more
                const uint32_t at = base + Sh::oM + (uint32_t)((row & 63) * 64 + col0) * 4u;
                if (w4 >= 2) {
#pragma unroll
                    for (int i = 0; i < kN; i += 4)
                        sts128(at + i * 4, __float_as_uint(mv[i]), __float_as_uint(mv[i + 1]), __float_as_uint(mv[i + 2]),
                               __float_as_uint(mv[i + 3]));
                    warp_arrive(sum_ready, lane);
                } else {
                    ok = waits(sum_ready, 0, kErrEpilogue);
#pragma unroll
                    for (int i = 0; i < kN; i += 4) {
                        uint32_t u[4];
                        lds128(at + i * 4, u);
#pragma unroll
                        for (int k = 0; k < 4; ++k) mv[i + k] += __uint_as_float(u[k]);
                    }
                }
            }
        }
        // What is not finite in x or y leaves its trace in M: then the outputs
        // are formed once more (also those of a walk whose M began so).
        bool once_more = false;
        if constexpr (!STATE) {
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kN; i += 2) t = __ffma2_rn(make_float2(mv[i], mv[i + 1]), make_float2(0.f, 0.f), t);
            once_more = workers_any(row < P.Da && !(t.x + t.y == 0.f));
            if (once_more && threadIdx.x == 0) again |= Q.quota ? 1u << (run / Q.chunks - run0 / Q.chunks) : 1u;
        }
        if (ok && m_out && row < P.Da && (!once_more || handed)) {  // (m_in may be m_out, and is read once more)
            const float last = P.reverse && last_piece ? pw[1] : 1.f;
#pragma unroll
            for (int i = 0; i < kN; ++i) mv[i] *= last;
            float* to = m_out + (int64_t)row * P.Db + col0;
            if (wide) {
#pragma unroll
                for (int i = 0; i < kN; i += 8)
                    if (col0 + i < P.Db) store8(to + i, mv + i);
            } else {
#pragma unroll
                for (int i = 0; i < kN; ++i)
                    if (col0 + i < P.Db) to[i] = mv[i];
            }
        }
        if constexpr (!STATE)
            if (ok && waits(o_ready, n_chunks - 1, kErrEpilogue)) {
                tc_fence_after();
                float v[kN];
                tmem_ldn<kN>(lane_base + kTmemO + col0, v);
                tmem_ld_wait();
                write_out(n_chunks - 1, Sh::x(n_chunks - 1), v);
            }
        if (!STATE && lane == 0) bulk_wait_all();
        __syncwarp();
        tmem_st_wait();  // stores that a warp which gave up has not waited for
        if constexpr (kHalf)
            if (!(top <= kF16Max)) P.flags[bh] = 1;
    } else if (warp == kLaWorkers) {
        // ------------------------------------------------------- TMA loads
        if (lane == 0) {
            int nx = 0, ny = 0;  // fills issued
            bool ok = true;
            auto fill = [&](const CUtensorMap* map, uint64_t& full, uint32_t place, int D, int t0) {
                for (int k = 0; k < D / 64; ++k) tma_load_4d(base + place + k * 16384u, map, smem_u32(&full), k * 64, t0, h, b);
            };
            // a place was last used by the tile five before: X of two chunks
            // ago for Z, Y of two chunks ago for X, the last chunk's Z for Y
            for (int c = 0; c < n_chunks; ++c) {
                const int t0 = s0 + chunk_at(c) * kC, s = c & 1;
                ok = c < 2 || (mbar_wait(smem_u32(&x_free[s]), ((c >> 1) - 1) & 1, kErrProducer, &abort_flag, P.wait_ns) &&
                               mbar_wait(smem_u32(&y_free[s]), ((c >> 1) - 1) & 1, kErrProducer, &abort_flag, P.wait_ns));
                if (!ok) break;
                mbar_expect_tx(smem_u32(&x_full[s]), 256 * DA * (STATE ? 1 : 2));
                if (!STATE) fill(&P.tz, x_full[s], Sh::z(c), DA, t0);
                fill(&P.tx, x_full[s], Sh::x(c), DA, t0);
                ++nx;
                ok = STATE || c < 1 || mbar_wait(smem_u32(&z_free[s ^ 1]), ((c - 1) >> 1) & 1, kErrProducer, &abort_flag, P.wait_ns);
                if (!ok) break;
                mbar_expect_tx(smem_u32(&y_full[s]), 256 * DB);
                fill(&P.ty, y_full[s], Sh::y(c), DB, t0);
                ++ny;
            }
            // what was issued must land before the CTA exits or makes its
            // barriers anew: the last fills of each barrier.  Always, as
            // another warp may give up after the last fill, when no wait of
            // this one fails any more; on a walk that is done they have landed.
            for (int i = max(0, nx - 2); i < nx; ++i) mbar_drain(smem_u32(&x_full[i & 1]), (i >> 1) & 1);
            for (int i = max(0, ny - 2); i < ny; ++i) mbar_drain(smem_u32(&y_full[i & 1]), (i >> 1) & 1);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- MMA issue
        // the whole warp walks and waits; one elected lane issues
        auto wait1 = [&](uint64_t& bar, int parity) { return waits(bar, parity, kErrMma); };
        // D += A B over the chunk's tokens, A = hi + lo in TMEM.  f16: D comes
        // in lo's scale, takes the lo products and then, scaled down, the others
        auto by_y = [&](uint32_t d, uint32_t at, int c) {
            const uint64_t yd = desc_mn(base + Sh::y(c), 16384);
            auto ad = [&](int k) { return at + (k / 2) * 32 + (k & 1) * 8; };
            if constexpr (kDown == 0) {
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) {
                    mma_ts_one(d, ad(k), yd + 128 * k, P.idesc_n);
                    mma_ts_one(d, ad(k) + 16, yd + 128 * k, P.idesc_n);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) mma_ts_one(d, ad(k) + 16, yd + 128 * k, P.idesc_n);
                mma_ts_down<kDown>(d, ad(0), yd, P.idesc_n);
#pragma unroll
                for (int k = 1; k < kC / 16; ++k) mma_ts_one(d, ad(k), yd + 128 * k, P.idesc_n);
            }
        };
        auto form_s = [&](int c) {  // false where a wait gave up
            const uint64_t zd = smem_desc_sw128(base + Sh::z(c)), xd = smem_desc_sw128(base + Sh::x(c));
            if (!wait1(x_full[c & 1], c >> 1)) return false;
            // the P that was in its place has been multiplied
            const int before = kTwoS ? c - 2 : c - 1;
            if (before >= 0 && !wait1(o_ready, before)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DA / 16; ++k) {
                const uint32_t o = (k / 4) * 1024 + (k & 3) * 2;  // 64 columns on: 16384 bytes; 16: 32 bytes
                mma_ss_one(tmem + p_at(c), zd + o, xd + o, P.idesc_s, k > 0);
            }
            commit_one(s_ready);
            commit_one(x_free[c & 1]);
            return true;
        };
        bool ok = STATE || form_s(0);
        int c = 0;
        for (; c < n_chunks && ok; ++c) {
            const int s = c & 1;
            if (!STATE && !kTwoS && c > 0 && !form_s(c)) break;
            if (!wait1(y_full[s], c >> 1) || !wait1(a_done, c)) break;
            tc_fence_after();
            if constexpr (kStacked) {
                const uint64_t xd = desc_mn(x_smem(c), 16384), yd = desc_mn(base + Sh::y(c), 16384);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k) mma_ss_one(tmem + kTmemM, xd + 128 * k, yd + 128 * k, P.idesc_n | (1u << 15), 1);
            } else {
                by_y(tmem + kTmemM, tmem + x_at(c), c);
            }
            if constexpr (!STATE) {
                if (!wait1(o_free, c)) break;
                tc_fence_after();
                const uint64_t zd = smem_desc_sw128(base + Sh::z(c));
                const uint64_t mh = desc_mn(base + Sh::oM, DA * 128), ml = desc_mn(base + Sh::oM + Sh::kM, DA * 128);
                auto zo = [&](int k) { return zd + (k / 4) * 1024 + (k & 3) * 2; };
                if constexpr (kDown == 0) {
#pragma unroll
                    for (int k = 0; k < DA / 16; ++k) {
                        mma_ss_one(tmem + kTmemO, zo(k), mh + 128 * k, P.idesc_n, k > 0);
                        mma_ss_one(tmem + kTmemO, zo(k), ml + 128 * k, P.idesc_n, 1);
                        if constexpr (kStacked) mma_ss_one(tmem + kTmemO, zo(k), ml + (Sh::kM >> 4) + 128 * k, P.idesc_n, 1);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < DA / 16; ++k) {
                        mma_ss_one(tmem + kTmemO, zo(k), ml + 128 * k, P.idesc_n, k > 0);
                        if constexpr (kStacked) mma_ss_one(tmem + kTmemO, zo(k), ml + (Sh::kM >> 4) + 128 * k, P.idesc_n, 1);
                    }
                    mma_ss_down<kDown>(tmem + kTmemO, zo(0), mh, P.idesc_n);
#pragma unroll
                    for (int k = 1; k < DA / 16; ++k) mma_ss_one(tmem + kTmemO, zo(k), mh + 128 * k, P.idesc_n, 1);
                }
                commit_one(z_free[s]);
                commit_one(m_ready);  // the new M and Z M
                // (every warp has seen this chunk's s_ready: o_free follows it)
                if (kTwoS && c + 1 < n_chunks && !form_s(c + 1)) break;
                if (!wait1(p_done, c)) break;
                tc_fence_after();
                by_y(tmem + kTmemO, tmem + p_at(c), c);
                commit_one(o_ready);
            } else {
                commit_one(m_ready);
            }
            commit_one(y_free[s]);
        }
        // no MMA may be in flight when TMEM is released
        commit_one(drain_bar);
        mbar_drain(smem_u32(&drain_bar), 0);
        // nor any arrival, before the barriers are made anew
        if (c == n_chunks)
            for (int i = max(0, c - 2); i < c; ++i) {
                mbar_drain(smem_u32(&y_free[i & 1]), (i >> 1) & 1);
                mbar_drain(smem_u32(&x_free[i & 1]), (i >> 1) & 1);
                if (!STATE) mbar_drain(smem_u32(&z_free[i & 1]), (i >> 1) & 1);
            }
        __syncwarp();
    }
    }
    // nothing of the piece is in flight any more
    tc_fence_before();
    if (__syncthreads_or(abort_flag)) break;
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (n_chunks > 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_inval(smem_u32(&y_full[i]));
                mbar_inval(smem_u32(&y_free[i]));
                mbar_inval(smem_u32(&z_free[i]));
                mbar_inval(smem_u32(&x_full[i]));
                mbar_inval(smem_u32(&x_free[i]));
            }
            mbar_inval(smem_u32(&s_ready));
            mbar_inval(smem_u32(&a_done));
            mbar_inval(smem_u32(&p_done));
            mbar_inval(smem_u32(&o_ready));
            mbar_inval(smem_u32(&m_ready));
            mbar_inval(smem_u32(&o_free));
            mbar_inval(smem_u32(&sum_ready));
            mbar_inval(smem_u32(&drain_bar));
        }
        if (handed) set_done(Q.done + me);  // every thread's part was stored before the barrier above
    }
    } while (run > run0);

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kLaWorkers + 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    if constexpr (!STATE)
        if (again && !abort_flag && warp < kLaWorkers) la_token_by_token<T>(Q, number, again, reinterpret_cast<float*>(smem_raw));
}

// cur <- decay^n cur + sum, element by element along the walk.
__global__ void __launch_bounds__(256) la_chain(const __grid_constant__ LaChainBatch Q) {
    const LaChain& P = Q.core[blockIdx.y];
    const int64_t msize = (int64_t)P.Da * P.Db, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= msize * Q.BH) return;
    const int bh = (int)(i / msize);
    const int64_t e = i % msize;
    const int len = Q.lengths ? max(0, min(Q.T, Q.lengths[bh / Q.H])) : Q.T;
    const float g = la_log_decay(Q.log_decay[bh % Q.H]);
    float cur = P.m_in ? P.m_in[bh * msize + (P.m_in_t ? (e % P.Db) * P.Da + e / P.Db : e)] : 0.f;
    auto seg_of = [&](int k) { return P.reverse ? Q.segs - 1 - k : k; };
    const int64_t step = (int64_t)Q.BH * msize;
    for (int k0 = 0; k0 < Q.segs; k0 += 8) {  // eight loads in flight
        float sum[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = k0 + k < Q.segs ? P.sums[seg_of(k0 + k) * step + i] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k0 + k >= Q.segs) break;
            const int seg = seg_of(k0 + k), s0 = seg * Q.seg_tokens;
            const int n = max(0, min(len, min(Q.T, s0 + Q.seg_tokens)) - s0);
            P.sums[seg * step + i] = cur;
            if (n > 0) cur = fmaf(expf((float)(n - (P.reverse && s0 + n == len ? 1 : 0)) * g), cur, sum[k]);
        }
    }
    if (P.m_out) P.m_out[i] = P.reverse && len > 0 ? expf(g) * cur : cur;
}

bool map_tensor(CUtensorMap* m, const LaCore& c, const void* p, const int64_t (&st)[3], int D, int cols = 64, int rows = kC) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)c.T, (cuuint64_t)c.H, (cuuint64_t)c.B};
    // an axis of one element may have any stride
    const cuuint64_t strides[3] = {c.T > 1 ? (cuuint64_t)st[1] * 2 : 256, c.H > 1 ? (cuuint64_t)st[2] * 2 : 256,
                                   c.B > 1 ? (cuuint64_t)st[0] * 2 : 256};
    const cuuint32_t box[4] = {(cuuint32_t)cols, (cuuint32_t)rows, 1, 1}, es[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                    : CU_TENSOR_MAP_SWIZZLE_32B;
    return enc(m, c.dtype == CT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
               const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA can read (or write) the tensor where it is.
bool tma_ok(const LaCore& c, const void* p, const int64_t (&st)[3]) {
    const int64_t n[3] = {c.B, c.T, c.H};
    if ((uintptr_t)p % 16 != 0) return false;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] <= 0 || st[i] % 8 != 0 || st[i] >= (1ll << 38))) return false;
    return true;
}

template <typename T, int DA, int DB, bool STATE>
cudaError_t launch_k(const LaTcBatch& Q, int cores, cudaStream_t s) {
    auto k = la_chunks<T, DA, DB, STATE>;
    constexpr int bytes = (int)LaShape<DA, DB>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = Q.quota ? (unsigned)(((int64_t)Q.walks * Q.chunks + Q.quota - 1) / Q.quota) : (unsigned)(Q.ctas * cores);
    k<<<grid, kLaThreads, bytes, s>>>(Q);
    return cudaGetLastError();
}

template <typename T, bool STATE>
cudaError_t launch_d(const LaTcBatch& Q, int cores, cudaStream_t s) {
    const LaTcParams& P = Q.core[0];
    if (P.Da <= 64) return P.Db <= 64 ? launch_k<T, 64, 64, STATE>(Q, cores, s) : launch_k<T, 64, 128, STATE>(Q, cores, s);
    return P.Db <= 64 ? launch_k<T, 128, 64, STATE>(Q, cores, s) : launch_k<T, 128, 128, STATE>(Q, cores, s);
}

template <bool STATE>
cudaError_t launch_t(const LaTcBatch& Q, int cores, int dtype, cudaStream_t s) {
    return dtype == CT_BF16 ? launch_d<__nv_bfloat16, STATE>(Q, cores, s) : launch_d<__half, STATE>(Q, cores, s);
}

// Segments of a sequence, and the tokens of one: as many as fill the GPU once
// with one CTA each, of at least four chunks.  A segment's X and Y are read
// twice and its matrices pass through memory, so two segments do not pay
// (2048 tokens, 76 heads of 128 in two: 90 us; 77 in one: 66; of 64: 55 and
// 49), three do (39 heads of 128: 64 us, of 64: 42; four, 38 heads: 54 and 37;
// 8192 tokens, 50 heads of 128 in three: 161 us; 77 in one: 235).
void split(int64_t heads, int64_t T, int sm_count, int* segs, int* tokens) {
    const int64_t chunks = (T + kC - 1) / kC;
    int64_t want = std::min<int64_t>(sm_count / std::max<int64_t>(1, heads), chunks / 4);
    if (want < 3) want = 1;
    const int64_t per = (chunks + want - 1) / want;
    *tokens = (int)(per * kC);
    *segs = (int)((chunks + per - 1) / per);
}

// More walks than SMs: the chunks a CTA gets where walks are shared, 0 where
// each has its own CTA and the last turn leaves SMs empty.  A further piece
// costs a CTA 5 to 8 us (tables, first loads, the matrix through memory), so
// the chunks saved have to be two and a sixth of the quota.  bf16, 2048
// tokens, us shared / two turns: 160 heads of 128 86 / 138, 228 125 / 138, 256
// (27 chunks of 32) 146 / 138; 192 heads of 64 80 / 101, 256 100 / 101; 300
// tokens, 192 heads of 128 38 / 43.
int share(int64_t walks, int64_t T, int sm_count) {
    const int64_t chunks = (T + kC - 1) / kC;
    if (walks <= sm_count || walks * chunks >= (1ll << 30)) return 0;
    const int64_t quota = (walks * chunks + sm_count - 1) / sm_count, turns = (walks + sm_count - 1) / sm_count;
    return turns * chunks - quota >= 2 + quota / 6 ? (int)quota : 0;
}

size_t shared_bytes(int64_t msize, int sm_count) {
    return round256((size_t)sm_count * msize * sizeof(float)) + round256((size_t)(2 * sm_count + 1) * sizeof(unsigned));
}

size_t core_bytes(int64_t BH, int64_t msize, int segs, int dtype) {
    const size_t m = (size_t)BH * msize * sizeof(float);
    return (segs > 1 ? round256(m * segs) : 0) + (dtype == CT_F16 ? round256(m) + round256((size_t)BH * sizeof(int)) : 0);
}

}  // namespace

bool la_tc_fits(int64_t T, int64_t Dk, int64_t Dv, int dtype) {
    if ((dtype != CT_BF16 && dtype != CT_F16) || Dk > 128 || Dv > 128 || T <= kLaScanTokens) return false;
    DeviceInfo d;
    return device_info(&d) != cudaSuccess || (d.cc_major == 10 && d.cc_minor == 3);
}

bool la_tc_supports(const LaCore& c) {
    return la_tc_fits(c.T, c.Da, c.Db, c.dtype) && c.B * c.H < (1ll << 22) && tma_ok(c, c.z, c.zs) && tma_ok(c, c.x, c.xs) &&
           tma_ok(c, c.y, c.ys) && (!c.out || tma_ok(c, c.out, c.os));
}

size_t la_tc_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, int dtype, int backward) {
    if (!la_tc_fits(T, Dk, Dv, dtype)) return 0;
    DeviceInfo d;
    int sm = 152, tokens;
    if (device_info(&d) == cudaSuccess) sm = d.sm_count;
    size_t most = 0;
    // however many of the gradients are asked for
    for (int cores = 1; cores <= (backward ? 3 : 1); ++cores) {
        int segs;
        split(B * H * cores, T, sm, &segs, &tokens);
        const size_t extra = share(B * H * cores, T, sm) ? shared_bytes(Dk * Dv, sm) : 0;
        most = std::max(most, cores * core_bytes(B * H, Dk * Dv, segs, dtype) + extra);
    }
    return most;
}

cudaError_t launch_la_chain(const LaChainBatch& C, int n, cudaStream_t s) {
    const int64_t elements = (int64_t)C.BH * C.core[0].Da * C.core[0].Db;
    la_chain<<<dim3((unsigned)((elements + 255) / 256), n), 256, 0, s>>>(C);
    return cudaGetLastError();
}

cudaError_t launch_la_tc(const LaCore* cores, int n, void* workspace, cudaStream_t s) {
    DeviceInfo d;
    cudaError_t e = device_info(&d);
    if (e != cudaSuccess) return e;
    const LaCore& one = cores[0];
    const int64_t BH = one.B * one.H, msize = (int64_t)one.Da * one.Db;
    int segs, seg_tokens;
    split(BH * n, one.T, d.sm_count, &segs, &seg_tokens);
    // f16: a last matrix that takes the first one's place is kept aside until
    // it is known that no value left the type's range (the second try reads
    // the first one)
    int* flags[3] = {};
    float* kept[3] = {};
    LaTcBatch Q;
    LaChainBatch C;
    std::memset(&Q, 0, sizeof(Q));
    std::memset(&C, 0, sizeof(C));
    Q.ctas = (int)(BH * segs);
    C.log_decay = one.log_decay;
    C.lengths = one.lengths;
    C.T = one.T;
    C.H = one.H;
    C.BH = (int)BH;
    C.seg_tokens = seg_tokens;
    C.segs = segs;
    char* ws = static_cast<char*>(workspace);
    for (int i = 0; i < n; ++i) {
        const LaCore& c = cores[i];
        LaTcParams& P = Q.core[i];
        if (!map_tensor(&P.tz, c, c.z, c.zs, c.Da) || !map_tensor(&P.tx, c, c.x, c.xs, c.Da) || !map_tensor(&P.ty, c, c.y, c.ys, c.Db) ||
            (c.out && !map_tensor(&P.to, c, c.out, c.os, c.Db, c.Db <= 64 ? 16 : 32, 32)))
            return cudaErrorInvalidValue;
        C.core[i] = {nullptr, c.m_in, c.m_out, c.m_in_t, c.reverse, c.Da, c.Db};
        if (segs > 1) {
            C.core[i].sums = reinterpret_cast<float*>(ws);
            ws += round256((size_t)BH * msize * segs * sizeof(float));
        }
        if (c.dtype == CT_F16) {
            if (c.m_out && c.m_out == c.m_in) kept[i] = C.core[i].m_out = reinterpret_cast<float*>(ws);
            ws += round256((size_t)BH * msize * sizeof(float));
            flags[i] = reinterpret_cast<int*>(ws);
            ws += round256((size_t)BH * sizeof(int));
            e = cudaMemsetAsync(flags[i], 0, (size_t)BH * sizeof(int), s);
            if (e != cudaSuccess) return e;
        }
        P.out = c.out;
        P.z = c.z;
        P.x = c.x;
        P.y = c.y;
        for (int k = 0; k < 3; ++k) {
            P.os[k] = c.os[k];
            P.zs[k] = c.zs[k];
            P.xs[k] = c.xs[k];
            P.ys[k] = c.ys[k];
        }
        P.log_decay = c.log_decay;
        P.lengths = c.lengths;
        P.flags = flags[i];
        P.mscale = c.mscale;
        P.oscale = c.oscale;
        P.reverse = c.reverse;
        P.T = c.T;
        P.H = c.H;
        P.Da = c.Da;
        P.Db = c.Db;
        P.BH = (int)BH;
        P.segs = segs;
        P.seg_tokens = seg_tokens;
        P.wait_ns = wait_limit_ns();
        const uint32_t type = c.dtype == CT_BF16 ? 1u : 0u;
        const uint32_t common = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(128 >> 4) << 24);  // D f32, M = 128
        P.idesc_s = common | ((uint32_t)(kC >> 3) << 17);
        P.idesc_n = common | (1u << 16) | ((uint32_t)((c.Db <= 64 ? 64 : 128) >> 3) << 17);
        if (segs > 1) {
            P.m_out = C.core[i].sums;
        } else {
            P.m_in = c.m_in;
            P.m_in_t = c.m_in_t;
            P.m_out = C.core[i].m_out;
            P.final = 1;
        }
    }
    Q.quota = share(BH * n, one.T, d.sm_count);
    if (Q.quota) {
        Q.chunks = (int)((one.T + kC - 1) / kC);
        Q.walks = (int)(BH * n);
        Q.handed = reinterpret_cast<float*>(ws);
        Q.done = reinterpret_cast<unsigned*>(ws + round256((size_t)d.sm_count * msize * sizeof(float)));
        Q.read = Q.done + d.sm_count;
        Q.started = Q.read + d.sm_count;
        e = cudaMemsetAsync(Q.done, 0, (size_t)(2 * d.sm_count + 1) * sizeof(unsigned), s);
        if (e != cudaSuccess) return e;
    }
    if (segs > 1) {
        e = launch_t<true>(Q, n, one.dtype, s);
        if (e != cudaSuccess) return e;
        e = launch_la_chain(C, n, s);
        if (e != cudaSuccess) return e;
        for (int i = 0; i < n; ++i) {
            Q.core[i].m_in = C.core[i].sums;
            Q.core[i].m_in_seg = 1;
            Q.core[i].m_out = nullptr;
        }
    }
    if (one.out) e = launch_t<false>(Q, n, one.dtype, s);
    else if (segs == 1) e = launch_t<true>(Q, n, one.dtype, s);  // only the last matrix is asked for
    for (int i = 0; i < n && e == cudaSuccess && flags[i]; ++i) e = launch_la_scan_again(cores[i], flags[i], kept[i], s);
    return e;
}

cudaError_t la_error_word(unsigned int* v, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(v, g_device_error, sizeof(*v));
    if (e == cudaSuccess && clear && *v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace ct
