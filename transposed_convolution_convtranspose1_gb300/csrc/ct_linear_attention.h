// ct_linear_attention.h -- the one recurrence behind linear attention with a
// decay and all of its gradients, and the kernels that run it.
//
//   M_t   = decay * M_{t-1} + mscale * x_t y_t^T          (M: Da x Db, fp32)
//   out_t = oscale * M_t^T z_t
//
// forward in time over the first `length` tokens of each sequence, or
// backward (reverse) from the last of them to the first:
//   o  : x = k,  y = v,  z = q,  forward,  M starts from the state
//   dq : x = v,  y = k,  z = do, forward,  M starts from the state transposed
//   dv : x = q,  y = do, z = k,  reverse,  M starts from the last state's gradient
//   dk : x = do, y = q,  z = v,  reverse,  M starts from that transposed
// Backward in time the starting matrix enters the last token undecayed (it is
// a gradient of the state after that token) and the matrix left after the
// first token is decayed once more (it is a gradient of that token's state,
// asked for the one before it).
#pragma once

#include "ct_internal.h"

namespace ct {

constexpr int kLaMaxD = 256;  // head sizes

// The logarithm of a decay as the kernels multiply it: a finite one, as
// exp(0 * g) must be 1 for a decay of zero (g = -infinity) too.  A comparison,
// not a maximum, so that NaN stays NaN.
__device__ __forceinline__ float la_log_decay(float g) { return g < -1e30f ? -1e30f : g; }

struct LaCore {
    const void *z, *x, *y;
    void* out;
    int64_t zs[3], xs[3], ys[3], os[3];  // element strides of batch, token, head; the last axis is dense
    int Da, Db;
    const float* m_in;   // [B][H][Da][Db] ([B][H][Db][Da] if m_in_t), or null: zero
    int m_in_t;
    float* m_out;        // [B][H][Da][Db], or null
    const float* log_decay;  // [H]
    const int32_t* lengths;  // [B], or null: T each
    float mscale, oscale;
    int reverse;
    int64_t B;
    int T, H;
    int dtype;
};

// Sequences cut into segments: the matrix before each segment from the
// segments' own sums ([seg][B * H][Da][Db]), in place, for up to three walks of
// one Da * Db; the last one is the walk's result (m_out, or null).
struct LaChain {
    float* sums;
    const float* m_in;
    float* m_out;
    int m_in_t, reverse, Da, Db;
};
struct LaChainBatch {
    LaChain core[3];
    const float* log_decay;
    const int32_t* lengths;
    int T, H, BH, seg_tokens, segs;
};
cudaError_t launch_la_chain(const LaChainBatch& c, int n, cudaStream_t stream);

// Sequences of at most this many tokens go token by token.  A chunk costs the
// same for 33 tokens as for 128, a scan grows by the token (bf16, us on the
// GPU, scan / chunks: 64 heads of 64, 9.9 / 10.6 at 32 tokens, 12.8 / 11.0 at
// 48; of 128, 13.4 / 14.7 at 24, 15.9 / 14.3 at 32; 512 heads, several turns of
// chunks: of 64, 23.8 / 40.1 at 32, 40.4 / 40.3 at 64; of 128, 41.8 / 54.6 at
// 16, 69.8 / 57.2 at 24).
constexpr int kLaScanTokens = 32;

// Token by token on CUDA cores, the matrix in registers
// (ct_linear_attention.cu); long sequences on few heads in segments.
size_t la_scan_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Da, int64_t Db);
cudaError_t launch_la_scan(const LaCore& c, void* workspace, cudaStream_t stream);
// The same again for the heads whose flag ([B * H]) is not 0, in one segment;
// of the others only m_out is written, copied from `kept` where given.
cudaError_t launch_la_scan_again(const LaCore& c, const int* flags, const float* kept, cudaStream_t stream);

// In chunks on the tensor cores (ct_linear_attention_tc.cu): 16-bit types,
// head sizes up to 128, tensors that TMA can address.
bool la_tc_fits(int64_t T, int64_t Dk, int64_t Dv, int dtype);
bool la_tc_supports(const LaCore& c);
size_t la_tc_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, int dtype, int backward);
// Up to three walks at once, of one (Da, Db) up to the tiles' 64 or 128 and
// one Da * Db, each with an output or none with one.
cudaError_t launch_la_tc(const LaCore* cores, int n, void* workspace, cudaStream_t stream);
cudaError_t la_error_word(unsigned int* v, bool clear);

}  // namespace ct
