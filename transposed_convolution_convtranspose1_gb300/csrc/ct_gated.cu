// ct_gated.cu -- the gated projection of a feed-forward layer and its
// gradients: operands, workspace and the order of the products
// (ct_gated_tc.cu) behind them.
//
//   g = x Wg, u = x Wu, y = act(g) * u           x [rows, C], W [C, F]
//   dg = dy * u * act'(g), du = dy * act(g)      (g and u formed again)
//   dx = dg Wg^T + du Wu^T,  dWg = x^T dg,  dWu = x^T du
//
// 16-bit operands go to the tensor cores as they lie in memory, whichever axis
// is dense, where pointers and row strides are multiples of 16 bytes (what TMA
// asks for); others are copied into aligned rows first.
//
// An fp32 factor becomes three bf16 numbers, a = a1 + a2 + a3: each the nearest
// to what the ones before it leave, 8 bits at a time, which keeps all 24 bits (of
// factors from 2^-110 on: bf16's smallest step is 2^-133).
// a b = a2 b2 + a1 b3 + a3 b1 + a1 b2 + a2 b1 + a1 b1 leaves out terms below
// 2^-25 of the product.  (Two TF32 parts take as long, need copies that are
// dense along K, transposed where they are not, and came out 4 times as far off:
// 2.5e-6 of the result's size with 512 terms.)
#include <algorithm>
#include <type_traits>

#include "ct_gated.h"
#include "ct_internal.h"
#include "ct_types.cuh"

namespace ct {
namespace {

// A matrix as a call gives it.
struct Matrix {
    const void* p;
    int64_t rows, cols, s0, s1;  // sizes, element strides; one of the strides is 1
    Matrix turned() const { return {p, cols, rows, s1, s0}; }
};

// Matrices to lay out anew, up to three in one launch: aligned copies of 16-bit
// or fp32 ones, or an fp32 one's three bf16 parts.  Rows stay rows.
struct Layouts {
    Matrix src[3];
    void* dst[3];
    size_t part[3];  // bytes from a part to the next
    int64_t pitch[3];
    int n = 0;
};

constexpr int kSpan = 256;  // columns a warp takes at a time

// Bound by memory: the parts of 4096 x 2048 and twice 2048 x 8192 fp32 (420 MB read
// and written) 66 us, 6360 GB/s, 95% of the copy rate.
// E: bytes of an element.
template <int E, bool SPLIT>
__global__ void __launch_bounds__(256) gated_lay_out(Layouts A) {
    using T = typename std::conditional<E == 4, float, unsigned short>::type;
    const int lane = threadIdx.x & 31, m = blockIdx.y;
    const Matrix src = A.src[m];
    const T* p = static_cast<const T*>(src.p);
    const int64_t pitch = A.pitch[m], spans = (src.cols + kSpan - 1) / kSpan, n = spans * src.rows;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
        const int64_t r = i / spans, c = (i - r * spans) * kSpan + lane;
        T v[kSpan / 32];
#pragma unroll
        for (int j = 0; j < kSpan / 32; ++j) v[j] = c + j * 32 < src.cols ? p[r * src.s0 + c + j * 32] : T(0);
#pragma unroll
        for (int j = 0; j < kSpan / 32; ++j) {
            if (c + j * 32 >= src.cols) break;
            const int64_t at = r * pitch + c + j * 32;
            if constexpr (SPLIT) {
                char* d = static_cast<char*>(A.dst[m]);
                float rest = v[j];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    __nv_bfloat16 h = __float2bfloat16_rn(rest);
                    // close to the largest fp32 number the nearest one would be infinity
                    if (k == 0 && __hisinf(h)) h = __float2bfloat16_rz(rest);
                    reinterpret_cast<__nv_bfloat16*>(d + k * A.part[m])[at] = h;
                    rest = isfinite(v[j]) ? rest - __bfloat162float(h) : 0.f;
                }
            } else {
                static_cast<T*>(A.dst[m])[at] = v[j];
            }
        }
    }
}

int64_t pitch_of(int64_t inner, size_t eb) { return (inner + 16 / eb - 1) / (16 / eb) * (16 / eb); }
size_t bytes_of(int64_t outer, int64_t inner, size_t eb) { return ((size_t)outer * pitch_of(inner, eb) * eb + 255) / 256 * 256; }

// What TMA can read in place: the inner axis dense, pointer and row stride
// multiples of 16 bytes, rows that do not overlap.
bool in_place(const Matrix& m, size_t eb) {
    return (uintptr_t)m.p % 16 == 0 && (m.rows <= 1 || (m.s0 >= m.cols && m.s0 * eb % 16 == 0));
}

// Hands out a call's workspace in order.
struct Room {
    char* p;
    size_t used = 0;
    void* take(size_t n) {
        void* q = p + used;
        used += n;
        return q;
    }
};

struct Gated {
    Matrix x, wg, wu, dy, dx, dwg, dwu;  // dx, dwg and dwu are written
    int64_t y_stride;
    void* y;
    bool f_dense;  // of the weights
    int64_t rows, C, F;
    int act, dtype, sm;
    float alpha;
    size_t eb;
};

// An operand with dense, aligned rows: m itself, or a copy that `todo` makes.
GemmOperand operand(const Matrix& m, const Gated& A, Room& room, Layouts& todo) {
    const int64_t pitch = pitch_of(m.cols, A.eb);
    if (in_place(m, A.eb)) return {m.p, m.cols, m.rows, m.rows <= 1 ? pitch : m.s0};
    void* d = room.take(bytes_of(m.rows, m.cols, A.eb));
    todo.src[todo.n] = m;
    todo.dst[todo.n] = d;
    todo.pitch[todo.n++] = pitch;
    return {d, m.cols, m.rows, pitch};
}

// The three parts of an fp32 matrix.
void split(GemmOperand* out, const Matrix& m, Room& room, Layouts& todo) {
    const size_t n = bytes_of(m.rows, m.cols, 2);
    char* d = static_cast<char*>(room.take(3 * n));
    todo.src[todo.n] = m;
    todo.dst[todo.n] = d;
    todo.part[todo.n] = n;
    todo.pitch[todo.n++] = pitch_of(m.cols, 2);
    for (int i = 0; i < 3; ++i) out[i] = {d + i * n, m.cols, m.rows, pitch_of(m.cols, 2)};
}

cudaError_t lay_out(const Layouts& todo, bool splits, const Gated& A, cudaStream_t s) {
    if (todo.n == 0) return cudaSuccess;
    int64_t most = 1;
    for (int i = 0; i < todo.n; ++i) most = std::max(most, (todo.src[i].cols + kSpan - 1) / kSpan * todo.src[i].rows);
    const dim3 grid((unsigned)std::min<int64_t>((most + 7) / 8, 8 * A.sm), (unsigned)todo.n);
    if (splits) gated_lay_out<4, true><<<grid, 256, 0, s>>>(todo);
    else if (A.eb == 4) gated_lay_out<4, false><<<grid, 256, 0, s>>>(todo);
    else gated_lay_out<2, false><<<grid, 256, 0, s>>>(todo);
    return cudaGetLastError();
}

// Parts of `pairs` products of split operands, the small terms of all pairs
// first: what the accumulator drops of a sum goes by its size.
void split_parts(Gemm& g, int pairs) {
    constexpr int a[6] = {1, 0, 2, 0, 1, 0}, b[6] = {1, 2, 0, 1, 0, 0};
    g.parts = 6 * pairs;
    for (int j = 0; j < 6; ++j)
        for (int i = 0; i < pairs; ++i) {
            g.a_part[j * pairs + i] = 3 * i + a[j];
            g.b_part[j * pairs + i] = 3 * i + b[j];
        }
}

// g and u: the operands of the forward product and of the gradients' first.
cudaError_t first_product(Gemm& g, const Gated& A, Room& room, cudaStream_t s) {
    const Matrix wg = A.f_dense ? A.wg : A.wg.turned(), wu = A.f_dense ? A.wu : A.wu.turned();
    const bool wide = A.dtype == CT_F32;
    g.dtype = A.dtype;
    g.M = A.rows;
    g.N = A.F;
    g.K = A.C;
    g.act = A.act;
    g.alpha = A.alpha;
    g.b_mn = A.f_dense;
    Layouts todo;
    if (wide) {
        g.n_a = g.b_block = 3;
        g.n_b = 6;
        split_parts(g, 1);
        split(g.a, A.x, room, todo);
        split(g.b, wg, room, todo);
        split(g.b + 3, wu, room, todo);
    } else {
        g.n_a = g.b_block = 1;
        g.n_b = 2;
        g.a[0] = operand(A.x, A, room, todo);
        g.b[0] = operand(wg, A, room, todo);
        g.b[1] = operand(wu, A, room, todo);
    }
    g.follows = todo.n > 0;
    return lay_out(todo, wide, A, s);
}

// Few rows go past the tensor cores where the weights can be read in place.
bool few(const Gated& A) {
    return gated_few_fits(A.rows, A.C, A.F, A.f_dense, A.dtype) && in_place(A.f_dense ? A.wg : A.wg.turned(), A.eb) &&
           in_place(A.f_dense ? A.wu : A.wu.turned(), A.eb);
}

cudaError_t forward(const Gated& A, void* ws, cudaStream_t s) {
    if (few(A)) {
        const Matrix wg = A.f_dense ? A.wg : A.wg.turned(), wu = A.f_dense ? A.wu : A.wu.turned();
        return launch_gated_few({A.x.p, A.C, A.rows, A.x.s0}, {wg.p, wg.cols, wg.rows, wg.s0}, {wu.p, wu.cols, wu.rows, wu.s0}, A.f_dense, A.y,
                                A.y_stride, A.act, A.alpha, A.dtype, A.sm, s);
    }
    Room room{static_cast<char*>(ws)};
    Gemm g;
    g.kind = kGatedForward;
    cudaError_t e = first_product(g, A, room, s);
    if (e != cudaSuccess) return e;
    g.out[0] = A.y;
    g.out_stride[0] = A.y_stride;
    g.part = static_cast<float*>(room.take(gemm_part_bytes(kGatedForward, A.rows, A.F, A.C, g.parts, 1, A.sm)));
    return launch_gemm(g, A.sm, s);
}

// The largest of the gradients' products (dw: of one weight or of both).
size_t backward_part_bytes(int64_t rows, int64_t C, int64_t F, bool f_dense, int dtype, int sm) {
    const int64_t M = f_dense ? C : F, N = f_dense ? F : C;
    const int one = dtype == CT_F32 ? 6 : 1;  // parts of a product
    return std::max({gemm_part_bytes(kGatedBackward, rows, F, C, one, 1, sm), gemm_part_bytes(kProduct, rows, C, F, 2 * one, 1, sm),
                     gemm_part_bytes(kProduct, M, N, rows, one, 1, sm), gemm_part_bytes(kProduct, M, N, rows, one, 2, sm)});
}

cudaError_t backward(const Gated& A, void* ws, cudaStream_t s) {
    Room room{static_cast<char*>(ws)};
    const bool wide = A.dtype == CT_F32;
    const int64_t pitch = pitch_of(A.F, A.eb);
    const size_t n = bytes_of(A.rows, A.F, A.eb);
    Matrix d[2];  // dg, du
    for (Matrix& m : d) m = {room.take(n), A.rows, A.F, pitch, 1};
    Gemm g;
    g.kind = kGatedBackward;
    Layouts todo;
    g.dy = operand(A.dy, A, room, todo);
    cudaError_t e = lay_out(todo, false, A, s);
    if (e == cudaSuccess) e = first_product(g, A, room, s);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 2; ++i) {
        g.out[i] = const_cast<void*>(d[i].p);
        g.out_stride[i] = pitch;
    }
    // the products run one after the other: one room for the parts of each
    float* const part = static_cast<float*>(room.take(backward_part_bytes(A.rows, A.C, A.F, A.f_dense, A.dtype, A.sm)));
    g.part = part;
    if ((e = launch_gemm(g, A.sm, s)) != cudaSuccess) return e;

    // dg and du as operands.  16-bit ones were rounded to the dtype in the epilogue above: kept
    // in two parts each they would take the second products from 8 to 16 M C F operations
    // (16384 x 1024 x 4096 from 428 to 713 us at the measured product rate) for an error of
    // 1.7e-3 instead of 2.3e-3 of the gradients' size, of which 1.7e-3 is the results' own rounding
    const int one = wide ? 3 : 1;
    GemmOperand dd[6];
    if (wide) {
        Layouts both;
        for (int i = 0; i < 2; ++i) split(dd + 3 * i, d[i], room, both);
        if ((e = lay_out(both, true, A, s)) != cudaSuccess) return e;
    } else {
        for (int i = 0; i < 2; ++i) dd[i] = {d[i].p, A.F, A.rows, pitch};
    }

    Gemm of_weights;
    if (A.dwg.p || A.dwu.p) {
        // [C][F] = x^T d, or [F][C] = d^T x where C is the dense axis
        Gemm& p = of_weights;
        p.dtype = A.dtype;
        p.M = A.f_dense ? A.C : A.F;
        p.N = A.f_dense ? A.F : A.C;
        p.K = A.rows;
        p.a_mn = p.b_mn = p.follows = true;
        if (wide) split_parts(p, 1);
        GemmOperand *x = A.f_dense ? p.a : p.b, *y = A.f_dense ? p.b : p.a;
        for (int i = 0; i < one; ++i) x[i] = g.a[i];
        p.z = 0;
        for (int i = 0; i < 2; ++i) {
            const Matrix& w = i ? A.dwu : A.dwg;
            if (!w.p) continue;
            for (int j = 0; j < one; ++j) y[one * p.z + j] = dd[one * i + j];
            p.out[p.z] = const_cast<void*>(w.p);
            p.out_stride[p.z] = A.f_dense ? w.s0 : w.s1;
            ++p.z;
        }
        (A.f_dense ? p.n_a : p.n_b) = one;
        (A.f_dense ? p.n_b : p.n_a) = one * p.z;
        (A.f_dense ? p.b_z : p.a_z) = one;
        p.part = part;
        if ((e = launch_gemm(p, A.sm, s)) != cudaSuccess) return e;
    }

    if (A.dx.p) {
        Gemm p;
        p.dtype = A.dtype;
        p.M = A.rows;
        p.N = A.C;
        p.K = A.F;
        p.n_a = p.n_b = 2 * one;
        p.b_mn = !A.f_dense;
        for (int i = 0; i < 2 * one; ++i) {
            p.a[i] = dd[i];
            p.b[i] = g.b[i];
        }
        if (wide) {
            split_parts(p, 2);
        } else {
            p.parts = 2;
            p.a_part[1] = p.b_part[1] = 1;
        }
        p.follows = true;
        if (A.dwg.p || A.dwu.p) p.ahead = &of_weights;
        p.out[0] = const_cast<void*>(A.dx.p);
        p.out_stride[0] = A.dx.s0;
        p.part = part;
        if ((e = launch_gemm(p, A.sm, s)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// ---- host -------------------------------------------------------------------

bool bad_ptr(const void* p, size_t a) { return p && (uintptr_t)p % a != 0; }

int check_problem(int64_t rows, int64_t C, int64_t F, int dtype) {
    if (dtype != CT_F32 && dtype != CT_F16 && dtype != CT_BF16)
        return report_error(CT_ERR_DTYPE, "dtype %d is not a supported floating type (CT_F32, CT_F16, CT_BF16)", dtype);
    if (rows < 0 || C < 0 || F < 0)
        return report_error(CT_ERR_SHAPE, "rows, C and F must be >= 0 (got %lld, %lld, %lld)", (long long)rows, (long long)C, (long long)F);
    if (rows > (1 << 22) || C > (1 << 20) || F > (1 << 20))
        return report_error(CT_ERR_TOO_LARGE, "rows <= 2^22, C and F <= 2^20 supported");
    return CT_OK;
}

// Bit 0: the F axis may be read as the dense one; bit 1: the C axis.
int dense_axes(const int64_t* s, int64_t C, int64_t F) { return (s[1] == 1 || F <= 1 ? 1 : 0) | (s[0] == 1 || C <= 1 ? 2 : 0); }

// The strides of the weights, and of their gradients where there are any:
// one axis is dense in all of them (*dense: bits as above).
int check_call(int64_t C, int64_t F, const int64_t* const* strides, int n, int activation, int* dense) {
    if (activation < CT_ACT_NONE || activation > CT_ACT_SIGMOID)
        return report_error(CT_ERR_PARAM, "activation %d is not a ct_activation", activation);
    *dense = 3;
    for (int i = 0; i < n; ++i) {
        if (!strides[i]) return report_error(CT_ERR_NULL, "strides must not be NULL");
        *dense &= dense_axes(strides[i], C, F);
    }
    if (!*dense) return report_error(CT_ERR_PARAM, "one axis of the weights (and their gradients) must be dense, the same for all");
    return CT_OK;
}

// Copies of unaligned operands, parts of fp32 ones, dg and du, pieces of split sums.
size_t workspace_bytes_of(int64_t rows, int64_t C, int64_t F, int dtype, int backward, int aligned) {
    DeviceInfo dev;
    const int sm = device_info(&dev) == cudaSuccess ? dev.sm_count : 152;
    const size_t eb = dtype == CT_F32 ? 4 : 2;
    if (rows == 0 || C == 0 || F == 0) return 0;
    const size_t x = bytes_of(rows, C, 2), w = std::max(bytes_of(C, F, 2), bytes_of(F, C, 2)), d = bytes_of(rows, F, eb);
    size_t n = 0;
    if (dtype == CT_F32) n = 3 * x + 6 * w;
    else if (!aligned) n = x + 2 * w;
    if (!backward) return n + gemm_part_bytes(kGatedForward, rows, F, C, dtype == CT_F32 ? 6 : 1, 1, sm);
    if (dtype == CT_F32) n += 6 * bytes_of(rows, F, 2);
    return n + 2 * d + (aligned ? 0 : d) + std::max(backward_part_bytes(rows, C, F, true, dtype, sm), backward_part_bytes(rows, C, F, false, dtype, sm));
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
            return CT_OK;
        }
        const cudaError_t e = cudaMallocAsync(&p, need, s);
        if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "cudaMallocAsync(workspace): %s", cudaGetErrorString(e));
        owned = true;
        return CT_OK;
    }
    cudaError_t give(cudaError_t e, cudaStream_t s) {
        if (!owned) return e;
        const cudaError_t f = cudaFreeAsync(p, s);
        return e == cudaSuccess ? f : e;
    }
};

// Zeros in `outer` rows of `inner` elements.
cudaError_t zero(const Matrix& m, bool s0_outer, size_t eb, cudaStream_t s) {
    const int64_t outer = s0_outer ? m.rows : m.cols, inner = s0_outer ? m.cols : m.rows, stride = s0_outer ? m.s0 : m.s1;
    if (outer == 0 || inner == 0) return cudaSuccess;
    return cudaMemset2DAsync(const_cast<void*>(m.p), outer == 1 ? inner * eb : stride * eb, 0, inner * eb, outer, s);
}

}  // namespace
}  // namespace ct

using namespace ct;

extern "C" int ct_gated_projection_workspace_bytes(int64_t rows, int64_t C, int64_t F, int dtype, int backward, int aligned, size_t* bytes) {
    if (!bytes) return report_error(CT_ERR_NULL, "bytes is NULL");
    const int rc = check_problem(rows, C, F, dtype);
    if (rc != CT_OK) return rc;
    // few rows go past the tensor cores (few() above), which needs none
    const bool none = !backward && (((aligned & CT_GATED_WEIGHTS_F) && gated_few_fits(rows, C, F, true, dtype)) ||
                                    ((aligned & CT_GATED_WEIGHTS_C) && gated_few_fits(rows, C, F, false, dtype)));
    *bytes = none ? 0 : workspace_bytes_of(rows, C, F, dtype, backward, aligned & CT_GATED_ALIGNED);
    return CT_OK;
}

extern "C" int ct_gated_projection_forward(const void* x, int64_t x_stride, const void* w_gate, const int64_t* gate_strides,
                                           const void* w_up, const int64_t* up_strides, void* y, int64_t y_stride, void* workspace,
                                           size_t workspace_bytes, int64_t rows, int64_t C, int64_t F, int activation, float alpha,
                                           int dtype, void* stream) {
    int rc = check_problem(rows, C, F, dtype);
    const int64_t* const strides[] = {gate_strides, up_strides};
    int dense = 0;
    if (rc == CT_OK) rc = check_call(C, F, strides, 2, activation, &dense);
    if (rc != CT_OK) return rc;
    if (rows == 0 || F == 0) return CT_OK;
    if (!y || (C > 0 && (!x || !w_gate || !w_up))) return report_error(CT_ERR_NULL, "x, the weights and y must not be NULL");
    Gated A{};
    A.eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(x, A.eb) || bad_ptr(w_gate, A.eb) || bad_ptr(w_up, A.eb) || bad_ptr(y, A.eb))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "gated projection: %s", cudaGetErrorString(e));
    A.x = {x, rows, C, x_stride, 1};
    A.wg = {w_gate, C, F, gate_strides[0], gate_strides[1]};
    A.wu = {w_up, C, F, up_strides[0], up_strides[1]};
    A.f_dense = dense & 1;
    A.y = y; A.y_stride = y_stride;
    A.rows = rows; A.C = C; A.F = F; A.act = activation; A.alpha = alpha; A.dtype = dtype; A.sm = dev.sm_count;
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    if (C == 0) {
        e = zero({y, rows, F, y_stride, 1}, true, A.eb, s);
    } else {
        const int aligned = in_place(A.x, A.eb) && in_place(A.f_dense ? A.wg : A.wg.turned(), A.eb) &&
                            in_place(A.f_dense ? A.wu : A.wu.turned(), A.eb);
        if ((rc = ws.take(workspace, workspace_bytes, few(A) ? 0 : workspace_bytes_of(rows, C, F, dtype, 0, aligned), s)) != CT_OK) return rc;
        e = ws.give(forward(A, ws.p, s), s);
    }
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "gated projection: %s", cudaGetErrorString(e));
    return CT_OK;
}

extern "C" int ct_gated_projection_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, const void* w_gate,
                                            const int64_t* gate_strides, const void* w_up, const int64_t* up_strides, void* dx,
                                            int64_t dx_stride, void* dw_gate, const int64_t* dgate_strides, void* dw_up,
                                            const int64_t* dup_strides, void* workspace, size_t workspace_bytes, int64_t rows, int64_t C,
                                            int64_t F, int activation, float alpha, int dtype, void* stream) {
    int rc = check_problem(rows, C, F, dtype);
    const int64_t* strides[4] = {gate_strides, up_strides};
    int n = 2, dense = 0;
    if (dw_gate) strides[n++] = dgate_strides;
    if (dw_up) strides[n++] = dup_strides;
    if (rc == CT_OK) rc = check_call(C, F, strides, n, activation, &dense);
    if (rc != CT_OK) return rc;
    if (C == 0 || (rows == 0 && !dw_gate && !dw_up) || (!dx && !dw_gate && !dw_up)) return CT_OK;
    if (rows > 0 && F > 0 && (!dy || !x || !w_gate || !w_up)) return report_error(CT_ERR_NULL, "dy, x and the weights must not be NULL");
    Gated A{};
    A.eb = dtype == CT_F32 ? 4 : 2;
    if (bad_ptr(dy, A.eb) || bad_ptr(x, A.eb) || bad_ptr(w_gate, A.eb) || bad_ptr(w_up, A.eb) || bad_ptr(dx, A.eb) ||
        bad_ptr(dw_gate, A.eb) || bad_ptr(dw_up, A.eb))
        return report_error(CT_ERR_ALIGN, "pointers must be aligned to their element size");
    A.x = {x, rows, C, x_stride, 1};
    A.wg = {w_gate, C, F, gate_strides[0], gate_strides[1]};
    A.wu = {w_up, C, F, up_strides[0], up_strides[1]};
    A.dy = {dy, rows, F, dy_stride, 1};
    A.dx = {dx, rows, C, dx_stride, 1};
    if (dw_gate) A.dwg = {dw_gate, C, F, dgate_strides[0], dgate_strides[1]};
    if (dw_up) A.dwu = {dw_up, C, F, dup_strides[0], dup_strides[1]};
    A.f_dense = dense & 1;
    A.rows = rows; A.C = C; A.F = F; A.act = activation; A.alpha = alpha; A.dtype = dtype;
    cudaStream_t s = (cudaStream_t)stream;
    Workspace ws;
    cudaError_t e = cudaSuccess;
    if (rows == 0 || F == 0) {
        if (dx && rows > 0) e = zero(A.dx, true, A.eb, s);
        if (dw_gate && e == cudaSuccess) e = zero(A.dwg, A.f_dense, A.eb, s);
        if (dw_up && e == cudaSuccess) e = zero(A.dwu, A.f_dense, A.eb, s);
    } else {
        const int aligned = in_place(A.x, A.eb) && in_place(A.dy, A.eb) && in_place(A.f_dense ? A.wg : A.wg.turned(), A.eb) &&
                            in_place(A.f_dense ? A.wu : A.wu.turned(), A.eb);
        if ((rc = ws.take(workspace, workspace_bytes, workspace_bytes_of(rows, C, F, dtype, 1, aligned), s)) != CT_OK) return rc;
        DeviceInfo dev;
        e = device_info(&dev);
        A.sm = dev.sm_count;
        if (e == cudaSuccess) e = backward(A, ws.p, s);
        e = ws.give(e, s);
    }
    if (e != cudaSuccess) return report_error(CT_ERR_CUDA, "gated projection backward: %s", cudaGetErrorString(e));
    return CT_OK;
}
