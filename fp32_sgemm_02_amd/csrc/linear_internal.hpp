// linear_internal.hpp -- types shared by the feed-forward operators (linear
// layers, their backward pass, the mixture-of-experts layer) and the C-ABI
// entry points of linear.cpp.  Internal to the library.
#pragma once

#include <type_traits>
#include <utility>

#include "gemm_internal.hpp"

namespace sg {

typedef unsigned short u16;

// One product of a linear layer,
//     C(m, n) = act(sum_k A(m, k) B(n, k) + bias(n)) + R(m, n),
// all of one type (SGEMM_DTYPE_*), summed and finished in fp32 and rounded
// once.  Each operand is stored with k contiguous (A(m, k) = A[m * lda + k])
// or, with a_mc / b_mc, with its own index contiguous (A(m, k) =
// A[k * lda + m]).  Z, when given, receives the sum plus bias before the
// activation.  Sizes and leading dimensions in elements.
struct Prod {
    int M, N, K;
    const void *A;
    long long lda;
    const void *B;
    long long ldb;
    void *C;
    long long ldc;
    int a_mc = 0, b_mc = 0;
    const void *bias = nullptr;
    const void *R = nullptr;
    long long ldr = 0;
    void *Z = nullptr;
    long long ldz = 0;
    int act = SGEMM_ACT_NONE;
    int a_pad = 0, b_pad = 0;   // the stored rows are filled up with zeros to 16 bytes
    // What the rounding of A left over, laid out as A (few-rows kernels only).
    const void *lo = nullptr;
};

// Tile kernels of 16-bit products (linear16.hip): bytes of partial sums (after
// the workspace's counters) that a launch takes, and the launch.  `ws` may be
// empty when no bytes are needed.
size_t prod16_workspace(int dtype, const Prod &p);
hipError_t launch_prod16(int dtype, const Prod &p, const Workspace &ws, hipStream_t stream);

// dX and dW of one backward pass (a_mc 0 and 1, both b_mc), in one launch where
// both are small.
size_t prod16_pair_workspace(const Prod &x, const Prod &w);
hipError_t launch_prod16_pair(int dtype, const Prod &x, const Prod &w, const Workspace &ws,
                              hipStream_t stream);

// The tile kernel of large products (linear16_big.hip), for operands whose
// rows take direct 16-byte loads.
hipError_t launch_prod16_big(int dtype, const Prod &p, hipStream_t stream);

// Few-rows kernels (linear_rows.hip), M <= kFewRows, every type, A with k
// contiguous and either B: B is streamed once, from memory into registers.
constexpr int kFewRows = 64;
size_t rows_workspace(int dtype, const Prod &p);
hipError_t launch_rows(int dtype, const Prod &p, const Workspace &ws, hipStream_t stream);
// K <= kFewRows, both operands with their own index contiguous.
hipError_t launch_outer(int dtype, const Prod &p, hipStream_t stream);

// G = dY * act'(Z) over M x N and its column sums (dtype SGEMM_DTYPE_*): G is
// written where it is not null (rows of ldg values, 16-byte aligned, zeros from N
// to the end of its last 16 bytes), rounded to dtype, with what the rounding left
// over in lo where that is not null; db, where it is not null, receives the
// sums, rounded to dtype.  They are added in fp32 from the unrounded values in
// an order that is fixed for a shape.  part: grad_workspace bytes; count:
// arrival counters, zero between launches.
size_t grad_workspace(int dtype, int M, int N);
hipError_t launch_grad(int dtype, int M, int N, const void *dY, long long lddy, const void *Z,
                       long long ldz, int act, void *G, void *lo, long long ldg, void *db,
                       float *part, unsigned *count, hipStream_t stream);

// A mixture-of-experts layer for few tokens (moe.hip); see sgemm_moe.
constexpr int kMoeTokens = 64, kMoeExperts = 512, kMoeChoices = 16;
constexpr int kMoeWidth = 64512;   // an arrival counter for every 32 columns of Y
struct Moe {
    int T, D, F, E, k;
    int gated, renorm, act;
    const void *X;
    long long ldx;
    const void *Wr;
    long long ldwr;
    const void *W1;
    long long ld1, stride1;
    const void *W2;
    long long ld2, stride2;
    void *Y;
    long long ldy;
    int *ids;         // T x k, or null
    float *weights;   // T x k, or null
};
size_t moe_workspace(const Moe &m);
hipError_t launch_moe(int dtype, const Moe &m, const Workspace &ws, hipStream_t stream);

// C = the sum of the `count` M x N arrays at `parts`, `step` floats apart with
// rows of ldp floats, in order.
hipError_t launch_sum32(int M, int N, const float *parts, long long ldp, long long step, int count,
                        float *C, long long ldc, hipStream_t stream);

// Y = act(Z) + R elementwise over M x N in fp32, in place where Y is Z.
hipError_t launch_finish32(int M, int N, const float *Z, long long ldz, int act, const float *R,
                           long long ldr, float *Y, long long ldy, hipStream_t stream);

// Whether rows of an array take 16-byte accesses.
__host__ __device__ inline bool rows16(const void *q, long long ld, int elem) {
    return reinterpret_cast<unsigned long long>(q) % 16 == 0 && ld * elem % 16 == 0;
}

// ---- device helpers ---------------------------------------------------------

// Slope of an activation at its input (SGEMM_ACT_*), in fp32.  ReLU's slope at
// 0 is 0.
template <int ACT>
__device__ __forceinline__ float slope_t(float x) {
    if constexpr (ACT == SGEMM_ACT_RELU) {
        return x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);   // NaN stays NaN
    } else if constexpr (ACT == SGEMM_ACT_SILU) {
        // s (1 + x (1 - s)) with 1 - s = sigmoid(-x), which keeps its digits
        // where s rounds to 1; x (1 - s) -> 0 for x -> inf through e^-x
        const float e = expf(-fabsf(x));
        const float r = 1.f / (1.f + e);
        const float s = x >= 0.f ? r : e * r, c = x >= 0.f ? e * r : r;
        return x == -INFINITY || x == INFINITY ? s : s * (1.f + x * c);
    } else if constexpr (ACT == SGEMM_ACT_GELU_ERF) {
        const float phi = 0.39894228040143268f * expf(-0.5f * x * x);
        return 0.5f * erfcf(-0.70710678118654752f * x) +
               (fabsf(x) == INFINITY ? 0.f : x * phi);
    } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) {
        // q = (1 + tanh u) / 2 = sigmoid(2u): slope q + 2 x q (1 - q) u'
        const float x2 = x * x;
        const float u = 0.79788456080286536f * fmaf(0.044715f * x, x2, x);
        const float du = 0.79788456080286536f * fmaf(0.134145f, x2, 1.f);
        const float e = expf(-2.f * fabsf(u));
        const float r = 1.f / (1.f + e);
        const float q = u >= 0.f ? r : e * r;
        // e r^2 = q (1 - q); it is 0 in fp32 long before x du overflows
        const float t = e * r * r;
        return t == 0.f ? q : q + 2.f * x * t * du;
    } else {
        return 1.f;
    }
}

// The same functions where the result is rounded to 16 bits: 2^x and 1 / x by
// the hardware's instructions, about one unit in the last place each (a large
// exponent loses more in its own rounding, 2^-17 of the value at the ends of the
// range, where a 16-bit result keeps 2^-8 or 2^-11).  The full functions took half
// of the epilogue's time: 8192 x 14336 x 4096 bf16 with GELU (tanh) 793 us, 736 with these; the
// erf form has no such short one.

// x / (1 + 2^v).  Far out both sides are taken 2^64 times smaller: 1 / (1 + 2^v)
// falls below the normal numbers there, which the instructions flush to zero,
// before x times it does.
__device__ __forceinline__ float over_one_plus(float x, float v) {
    const bool far = v > 64.f;
    const float k = far ? 0x1p-64f : 1.f;
    return x * k * __builtin_amdgcn_rcpf(k + __builtin_amdgcn_exp2f(far ? v - 64.f : v));
}
template <int ACT>
__device__ __forceinline__ float activate_short(float x) {
    if constexpr (ACT == SGEMM_ACT_SILU)
        return over_one_plus(x, -1.44269504f * x);
    else if constexpr (ACT == SGEMM_ACT_GELU_TANH)   // -2 log2(e) sqrt(2 / pi) (x + 0.044715 x^3)
        return over_one_plus(x, -2.30220820f * fmaf(0.044715f * x, x * x, x));
    else
        return activate_t<ACT>(x);
}
template <int ACT>
__device__ __forceinline__ float slope_short(float x) {
    if constexpr (ACT == SGEMM_ACT_SILU) {
        // (the clamp keeps an infinite x from meeting 1 - s = 0; NaN stays in s)
        const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
        const float c = __builtin_amdgcn_fmed3f(x, -100.f, 100.f);
        return s * fmaf(c, 1.f - s, 1.f);
    } else if constexpr (ACT == SGEMM_ACT_GELU_TANH) {
        const float x2 = x * x;
        const float q = __builtin_amdgcn_rcpf(
            1.f + __builtin_amdgcn_exp2f(-2.30220820f * fmaf(0.044715f * x, x2, x)));
        const float c = __builtin_amdgcn_fmed3f(x, -30.f, 30.f);
        // 2 sqrt(2 / pi) (1 + 3 * 0.044715 x^2)
        const float du = fmaf(0.21406445f, c * c, 1.59576912f);
        return q * fmaf(c * du, 1.f - q, 1.f);
    } else {
        return slope_t<ACT>(x);
    }
}

// 16-bit values to and from fp32 (round to nearest, ties to even).
template <int DT>
__device__ __forceinline__ float widen(u16 v) {
    if constexpr (DT == SGEMM_DTYPE_BF16)
        return __builtin_bit_cast(float, (unsigned)v << 16);
    else
        return (float)__builtin_bit_cast(_Float16, v);
}
template <int DT>
__device__ __forceinline__ u16 narrow(float v) {
    if constexpr (DT == SGEMM_DTYPE_BF16)
        return __builtin_bit_cast(u16, (__bf16)v);
    else
        return __builtin_bit_cast(u16, (_Float16)v);
}

// Values of one type as the kernels load and store them, V to 16 bytes.
template <int DT>
struct Type {
    using T = u16;
    static constexpr int V = 8;
    static __device__ __forceinline__ float load(T v) { return widen<DT>(v); }
    static __device__ __forceinline__ T store(float v) { return narrow<DT>(v); }
};
template <>
struct Type<SGEMM_DTYPE_F32> {
    using T = float;
    static constexpr int V = 4;
    static __device__ __forceinline__ float load(T v) { return v; }
    static __device__ __forceinline__ T store(float v) { return v; }
};

template <int DT, int ACT>
__device__ __forceinline__ float activate_for(float x) {
    if constexpr (DT == SGEMM_DTYPE_F32)
        return activate_t<ACT>(x);
    else
        return activate_short<ACT>(x);
}
template <int DT, int ACT>
__device__ __forceinline__ float slope_for(float x) {
    if constexpr (DT == SGEMM_DTYPE_F32)
        return slope_t<ACT>(x);
    else
        return slope_short<ACT>(x);
}

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));

// 16 bytes from any place where a value may start.  16-bit values that start in
// the middle of a dword are put together from the five aligned dwords that hold
// them (the hardware loads 16 bytes from any address, but slowly unless it is a
// dword's: 16 x 4097 x 4097 bf16 40 us, 26 so; the tile kernel's register path gains
// nothing by it).  Each of those dwords holds a value
// of the sixteen bytes, so none lies outside the array's memory pages.
template <int DT>
__device__ __forceinline__ uintx4 load_any(const typename Type<DT>::T *p) {
    uintx4 v;
    if constexpr (DT == SGEMM_DTYPE_F32) {
        __builtin_memcpy(&v, p, 16);
    } else {
        const unsigned mis = (unsigned)(unsigned long long)p & 2u;
        const unsigned *q = reinterpret_cast<const unsigned *>(
            reinterpret_cast<unsigned long long>(p) & ~3ull);
        __builtin_memcpy(&v, q, 16);
        const unsigned e = q[mis ? 4 : 3];
        const unsigned s = 8 * mis;
        v = uintx4{__builtin_amdgcn_alignbit(v[1], v[0], s), __builtin_amdgcn_alignbit(v[2], v[1], s),
                   __builtin_amdgcn_alignbit(v[3], v[2], s), __builtin_amdgcn_alignbit(e, v[3], s)};
    }
    return v;
}

// D += A B over 32 k values of 16-bit inputs.  Lane (i, g) = (lane % 16,
// lane / 16): a holds A(row i, k = 8g .. 8g+7), b holds B(column i, same k),
// and c holds D(rows 4g .. 4g+3, column i).
template <int DT>
__device__ __forceinline__ floatx4 mfma16(uintx4 a, uintx4 b, floatx4 c) {
    if constexpr (DT == SGEMM_DTYPE_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Transposing LDS reads of 16-bit values, with their wait in the same asm block
// (the builtin would have each read wait for every direct load in flight, since
// the compiler cannot tell the stages of the ring apart: 4096^3 with one operand
// read this way: 8192^3 dX 892 us, 752 with this).  at[b]: LDS address of block b's part for this
// lane; HI: bytes from its first four rows of k to the next four; with STEPS ==
// 2 also the next 32-k step, NEXT bytes further.  f[b][s]: the fragments.
template <int BLOCKS, int STEPS, int HI, int NEXT>
__device__ __forceinline__ void read_transposed(const unsigned (&at)[BLOCKS],
                                                uintx4 (&f)[BLOCKS][STEPS]) {
    static_assert((BLOCKS == 2 || BLOCKS == 4) && (STEPS == 1 || STEPS == 2), "2 or 4 blocks");
    uintx2 r[BLOCKS][STEPS][2];
    if constexpr (BLOCKS == 2 && STEPS == 1) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4\n"
            "ds_read_b64_tr_b16 %1, %4 offset:%6\n"
            "ds_read_b64_tr_b16 %2, %5\n"
            "ds_read_b64_tr_b16 %3, %5 offset:%6\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1])
            : "v"(at[0]), "v"(at[1]), "n"(HI)
            : "memory");
    } else if constexpr (BLOCKS == 2 && STEPS == 2) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n"
            "ds_read_b64_tr_b16 %1, %8 offset:%10\n"
            "ds_read_b64_tr_b16 %2, %8 offset:%11\n"
            "ds_read_b64_tr_b16 %3, %8 offset:%12\n"
            "ds_read_b64_tr_b16 %4, %9\n"
            "ds_read_b64_tr_b16 %5, %9 offset:%10\n"
            "ds_read_b64_tr_b16 %6, %9 offset:%11\n"
            "ds_read_b64_tr_b16 %7, %9 offset:%12\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[0][1][0]), "=&v"(r[0][1][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1]), "=&v"(r[1][1][0]), "=&v"(r[1][1][1])
            : "v"(at[0]), "v"(at[1]), "n"(HI), "n"(NEXT), "n"(NEXT + HI)
            : "memory");
    } else if constexpr (BLOCKS == 4 && STEPS == 1) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n"
            "ds_read_b64_tr_b16 %1, %8 offset:%12\n"
            "ds_read_b64_tr_b16 %2, %9\n"
            "ds_read_b64_tr_b16 %3, %9 offset:%12\n"
            "ds_read_b64_tr_b16 %4, %10\n"
            "ds_read_b64_tr_b16 %5, %10 offset:%12\n"
            "ds_read_b64_tr_b16 %6, %11\n"
            "ds_read_b64_tr_b16 %7, %11 offset:%12\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1]), "=&v"(r[2][0][0]), "=&v"(r[2][0][1]), "=&v"(r[3][0][0]), "=&v"(r[3][0][1])
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(HI)
            : "memory");
    } else if constexpr (BLOCKS == 4 && STEPS == 2) {
        asm volatile(
            "ds_read_b64_tr_b16 %0, %16\n"
            "ds_read_b64_tr_b16 %1, %16 offset:%20\n"
            "ds_read_b64_tr_b16 %2, %16 offset:%21\n"
            "ds_read_b64_tr_b16 %3, %16 offset:%22\n"
            "ds_read_b64_tr_b16 %4, %17\n"
            "ds_read_b64_tr_b16 %5, %17 offset:%20\n"
            "ds_read_b64_tr_b16 %6, %17 offset:%21\n"
            "ds_read_b64_tr_b16 %7, %17 offset:%22\n"
            "ds_read_b64_tr_b16 %8, %18\n"
            "ds_read_b64_tr_b16 %9, %18 offset:%20\n"
            "ds_read_b64_tr_b16 %10, %18 offset:%21\n"
            "ds_read_b64_tr_b16 %11, %18 offset:%22\n"
            "ds_read_b64_tr_b16 %12, %19\n"
            "ds_read_b64_tr_b16 %13, %19 offset:%20\n"
            "ds_read_b64_tr_b16 %14, %19 offset:%21\n"
            "ds_read_b64_tr_b16 %15, %19 offset:%22\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0][0][0]), "=&v"(r[0][0][1]), "=&v"(r[0][1][0]), "=&v"(r[0][1][1]), "=&v"(r[1][0][0]), "=&v"(r[1][0][1]), "=&v"(r[1][1][0]), "=&v"(r[1][1][1]), "=&v"(r[2][0][0]), "=&v"(r[2][0][1]), "=&v"(r[2][1][0]), "=&v"(r[2][1][1]), "=&v"(r[3][0][0]), "=&v"(r[3][0][1]), "=&v"(r[3][1][0]), "=&v"(r[3][1][1])
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(HI), "n"(NEXT), "n"(NEXT + HI)
            : "memory");
    }
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int q = 0; q < STEPS; ++q)
            f[b][q] = uintx4{r[b][q][0][0], r[b][q][0][1], r[b][q][1][0], r[b][q][1][1]};
}

// The LDS address of a pointer into shared memory.
__device__ __forceinline__ unsigned lds_address(const unsigned char *p) {
    return (unsigned)(unsigned long long)(
        const __attribute__((address_space(3))) unsigned char *)p;
}

// Calls f with the constants 0 .. N-1.
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F &&f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F &&f) {
    each_of(std::make_integer_sequence<int, N>{}, f);
}

// Calls f with the activation code as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
    case SGEMM_ACT_RELU: f(std::integral_constant<int, SGEMM_ACT_RELU>{}); break;
    case SGEMM_ACT_SILU: f(std::integral_constant<int, SGEMM_ACT_SILU>{}); break;
    case SGEMM_ACT_GELU_ERF: f(std::integral_constant<int, SGEMM_ACT_GELU_ERF>{}); break;
    case SGEMM_ACT_GELU_TANH: f(std::integral_constant<int, SGEMM_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, SGEMM_ACT_NONE>{}); break;
    }
}

// Bias, activation, residual and the store of the CN adjacent columns from n
// on of row m < p.M, 16 bytes at a time whatever their alignment (the target
// takes any address), those at the end value by value.  R may be C: each
// cell is read before it is written, by the same lane.
template <int DT, int ACT, int CN>
__device__ __forceinline__ void finish_run(const Prod &p, int m, int n, const float (&v)[CN]) {
    using Ty = Type<DT>;
    using T = typename Ty::T;
    constexpr int W = CN < Ty::V ? CN : Ty::V;   // values per access
    constexpr int BYTES = W * sizeof(T);
    static_assert(CN % W == 0, "whole accesses");
    T *c = static_cast<T *>(p.C) + (long long)m * p.ldc;
    const T *r = p.R ? static_cast<const T *>(p.R) + (long long)m * p.ldr : nullptr;
    T *z = p.Z ? static_cast<T *>(p.Z) + (long long)m * p.ldz : nullptr;
    const T *bias = static_cast<const T *>(p.bias);
#pragma unroll
    for (int h = 0; h < CN; h += W) {
        const int n1 = n + h;
        if (n1 >= p.N) return;
        if (n1 + W <= p.N) {   // (whole accesses go to any address)
            T t[W];
            float x[W], res[W];
            if (r) {
                __builtin_memcpy(t, r + n1, BYTES);
#pragma unroll
                for (int e = 0; e < W; ++e) res[e] = Ty::load(t[e]);
            }
            if (bias) {
                __builtin_memcpy(t, bias + n1, BYTES);
#pragma unroll
                for (int e = 0; e < W; ++e) x[e] = v[h + e] + Ty::load(t[e]);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) x[e] = v[h + e];
            }
            if (z) {
#pragma unroll
                for (int e = 0; e < W; ++e) t[e] = Ty::store(x[e]);
                __builtin_memcpy(z + n1, t, BYTES);
            }
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float y = activate_for<DT, ACT>(x[e]);
                t[e] = Ty::store(r ? y + res[e] : y);
            }
            __builtin_memcpy(c + n1, t, BYTES);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if (n1 + e >= p.N) continue;
                const float s = bias ? v[h + e] + Ty::load(bias[n1 + e]) : v[h + e];
                if (z) z[n1 + e] = Ty::store(s);
                const float y = activate_for<DT, ACT>(s);
                c[n1 + e] = Ty::store(r ? y + Ty::load(r[n1 + e]) : y);
            }
        }
    }
}

// The epilogue of a wave's 16 XB x 16 YB sums at (m0, n0), in MFMA layout:
// sum(y, x) holds, in lane (i, g), row 16 x + i and columns 16 y + 4g .. +3.
// They pass through `box` (LDS of this wave alone, 16 XB rows of 16 YB floats)
// so that a lane then has eight adjacent columns, 16 bytes of a 16-bit result,
// and neighbouring lanes neighbouring ones; the rows' 16-byte chunks are
// swizzled against bank conflicts.  The loop is not unrolled: unrolled it takes
// the same time and several times the code.
template <int DT, int XB, int YB, class F>
__device__ __forceinline__ void finish_wave(const Prod &p, int m0, int n0, int lane, float *box,
                                            F &&sum) {
    constexpr int CH = 4 * YB, LR = CH / 2;   // chunks per row, lanes per row
    static_assert(CH == 8 || CH == 16, "rows of 32 or 64 columns");
    auto swz = [](int row) { return CH == 16 ? row & 15 : (row >> 1) & 7; };
    const int i = lane & 15, g = lane >> 4;
    floatx4 *b4 = reinterpret_cast<floatx4 *>(box);
    each<XB * YB>([&](auto j) __attribute__((always_inline)) {
        constexpr int x = j / YB, y = j % YB;
        const int row = 16 * x + i;
        b4[row * CH + ((4 * y + g) ^ swz(row))] = sum(std::integral_constant<int, y>{},
                                                      std::integral_constant<int, x>{});
    });
    with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll 1
        for (int r = lane / LR; r < 16 * XB; r += 64 / LR) {
            const int q = lane % LR;
            const floatx4 u = b4[r * CH + ((2 * q) ^ swz(r))], w = b4[r * CH + ((2 * q + 1) ^ swz(r))];
            const float v[8] = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
            if (m0 + r < p.M) finish_run<DT, decltype(tag)::value>(p, m0 + r, n0 + 8 * q, v);
        }
    });
}

// Partial sums that another workgroup adds up are stored and loaded as
// device-coherent accesses, which bypass the per-XCD caches (these are not
// coherent with each other); a workgroup counts its arrival after every wave
// has waited for its stores.
__device__ __forceinline__ void store_partial(float *d, const floatx4 &v) {
    const float f[4] = {v[0], v[1], v[2], v[3]};
    unsigned long long w[2];
    __builtin_memcpy(w, f, 16);
    unsigned long long *q = reinterpret_cast<unsigned long long *>(d);
    __hip_atomic_store(q, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(q + 1, w[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ floatx4 load_partial(const float *d) {
    const unsigned long long *q = reinterpret_cast<const unsigned long long *>(d);
    unsigned long long w[2];
    w[0] = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    w[1] = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    float f[4];
    __builtin_memcpy(f, w, 16);
    return floatx4{f[0], f[1], f[2], f[3]};
}

// Counts this workgroup's arrival at *count and returns, to every thread,
// whether it is the last of n.  `flag`: one int of LDS.
__device__ __forceinline__ bool arrive_last(unsigned *count, unsigned n, int *flag) {
    __builtin_amdgcn_s_waitcnt(0);   // this wave's partial sums are in memory
    __syncthreads();
    if (threadIdx.x == 0)
        *flag = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                n - 1;
    __syncthreads();
    return *flag != 0;
}

}  // namespace sg
