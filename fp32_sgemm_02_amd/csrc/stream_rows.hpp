// stream_rows.hpp -- the inner loops of products with few rows, in which the
// weights are streamed once from memory into registers (no LDS staging: every
// weight value is used by one wave only, so a copy in LDS would be read once).
//
// A fragment is 16 bytes per lane: the 8 k values of one v_mfma_f32_16x16x32
// (16-bit types) or the 4 k values of four v_mfma_f32_16x16x4 (fp32; step s
// takes element s of every lane, so lane group g stands for k = 4g + s).  The
// weights are the A operand, the few rows ("tokens") the B operand: lane
// (i, g) of the result holds weight rows 4g .. 4g+3 of token i.
#pragma once

#include "linear_internal.hpp"

namespace sg {

template <int DT>
struct Step {
    static constexpr int V = Type<DT>::V;   // values per fragment
    static constexpr int K = 4 * V;         // k per step
};

template <int DT>
__device__ __forceinline__ floatx4 mfma_step(uintx4 w, uintx4 x, floatx4 c) {
    if constexpr (DT == SGEMM_DTYPE_F32) {
        const floatx4 a = __builtin_bit_cast(floatx4, w), b = __builtin_bit_cast(floatx4, x);
#pragma unroll
        for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
        return c;
    } else {
        return mfma16<DT>(w, x, c);
    }
}

// V values from p on, of which n lie inside (zeros for the others, which are
// not read).  Rows may start at any multiple of the value's size: the target
// loads 16 bytes from any address.
template <int DT>
__device__ __forceinline__ uintx4 load_frag(const typename Type<DT>::T *p, int n) {
    constexpr int V = Type<DT>::V;
    uintx4 v = {0, 0, 0, 0};
    if (n >= V) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) {
                if constexpr (DT == SGEMM_DTYPE_F32)
                    v[e] = __builtin_bit_cast(unsigned, p[e]);
                else
                    v[e / 2] |= (unsigned)p[e] << (16 * (e & 1));
            }
    }
    return v;
}

// acc[r][t] += the products over k in [k0, k1) of RB weight rows (w[r]: this
// lane's row of 16-row block r) and TB token rows (x[t]), k0 a multiple of the
// step; both pointers at k = 0, kend the length of the rows.  Two register
// sets of U steps each: the loads of a round are issued before the previous
// round's products.
template <int DT, int RB, int TB, int U>
__device__ __forceinline__ void stream_dot(const typename Type<DT>::T *const (&w)[RB],
                                           const typename Type<DT>::T *const (&x)[TB], int k0,
                                           int k1, int lane, floatx4 (&acc)[RB][TB]) {
    constexpr int V = Step<DT>::V, KS = Step<DT>::K, KR = U * KS;
    const int kg = V * (lane >> 4);
    struct Round {
        uintx4 w[U][RB], x[U][TB];
    } a, b;
    auto load = [&](Round &r, int k) {
        if (k + KR <= k1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kk = k + u * KS + kg;
#pragma unroll
                for (int q = 0; q < RB; ++q) __builtin_memcpy(&r.w[u][q], w[q] + kk, 16);
#pragma unroll
                for (int q = 0; q < TB; ++q) __builtin_memcpy(&r.x[u][q], x[q] + kk, 16);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kk = k + u * KS + kg;
#pragma unroll
                for (int q = 0; q < RB; ++q) r.w[u][q] = load_frag<DT>(w[q] + kk, k1 - kk);
#pragma unroll
                for (int q = 0; q < TB; ++q) r.x[u][q] = load_frag<DT>(x[q] + kk, k1 - kk);
            }
        }
    };
    auto products = [&](const Round &r) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < RB; ++q)
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    acc[q][t] = mfma_step<DT>(r.w[u][q], r.x[u][t], acc[q][t]);
    };
    if (k0 >= k1) return;
    load(a, k0);
    for (int k = k0; k < k1; k += 2 * KR) {
        if (k + KR < k1) load(b, k + KR);
        pipeline_fence();
        products(a);
        pipeline_fence();
        if (k + KR >= k1) break;
        if (k + 2 * KR < k1) load(a, k + 2 * KR);
        pipeline_fence();
        products(b);
        pipeline_fence();
    }
}

}  // namespace sg
