// stream_rows.hpp -- the inner loops of products with few rows, in which the
// weights are streamed once from memory.
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
// not read; n <= 0: none).  `safe`: any readable value.  Branch-free: loads behind
// per-lane branches wait for one another, and a tail of a few chunks then takes
// longer than the rows before it.
template <int DT>
__device__ __forceinline__ uintx4 load_frag(const typename Type<DT>::T *p, int n,
                                            const typename Type<DT>::T *safe) {
    constexpr int V = Type<DT>::V;
    typename Type<DT>::T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = *(e < n ? p + e : safe);
    uintx4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if constexpr (DT == SGEMM_DTYPE_F32)
            v[e] = e < n ? __builtin_bit_cast(unsigned, t[e]) : 0u;
        else
            v[e / 2] |= e < n ? (unsigned)t[e] << (16 * (e & 1)) : 0u;
    }
    return v;
}

// V values from p on, all inside; zeros where !keep (p is then any readable
// place).  Branch-free: loads behind per-lane branches wait for one another.
template <int DT>
__device__ __forceinline__ uintx4 load_whole(const typename Type<DT>::T *p, bool keep = true) {
    uintx4 v;
    __builtin_memcpy(&v, p, 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = keep ? v[q] : 0u;
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
                for (int q = 0; q < RB; ++q) r.w[u][q] = load_any<DT>(w[q] + kk);
#pragma unroll
                for (int q = 0; q < TB; ++q) r.x[u][q] = load_any<DT>(x[q] + kk);
            }
            return;
        }
        // the last round: whole steps, one that ends inside, and none
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ku = k + u * KS, kk = ku + kg;
            if (ku + KS <= k1) {
#pragma unroll
                for (int q = 0; q < RB; ++q) r.w[u][q] = load_any<DT>(w[q] + kk);
#pragma unroll
                for (int q = 0; q < TB; ++q) r.x[u][q] = load_any<DT>(x[q] + kk);
            } else if (ku < k1) {
#pragma unroll
                for (int q = 0; q < RB; ++q) r.w[u][q] = load_frag<DT>(w[q] + kk, k1 - kk, w[q]);
#pragma unroll
                for (int q = 0; q < TB; ++q) r.x[u][q] = load_frag<DT>(x[q] + kk, k1 - kk, x[q]);
            } else {
#pragma unroll
                for (int q = 0; q < RB; ++q) r.w[u][q] = uintx4{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < TB; ++q) r.x[u][q] = uintx4{0, 0, 0, 0};
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

// ---- staged form ---------------------------------------------------------------
// acc[r][t] += the products of 16 RB weight rows and 16 TB token rows, the weights
// passing through a ring of two stages in LDS that belongs to this wave alone
// (no barriers).  A direct load copies whole runs of 512 / RB bytes of a row,
// where fragments loaded straight into registers take 64 bytes of each of 16
// rows at a time: 16 x 14336 x 4096 bf16 24.5 us against 34.  A stage is 8 KB: KST
// values of k of every row.  The waves of a workgroup take the stages in turn.
// Needs rows of 16-byte chunks; what lies outside (rows past the end, chunks
// past kend) reads as zero.
//
// Order of the loads of stage s: its token fragments, then the weights of stage
// s + 1; with all but the last 8 loads waited for, both operands of stage s are
// there and the weights of stage s + 1 are in flight.
constexpr int kStageBytes = 8192;
template <int DT, int RB>
constexpr int kStageK = 512 / RB / (int)sizeof(typename Type<DT>::T);   // KST

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, 0x7fffffff, 0x00020000);
}

// Whether a matrix's rows serve the staged form: whole 16-byte chunks, and 64
// rows within 31 bits of byte offsets.
inline bool stage_ok(const void *p, long long ld, int len, int elem) {
    return rows16(p, ld, elem) && (long long)len * elem % 16 == 0 && 64 * ld * elem < 0x7fff0000LL;
}

// w: the weights at k = 0, row_at(r): byte offset of row r of the strip (kOut:
// outside, zeros); x: the tokens at k = 0, xoff[t]: byte offset of this lane's
// row of token block t.  The wave takes
// the stages first, first + step, ... below kend / KST.  ring: 2 * kStageBytes.
constexpr int kOut = (int)0x80000000u;
template <int DT, int RB, int TB, class RowAt>
__device__ __forceinline__ void staged_dot(const typename Type<DT>::T *w, RowAt row_at,
                                           const typename Type<DT>::T *x, const int (&xoff)[TB],
                                           int k0, int kend, int first, int step,
                                           unsigned char *ring, int lane, floatx4 (&acc)[RB][TB]) {
    using T = typename Type<DT>::T;
    constexpr int V = Step<DT>::V, KST = kStageK<DT, RB>, ROW = 512 / RB, CH = ROW / 16;
    constexpr int STEPS = CH / 4, E = (int)sizeof(T);
    typedef __attribute__((address_space(3))) void lds_void;
    const int i = lane & 15, g = lane >> 4;
    // 16 lanes read one chunk of 16 rows: their slots differ mod 256 bytes
    auto swz = [](int r) { return CH == 8 ? (r >> 1) & 7 : r & 15; };
    int off[8], kk[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int q = j * 64 + lane, r = q / CH, c = (q % CH) ^ swz(r);
        kk[j] = c * V;
        const int at = row_at(r);
        off[j] = at == kOut ? kOut : at + c * 16;
    }
    const int stages = (kend - k0 + KST - 1) / KST;
    auto load_w = [&](int s, int slot) {
        const int k = k0 + s * KST, krem = s < stages ? kend - k : 0;
        const __amdgpu_buffer_rsrc_t b = row_buffer(w + k);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                b, (lds_void *)(ring + slot * kStageBytes + j * 1024), 16,
                kk[j] < krem ? off[j] : kOut, 0, 0, 0);
    };
    if (first >= stages) return;
    load_w(first, 0);
    int slot = 0;
    for (int s = first; s < stages; s += step, slot ^= 1) {
        const int k = k0 + s * KST;
        const __amdgpu_buffer_rsrc_t xb = row_buffer(x + k);
        uintx4 fx[STEPS][TB];
#pragma unroll
        for (int u = 0; u < STEPS; ++u)
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int kc = V * (4 * u + g);
                fx[u][t] = __builtin_bit_cast(
                    uintx4, __builtin_amdgcn_raw_buffer_load_b128(
                                xb, k + kc < kend ? xoff[t] + kc * E : kOut, 0, 0));
            }
        pipeline_fence();
        load_w(s + step, slot ^ 1);
        pipeline_fence();
        __builtin_amdgcn_s_waitcnt(8 | (7 << 4) | (15 << 8));   // all but the last 8 loads
        pipeline_fence();
        const unsigned char *img = ring + slot * kStageBytes;
#pragma unroll
        for (int u = 0; u < STEPS; ++u)
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int row = 16 * r + i;
                const uintx4 fw = *reinterpret_cast<const uintx4 *>(
                    img + row * ROW + (((4 * u + g) ^ swz(row)) << 4));
#pragma unroll
                for (int t = 0; t < TB; ++t) acc[r][t] = mfma_step<DT>(fw, fx[u][t], acc[r][t]);
            }
        // the reads of this stage are done before its place is loaded again
        pipeline_fence();
        __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
        pipeline_fence();
    }
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));   // no load left in flight
    pipeline_fence();
}

}  // namespace sg
