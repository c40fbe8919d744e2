// moe.hip -- a whole mixture-of-experts layer for a few tokens:
//     logits = X Wr^T, p = softmax(logits), the k largest of each token
//     h_j = act(Wg[e_j] x) * (Wu[e_j] x)   (or act(W1[e_j] x), plain experts)
//     y   = sum_j w_j W2[e_j] h_j
// Bound by reading the chosen experts' weights once: with T tokens a weight
// value is used for at most 2T operations.
#include "stream_rows.hpp"

namespace sg {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kPairs = kMoeTokens * kMoeChoices;

struct MoeWs {
    double *logits;      // T x E
    int *ids;            // T x k
    float *w;            // T x k
    void *hi, *lo;       // T k x fp: h, and what its rounding left over
    float *part;         // T k x dp: the experts' results, unscaled
    unsigned *routed;    // per token: workgroups of the router that are done
    unsigned *joined;    // per 16 columns of Y: experts that are done
    int fp, dp;
};

// ---- router -----------------------------------------------------------------
// One wave per (token, expert): the logit is summed in fp64 (products of two
// inputs are exact there), so that the choice of the k largest does not depend
// on the order of a rounded sum; the workgroup of a token that ends last picks
// its k largest and their weights.
template <int DT>
__global__ void __launch_bounds__(kThreads) router_kernel(Moe m, MoeWs s) {
    using Ty = Type<DT>;
    using T = typename Ty::T;
    constexpr int V = Ty::V;
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.y, e = blockIdx.x * kWaves + wave;
    if (e < m.E) {
        const T *x = static_cast<const T *>(m.X) + (long long)t * m.ldx;
        const T *w = static_cast<const T *>(m.Wr) + (long long)e * m.ldwr;
        double sum = 0.0;
        for (int d = lane * V; d < m.D; d += 64 * V) {
            const uintx4 a = load_frag<DT>(x + d, m.D - d), b = load_frag<DT>(w + d, m.D - d);
            T av[V], bv[V];
            __builtin_memcpy(av, &a, 16);
            __builtin_memcpy(bv, &b, 16);
#pragma unroll
            for (int q = 0; q < V; ++q) sum = fma((double)Ty::load(av[q]), (double)Ty::load(bv[q]), sum);
        }
#pragma unroll
        for (int o = 32; o >= 1; o /= 2) sum += __shfl_xor(sum, o);
        if (lane == 0)
            __hip_atomic_store(reinterpret_cast<unsigned long long *>(s.logits + (long long)t * m.E + e),
                               __builtin_bit_cast(unsigned long long, sum), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!arrive_last(s.routed + t, gridDim.x, &last)) return;
    if (threadIdx.x == 0) __hip_atomic_store(s.routed + t, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (wave != 0) return;
    constexpr int PER = kMoeExperts / 64;
    double v[PER];
    bool free_[PER], nan = false;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int id = q * 64 + lane;
        free_[q] = id < m.E;
        v[q] = -INFINITY;
        if (free_[q]) {
            v[q] = __builtin_bit_cast(double,
                                      __hip_atomic_load(reinterpret_cast<unsigned long long *>(
                                                            s.logits + (long long)t * m.E + id),
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            if (v[q] != v[q]) {   // a NaN ranks lowest and makes every weight NaN
                nan = true;
                v[q] = -INFINITY;
            }
        }
    }
    nan = __any(nan);
    double top = 0.0, mine = 0.0, chosen = 0.0, all = 0.0;
    int id = 0;
    for (int j = 0; j < m.k; ++j) {
        double bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (free_[q] && (v[q] > bv || bi == 0x7fffffff)) {   // ascending ids: ties keep the first
                bv = v[q];
                bi = q * 64 + lane;
            }
#pragma unroll
        for (int o = 32; o >= 1; o /= 2) {
            const double ov = __shfl_xor(bv, o);
            const int oi = __shfl_xor(bi, o);
            if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) {
                bv = ov;
                bi = oi;
            }
        }
        if (j == 0) {
            top = bv;
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (free_[q]) all += exp(v[q] - top);
        }
        const double w = exp(bv - top);
        chosen += w;
        if (lane == j) {
            mine = w;
            id = bi;
        }
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (bi == q * 64 + lane) free_[q] = false;
    }
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) all += __shfl_xor(all, o);
    if (lane < m.k) {
        const float w = nan ? __builtin_nanf("") : (float)(mine / (m.renorm ? chosen : all));
        s.ids[t * m.k + lane] = id;
        s.w[t * m.k + lane] = w;
        if (m.ids) m.ids[t * m.k + lane] = id;
        if (m.weights) m.weights[t * m.k + lane] = w;
    }
}

// ---- experts ----------------------------------------------------------------
// The `want`-th expert in use (ascending) and its choices, as indexes t k + j.
struct Expert {
    int id[kPairs];
    int count[kMoeExperts];
    int pairs[kMoeTokens];
    int expert, n, active;   // n: choices of it; active: experts in use
};

__device__ __forceinline__ void find_expert(const Moe &m, const int *ids, int want, Expert &x) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int P = m.T * m.k;
    for (int e = tid; e < m.E; e += kThreads) x.count[e] = 0;
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) {
        x.id[p] = ids[p];
        atomicAdd(&x.count[x.id[p]], 1);
    }
    __syncthreads();
    if (tid < 64) {
        int seen = 0, found = -1;
        for (int e0 = 0; e0 < m.E; e0 += 64) {
            const bool used = e0 + lane < m.E && x.count[e0 + lane] > 0;
            const unsigned long long mask = __ballot(used);
            const int rank = seen + __popcll(mask & ((1ull << lane) - 1));
            const unsigned long long hit = __ballot(used && rank == want);
            if (hit) found = e0 + __ffsll(hit) - 1;
            seen += __popcll(mask);
        }
        int n = 0;
        if (found >= 0)
            for (int p0 = 0; p0 < P; p0 += 64) {
                const bool hit = p0 + lane < P && x.id[p0 + lane] == found;
                const unsigned long long mask = __ballot(hit);
                if (hit) x.pairs[n + __popcll(mask & ((1ull << lane) - 1))] = p0 + lane;
                n += __popcll(mask);
            }
        if (lane == 0) {
            x.expert = found;
            x.n = n;
            x.active = seen;
        }
    }
    __syncthreads();
}

// Sums of the four waves' accumulators of token block `wave`.
template <int RB, int TB>
__device__ __forceinline__ void join_waves(const floatx4 (&acc)[RB][TB],
                                           floatx4 (*red)[kWaves][64], int wave, int lane,
                                           floatx4 (&sum)[RB]) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
        for (int t = 0; t < TB; ++t) red[t][wave][lane] = acc[r][t];
        __syncthreads();
        sum[r] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (wave < TB)
#pragma unroll
            for (int z = 0; z < kWaves; ++z)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[r][e] += red[wave][z][lane][e];
        __syncthreads();
    }
}

// 16 rows of the first product(s) of one expert for its tokens.
template <int DT, bool GATED, int TB>
__device__ __forceinline__ void up_strip(const Moe &m, const MoeWs &s, const Expert &x, int f0,
                                         floatx4 (*red)[kWaves][64]) {
    using T = typename Type<DT>::T;
    constexpr int RB = GATED ? 2 : 1, KS = Step<DT>::K;
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const T *W = static_cast<const T *>(m.W1) + (long long)x.expert * m.stride1;
    const T *w[RB], *tok[TB];
    const int row = min(f0 + i, m.F - 1);
    w[0] = W + (long long)row * m.ld1;
    if constexpr (GATED) w[1] = W + (long long)(m.F + row) * m.ld1;
#pragma unroll
    for (int t = 0; t < TB; ++t)
        tok[t] = static_cast<const T *>(m.X) +
                 (long long)(x.pairs[min(16 * t + i, x.n - 1)] / m.k) * m.ldx;
    const int per = ((m.D + kWaves - 1) / kWaves + KS - 1) / KS * KS;
    floatx4 acc[RB][TB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[r][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    stream_dot<DT, RB, TB, TB == 1 ? 4 : 2>(w, tok, wave * per, min((wave + 1) * per, m.D), lane, acc);
    floatx4 sum[RB];
    join_waves<RB, TB>(acc, red, wave, lane, sum);
    const int slot = 16 * wave + i;
    if (wave >= TB || slot >= x.n) return;
    const long long at = (long long)x.pairs[slot] * s.fp + f0 + 4 * g;
    with_act(m.act, [&](auto tag) {
        float h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[e] = activate_t<decltype(tag)::value>(sum[0][e]);
            if constexpr (GATED) h[e] *= sum[1][e];
        }
        using Ty = Type<DT>;
        T hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = Ty::store(h[e]);
            const float d = h[e] - Ty::load(hi[e]);
            lo[e] = Ty::store(fabsf(d) < INFINITY ? d : 0.f);
        }
        __builtin_memcpy(static_cast<T *>(s.hi) + at, hi, sizeof(hi));
        if (DT != SGEMM_DTYPE_F32) __builtin_memcpy(static_cast<T *>(s.lo) + at, lo, sizeof(lo));
    });
}

template <int DT, bool GATED, int TB>
__global__ void __launch_bounds__(kThreads) up_kernel(Moe m, MoeWs s) {
    __shared__ Expert x;
    __shared__ floatx4 red[TB][kWaves][64];
    find_expert(m, s.ids, blockIdx.y, x);
    if (x.expert < 0) return;
    const int f0 = blockIdx.x * 16;
    if (TB == 1 || x.n <= 16)
        up_strip<DT, GATED, 1>(m, s, x, f0, red);
    else if (TB == 2 || x.n <= 32)
        up_strip<DT, GATED, TB < 2 ? 1 : 2>(m, s, x, f0, red);
    else
        up_strip<DT, GATED, TB>(m, s, x, f0, red);
}

// 16 rows of the second product of one expert for its tokens.  h in two parts
// (16-bit types): its rounding would otherwise be as large as that of Y.
template <int DT, int TB>
__device__ __forceinline__ void down_strip(const Moe &m, const MoeWs &s, const Expert &x, int d0,
                                           floatx4 (*red)[kWaves][64]) {
    using T = typename Type<DT>::T;
    constexpr int PARTS = DT == SGEMM_DTYPE_F32 ? 1 : 2, KS = Step<DT>::K;
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const T *w[1] = {static_cast<const T *>(m.W2) + (long long)x.expert * m.stride2 +
                     (long long)min(d0 + i, m.D - 1) * m.ld2};
    const T *h[PARTS * TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const long long at = (long long)x.pairs[min(16 * t + i, x.n - 1)] * s.fp;
        h[t] = static_cast<const T *>(s.hi) + at;
        if constexpr (PARTS == 2) h[TB + t] = static_cast<const T *>(s.lo) + at;
    }
    const int per = ((m.F + kWaves - 1) / kWaves + KS - 1) / KS * KS;
    floatx4 acc[1][PARTS * TB];
#pragma unroll
    for (int t = 0; t < PARTS * TB; ++t) acc[0][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    stream_dot<DT, 1, PARTS * TB, TB == 1 ? 4 : 2>(
        w, h, wave * per, min((wave + 1) * per, m.F), lane, acc);
    floatx4 both[1][TB], sum[1];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            both[0][t][e] = PARTS == 2 ? acc[0][t][e] + acc[0][PARTS * TB - TB + t][e] : acc[0][t][e];
    join_waves<1, TB>(both, red, wave, lane, sum);
    const int slot = 16 * wave + i;
    if (wave < TB && slot < x.n)
        store_partial(s.part + (long long)x.pairs[slot] * s.dp + d0 + 4 * g, sum[0]);
}

template <int DT, int TB>
__global__ void __launch_bounds__(kThreads) down_kernel(Moe m, MoeWs s) {
    __shared__ Expert x;
    __shared__ floatx4 red[TB][kWaves][64];
    __shared__ int last;
    find_expert(m, s.ids, blockIdx.y, x);
    if (x.expert < 0) return;
    const int d0 = blockIdx.x * 16;
    if (TB == 1 || x.n <= 16)
        down_strip<DT, 1>(m, s, x, d0, red);
    else if (TB == 2 || x.n <= 32)
        down_strip<DT, TB < 2 ? 1 : 2>(m, s, x, d0, red);
    else
        down_strip<DT, TB>(m, s, x, d0, red);
    // the expert that ends last adds up every token's choices, in order
    if (!arrive_last(s.joined + blockIdx.x, x.active, &last)) return;
    const int tid = threadIdx.x, t = tid >> 2, d = d0 + 4 * (tid & 3);
    if (t < m.T && d < m.D) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < m.k; ++j) {
            const floatx4 v = load_partial(s.part + (long long)(t * m.k + j) * s.dp + d);
            const float w = s.w[t * m.k + j];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = fmaf(w, v[e], y[e]);
        }
        Prod p{m.T, m.D, 0, nullptr, 0, nullptr, 0, m.Y, m.ldy};
        p.cvec = 0;
        finish_run<DT, SGEMM_ACT_NONE>(p, t, d, y);
    }
    if (tid == 0)
        __hip_atomic_store(s.joined + blockIdx.x, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// The workspace's parts, in order; returns the bytes.
size_t lay_out(int dtype, const Moe &m, const Workspace *ws, MoeWs &s) {
    const size_t elem = dtype == SGEMM_DTYPE_F32 ? 4 : 2, P = (size_t)m.T * m.k;
    s.fp = (int)round_up(m.F, 16);
    s.dp = (int)round_up(m.D, 16);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char *q = ws ? static_cast<unsigned char *>(ws->ptr) + at : nullptr;
        at += round_up(bytes, 256);
        return q;
    };
    s.logits = reinterpret_cast<double *>(take((size_t)m.T * m.E * 8));
    s.ids = reinterpret_cast<int *>(take(P * 4));
    s.w = reinterpret_cast<float *>(take(P * 4));
    s.hi = take(P * s.fp * elem);
    s.lo = take(elem == 2 ? P * s.fp * elem : 0);
    s.part = reinterpret_cast<float *>(take(P * s.dp * 4));
    s.routed = ws ? ws->counters : nullptr;
    s.joined = ws ? ws->counters + kMoeTokens : nullptr;
    return at;
}

template <int DT, int TB>
hipError_t launch_tb(const Moe &m, const MoeWs &s, hipStream_t stream) {
    const int active = m.T * m.k < m.E ? m.T * m.k : m.E;
    hipLaunchKernelGGL((router_kernel<DT>), dim3((m.E + kWaves - 1) / kWaves, m.T), dim3(kThreads),
                       0, stream, m, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 up(s.fp / 16, active), down(s.dp / 16, active);
    if (m.gated)
        hipLaunchKernelGGL((up_kernel<DT, true, TB>), up, dim3(kThreads), 0, stream, m, s);
    else
        hipLaunchKernelGGL((up_kernel<DT, false, TB>), up, dim3(kThreads), 0, stream, m, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((down_kernel<DT, TB>), down, dim3(kThreads), 0, stream, m, s);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const Moe &m, const MoeWs &s, hipStream_t stream) {
    if (m.T <= 16) return launch_tb<DT, 1>(m, s, stream);
    if (m.T <= 32) return launch_tb<DT, 2>(m, s, stream);
    return launch_tb<DT, 4>(m, s, stream);
}

}  // namespace

size_t moe_workspace(int dtype, const Moe &m) {
    MoeWs s;
    return lay_out(dtype, m, nullptr, s);
}

hipError_t launch_moe(int dtype, const Moe &m, const Workspace &ws, hipStream_t stream) {
    MoeWs s;
    lay_out(dtype, m, &ws, s);
    switch (dtype) {
    case SGEMM_DTYPE_BF16: return launch_dt<SGEMM_DTYPE_BF16>(m, s, stream);
    case SGEMM_DTYPE_F16: return launch_dt<SGEMM_DTYPE_F16>(m, s, stream);
    default: return launch_dt<SGEMM_DTYPE_F32>(m, s, stream);
    }
}

}  // namespace sg
