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

// How the tokens' choices are laid out for the experts: choice p = t k + j.
struct Routing {
    int active;                   // experts in use
    int expert[kMoeExperts];      // of the a-th: its index,
    int first[kMoeExperts];       // where its choices start in `list`,
    int count[kMoeExperts];       // and how many there are
    int list[kPairs];
};

struct MoeWs {
    double *logits;      // T x E
    int *ids;            // T x k
    float *w;            // T x k
    Routing *routing;
    void *h;             // T k x PARTS x fp: h, and what its rounding left over
    float *part;         // T k x dp: the experts' results, unscaled
    unsigned *routed;    // per token: workgroups of the router that are done
    unsigned *chosen;    // tokens whose experts are chosen
    unsigned *joined;    // per strip of Y: experts that are done
    int fp, dp;
};

// ---- router -----------------------------------------------------------------
// A wave takes one token and EPW experts.  The logits are summed in fp64
// (products of two inputs are exact there), so that the choice of the k largest
// does not depend on the order of a rounded sum.  The workgroup of a token that
// ends last chooses its experts: an expert's rank is the number of those before
// it, counted by one thread per expert, and rank j < k is choice j.  The
// workgroup that chooses for the last token lays out the choices by expert.
template <int DT, int EPW>
__global__ void __launch_bounds__(kThreads) router_kernel(Moe m, MoeWs s) {
    using Ty = Type<DT>;
    using T = typename Ty::T;
    constexpr int V = Ty::V;
    __shared__ int last;
    __shared__ double lg[kMoeExperts];
    __shared__ double red[kWaves];
    __shared__ double best[kMoeChoices];
    __shared__ int best_id[kMoeChoices];
    __shared__ unsigned long long users[kMoeExperts];   // the tokens that chose an expert
    __shared__ int first_of[kMoeExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = blockIdx.y, e0 = (blockIdx.x * kWaves + wave) * EPW;
    if (e0 < m.E) {
        const T *x = static_cast<const T *>(m.X) + (long long)t * m.ldx;
        const T *w[EPW];
        double sum[EPW];
#pragma unroll
        for (int q = 0; q < EPW; ++q) {
            w[q] = static_cast<const T *>(m.Wr) + (long long)min(e0 + q, m.E - 1) * m.ldwr;
            sum[q] = 0.0;
        }
        // U chunks' loads in flight: a few tokens' logits wait for memory only
        constexpr int U = EPW == 1 ? 4 : 2;
        for (int d1 = 0; d1 < m.D; d1 += U * 64 * V) {
            const int d0 = d1 + lane * V;
            uintx4 a[U], b[U][EPW];
            if (d1 + U * 64 * V <= m.D) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    a[u] = load_whole<DT>(x + d0 + u * 64 * V);
#pragma unroll
                    for (int q = 0; q < EPW; ++q) b[u][q] = load_whole<DT>(w[q] + d0 + u * 64 * V);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int d = d0 + u * 64 * V;
                    a[u] = load_frag<DT>(x + d, m.D - d, x);
#pragma unroll
                    for (int q = 0; q < EPW; ++q) b[u][q] = load_frag<DT>(w[q] + d, m.D - d, w[q]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                T av[V];
                __builtin_memcpy(av, &a[u], 16);
#pragma unroll
                for (int q = 0; q < EPW; ++q) {
                    T bv[V];
                    __builtin_memcpy(bv, &b[u][q], 16);
#pragma unroll
                    for (int z = 0; z < V; ++z)
                        sum[q] = fma((double)Ty::load(av[z]), (double)Ty::load(bv[z]), sum[q]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < EPW; ++q) {
#pragma unroll
            for (int o = 32; o >= 1; o /= 2) sum[q] += __shfl_xor(sum[q], o);
            if (lane == 0 && e0 + q < m.E)
                __hip_atomic_store(
                    reinterpret_cast<unsigned long long *>(s.logits + (long long)t * m.E + e0 + q),
                    __builtin_bit_cast(unsigned long long, sum[q]), __ATOMIC_RELAXED,
                    __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (!arrive_last(s.routed + t, gridDim.x, &last)) return;
    if (tid == 0) __hip_atomic_store(s.routed + t, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

    // a NaN ranks lowest, with -inf, and makes every weight NaN
    bool nan = false;
    for (int e = tid; e < m.E; e += kThreads) {
        const double v = __builtin_bit_cast(
            double, __hip_atomic_load(
                        reinterpret_cast<unsigned long long *>(s.logits + (long long)t * m.E + e),
                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        nan |= v != v;
        lg[e] = v == v ? v : -INFINITY;
    }
    nan = __syncthreads_or(nan);
    for (int e = tid; e < m.E; e += kThreads) {
        const double v = lg[e];
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < m.E; ++o) rank += lg[o] > v || (lg[o] == v && o < e);
        if (rank < m.k) {
            best[rank] = v;
            best_id[rank] = e;
        }
    }
    __syncthreads();
    const double top = best[0];
    const double mine = lane < m.k ? exp(best[lane] - top) : 0.0;
    double all = mine;
    if (!m.renorm) {
        all = 0.0;
        for (int e = tid; e < m.E; e += kThreads) all += exp(lg[e] - top);
    }
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) all += __shfl_xor(all, o);
    if (!m.renorm) {   // the waves hold different experts' terms
        if (lane == 0) red[wave] = all;
        __syncthreads();
        all = ((red[0] + red[1]) + red[2]) + red[3];
    }
    if (tid < m.k) {
        const float w = nan ? __builtin_nanf("") : (float)(mine / all);
        const int id = best_id[tid];
        __hip_atomic_store(s.ids + t * m.k + tid, id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s.w[t * m.k + tid] = w;
        if (m.ids) m.ids[t * m.k + tid] = id;
        if (m.weights) m.weights[t * m.k + tid] = w;
    }
    if (m.T > 1 && !arrive_last(s.chosen, m.T, &last)) return;
    if (m.T > 1 && tid == 0) __hip_atomic_store(s.chosen, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

    // the choices by expert, ascending: a token chooses an expert once at most,
    // so an expert's choices are a mask of tokens
    static_assert(kMoeTokens <= 64, "a bit per token");
    const int P = m.T * m.k;
    Routing *r = s.routing;
    for (int e = tid; e < kMoeExperts; e += kThreads) users[e] = 0;
    __syncthreads();
    int chosen[kPairs / kThreads];
#pragma unroll
    for (int q = 0; q < kPairs / kThreads; ++q) {
        const int p = q * kThreads + tid;
        if (p >= P) break;
        chosen[q] = m.T == 1 ? best_id[p]
                           : __hip_atomic_load(s.ids + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        atomicOr(&users[chosen[q]], 1ull << (p / m.k));
    }
    __syncthreads();
    if (wave == 0) {
        int active = 0, first = 0;
        for (int b = 0; b < m.E; b += 64) {
            const int n = __popcll(users[b + lane]);
            const unsigned long long mask = __ballot(n > 0);
            int before = n;   // inclusive sum over the lanes
#pragma unroll
            for (int o = 1; o < 64; o *= 2) {
                const int v = __shfl_up(before, o);
                if (lane >= o) before += v;
            }
            first_of[b + lane] = first + before - n;
            if (n > 0) {
                const int a = active + __popcll(mask & ((1ull << lane) - 1));
                r->expert[a] = b + lane;
                r->first[a] = first + before - n;
                r->count[a] = n;
            }
            active += __popcll(mask);
            first += __shfl(before, 63);
        }
        if (lane == 0) r->active = active;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPairs / kThreads; ++q) {
        const int p = q * kThreads + tid;
        if (p >= P) break;
        const unsigned long long earlier = users[chosen[q]] & ((1ull << (p / m.k)) - 1);
        r->list[first_of[chosen[q]] + __popcll(earlier)] = p;
    }
}

// ---- experts ----------------------------------------------------------------
// A strip is 32 rows of weights: of the first product 16 gate and 16 up rows, or
// 32 plain ones; of the second, 32 rows of W2.  NW waves share a strip, taking
// its stages (staged_dot) or quarters of k (stream_dot, rows of any alignment)
// in turn and meeting in LDS; with NW == 1 there is nothing to meet for, and
// eight strips and more stream on a CU independently.
//
// In the second product each choice of a 16-bit layer is two columns, h rounded
// and what the rounding left over (the rounding of h would otherwise add an
// error as large as that of Y; a matrix instruction has 16 columns, most of
// them idle with few choices per expert).
template <int DT>
constexpr int kParts = DT == SGEMM_DTYPE_F32 ? 1 : 2;
constexpr int kStrip = 32;

struct Strip {
    int expert, n;       // the expert and its choices
    const int *list;
};

template <int NW, bool STAGED>
constexpr int kLds = STAGED ? NW * 2 * kStageBytes : 2 * NW * 1024;   // (times TB)

// Sums of the waves' accumulators of 16-column block `tb` (each wave that calls
// takes another): [row block][rows of the lane].
template <int NW, int TB>
__device__ __forceinline__ void meet(floatx4 (&acc)[2][TB], unsigned char *smem, int wave, int lane) {
    if constexpr (NW > 1) {
        static_assert(TB <= 4 || NW == 1, "sums of all waves fit LDS");
        floatx4 *red = reinterpret_cast<floatx4 *>(smem);
        __syncthreads();   // no wave's stages are in use any more
#pragma unroll
        for (int q = 0; q < 2 * TB; ++q) red[(q * NW + wave) * 64 + lane] = acc[q / TB][q % TB];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2 * TB; ++q) {
            if ((q % TB) % NW != wave) continue;   // block t is wave t % NW's
            floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int z = 0; z < NW; ++z) {
                const floatx4 v = red[(q * NW + z) * 64 + lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += v[e];
            }
            acc[q / TB][q % TB] = s;
        }
    }
}

template <int DT, bool GATED, int NW, bool STAGED, int TB>
__device__ __forceinline__ void up_strip(const Moe &m, const MoeWs &s, const Strip &x, int f0,
                                         unsigned char *smem) {
    using Ty = Type<DT>;
    using T = typename Ty::T;
    constexpr int PARTS = kParts<DT>, E = (int)sizeof(T);
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *W = static_cast<const T *>(m.W1) + (long long)x.expert * m.stride1;
    const T *X = static_cast<const T *>(m.X);
    int pair[TB], xoff[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {   // columns past the last repeat it; they are not stored
        pair[t] = x.list[min(16 * t + i, x.n - 1)];
        xoff[t] = pair[t] / m.k * (int)m.ldx * E;
    }
    floatx4 acc[2][TB];
#pragma unroll
    for (int q = 0; q < 2 * TB; ++q) acc[q / TB][q % TB] = floatx4{0.f, 0.f, 0.f, 0.f};
    if constexpr (STAGED) {
        const int second = GATED ? (int)(m.F * m.ld1) * E : 16 * (int)m.ld1 * E;
        staged_dot<DT, 2, TB>(
            W + (long long)f0 * m.ld1,
            [&](int r) {
                const int in = r & 15, f = f0 + (GATED ? in : r);
                return f < m.F ? in * (int)m.ld1 * E + (r >= 16 ? second : 0) : kOut;
            },
            X, xoff, 0, m.D, wave, NW, smem + wave * 2 * kStageBytes, lane, acc);
    } else {
        constexpr int KS = Step<DT>::K;
        const T *w[2], *tok[TB];
        w[0] = W + (long long)min(f0 + i, m.F - 1) * m.ld1;
        w[1] = GATED ? w[0] + (long long)m.F * m.ld1 : W + (long long)min(f0 + 16 + i, m.F - 1) * m.ld1;
#pragma unroll
        for (int t = 0; t < TB; ++t) tok[t] = X + (long long)(pair[t] / m.k) * m.ldx;
        const int per = ((m.D + NW - 1) / NW + KS - 1) / KS * KS;
        stream_dot<DT, 2, TB, TB == 1 ? 4 : 2>(w, tok, wave * per, min((wave + 1) * per, m.D), lane, acc);
    }
    meet<NW, TB>(acc, smem, wave, lane);
    with_act(m.act, [&](auto tag) {
        constexpr int ACT = decltype(tag)::value;
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if (t % NW != wave || 16 * t + i >= x.n) continue;
#pragma unroll
            for (int r = 0; r < (GATED ? 1 : 2); ++r) {
                const int f = f0 + 16 * r + 4 * g;
                if (f >= s.fp) continue;
                T hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float h = activate_t<ACT>(acc[r][t][e]);
                    if constexpr (GATED) h *= acc[1][t][e];
                    hi[e] = Ty::store(h);
                    const float d = h - Ty::load(hi[e]);
                    lo[e] = Ty::store(fabsf(d) < INFINITY ? d : 0.f);
                }
                T *to = static_cast<T *>(s.h) + (long long)pair[t] * PARTS * s.fp + f;
                __builtin_memcpy(to, hi, sizeof(hi));
                if constexpr (PARTS == 2) __builtin_memcpy(to + s.fp, lo, sizeof(lo));
            }
        }
    });
}

template <int DT, int NW, bool STAGED, int TB>
__device__ __forceinline__ void down_strip(const Moe &m, const MoeWs &s, const Strip &x, int d0,
                                           unsigned char *smem) {
    using T = typename Type<DT>::T;
    constexpr int PARTS = kParts<DT>, E = (int)sizeof(T), KS = Step<DT>::K;
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *W = static_cast<const T *>(m.W2) + (long long)x.expert * m.stride2;
    const T *H = static_cast<const T *>(s.h);
    int pair[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) pair[t] = x.list[min((16 * t + i) / PARTS, x.n - 1)];
    const int part = PARTS == 2 ? i & 1 : 0;
    floatx4 acc[2][TB];
#pragma unroll
    for (int q = 0; q < 2 * TB; ++q) acc[q / TB][q % TB] = floatx4{0.f, 0.f, 0.f, 0.f};
    if constexpr (STAGED) {
        int hoff[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) hoff[t] = (pair[t] * PARTS + part) * s.fp * E;
        staged_dot<DT, 2, TB>(
            W + (long long)d0 * m.ld2,
            [&](int r) { return d0 + r < m.D ? r * (int)m.ld2 * E : kOut; }, H, hoff, 0, m.F, wave, NW,
            smem + wave * 2 * kStageBytes, lane, acc);
    } else {
        const T *w[2] = {W + (long long)min(d0 + i, m.D - 1) * m.ld2,
                         W + (long long)min(d0 + 16 + i, m.D - 1) * m.ld2};
        const T *h[TB];
#pragma unroll
        for (int t = 0; t < TB; ++t) h[t] = H + (long long)(pair[t] * PARTS + part) * s.fp;
        const int per = ((m.F + NW - 1) / NW + KS - 1) / KS * KS;
        stream_dot<DT, 2, TB, TB == 1 ? 4 : TB == 2 ? 2 : 1>(w, h, wave * per,
                                                             min((wave + 1) * per, m.F), lane, acc);
    }
    meet<NW, TB>(acc, smem, wave, lane);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        if (t % NW != wave) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            floatx4 v = acc[r][t];
            if constexpr (PARTS == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], 1);   // the two parts
            const int d = d0 + 16 * r + 4 * g;
            if (part == 0 && (16 * t + i) / PARTS < x.n && d < s.dp)
                store_partial(s.part + (long long)pair[t] * s.dp + d, v);
        }
    }
}

// The a-th expert in use, or none.
__device__ __forceinline__ bool strip_of(const Routing *r, int a, Strip &x) {
    if (a >= r->active) return false;
    x.expert = r->expert[a];
    x.n = r->count[a];
    x.list = r->list + r->first[a];
    return true;
}

template <int DT, bool GATED, int NW, bool STAGED, int TB>
__global__ void __launch_bounds__(64 * NW) up_kernel(Moe m, MoeWs s) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    __shared__ __attribute__((aligned(1024))) unsigned char smem[kLds<NW, STAGED> * (STAGED ? 1 : TB)];
    Strip x;
    if (!strip_of(s.routing, blockIdx.y, x)) return;
    const int f0 = blockIdx.x * (GATED ? 16 : kStrip);
    if (TB == 1 || x.n <= 16)
        up_strip<DT, GATED, NW, STAGED, 1>(m, s, x, f0, smem);
    else if (TB == 2 || x.n <= 32)
        up_strip<DT, GATED, NW, STAGED, TB < 2 ? 1 : 2>(m, s, x, f0, smem);
    else
        up_strip<DT, GATED, NW, STAGED, TB>(m, s, x, f0, smem);
#endif
}

template <int DT, int NW, bool STAGED, int TB>
__global__ void __launch_bounds__(64 * NW) down_kernel(Moe m, MoeWs s) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    __shared__ __attribute__((aligned(1024))) unsigned char smem[kLds<NW, STAGED> * (STAGED ? 1 : TB)];
    constexpr int PER = 16 / kParts<DT>;   // choices per 16-column block
    Strip x;
    if (!strip_of(s.routing, blockIdx.y, x)) return;
    const int d0 = blockIdx.x * kStrip;
    // four blocks at a time at most
    constexpr int MOST = TB < 4 ? TB : 4;
    for (int done = 0, n = x.n; done < n; done += MOST * PER) {
        Strip y = x;
        y.list += done;
        y.n = min(n - done, MOST * PER);
        if (done) __syncthreads();
        if (MOST == 1 || y.n <= PER)
            down_strip<DT, NW, STAGED, 1>(m, s, y, d0, smem);
        else if (MOST == 2 || y.n <= 2 * PER)
            down_strip<DT, NW, STAGED, MOST < 2 ? 1 : 2>(m, s, y, d0, smem);
        else
            down_strip<DT, NW, STAGED, MOST>(m, s, y, d0, smem);
    }
    __syncthreads();
    // the expert that ends last adds up every token's choices, in order
    int *last = reinterpret_cast<int *>(smem);
    if (!arrive_last(s.joined + blockIdx.x, s.routing->active, last)) return;
    const int tid = threadIdx.x;
    Prod p{m.T, m.D, 0, nullptr, 0, nullptr, 0, m.Y, m.ldy};
    for (int q = tid; q < m.T * 8; q += 64 * NW) {
        const int t = q >> 3, d = d0 + 4 * (q & 7);
        if (d >= m.D) continue;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < m.k; j0 += 8) {
            floatx4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = j0 + j < m.k
                           ? load_partial(s.part + (long long)(t * m.k + j0 + j) * s.dp + d)
                           : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= m.k) continue;
                const float w = s.w[t * m.k + j0 + j];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = fmaf(w, v[j][e], y[e]);
            }
        }
        finish_run<DT, SGEMM_ACT_NONE>(p, t, d, y);
    }
    if (tid == 0)
        __hip_atomic_store(s.joined + blockIdx.x, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#endif
}

size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// The workspace's parts, in order; returns the bytes.
size_t lay_out(const Moe &m, const Workspace *ws, MoeWs &s) {
    const size_t P = (size_t)m.T * m.k;
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
    s.routing = reinterpret_cast<Routing *>(take(sizeof(Routing)));
    s.h = take(P * s.fp * 4);   // two parts of 2 bytes, or one of 4
    s.part = reinterpret_cast<float *>(take(P * s.dp * 4));
    s.routed = ws ? ws->counters : nullptr;
    s.chosen = ws ? ws->counters + kMoeTokens : nullptr;
    s.joined = ws ? ws->counters + kMoeTokens + 1 : nullptr;
    return at;
}

template <int DT, int NW, bool STAGED, int TB>
hipError_t launch_experts(const Moe &m, const MoeWs &s, hipStream_t stream) {
    const int active = m.T * m.k < m.E ? m.T * m.k : m.E;
    const int per = m.gated ? 16 : kStrip;
    const dim3 up((m.F + per - 1) / per, active), down((m.D + kStrip - 1) / kStrip, active);
    if (m.gated)
        hipLaunchKernelGGL((up_kernel<DT, true, NW, STAGED, TB>), up, dim3(64 * NW), 0, stream, m, s);
    else
        hipLaunchKernelGGL((up_kernel<DT, false, NW, STAGED, TB>), up, dim3(64 * NW), 0, stream, m, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int DTB = TB * kParts<DT> < 4 ? TB * kParts<DT> : 4;
    hipLaunchKernelGGL((down_kernel<DT, NW, STAGED, DTB>), down, dim3(64 * NW), 0, stream, m, s);
    return hipGetLastError();
}

template <int DT, int NW, bool STAGED>
hipError_t launch_tokens(const Moe &m, const MoeWs &s, hipStream_t stream) {
    if (m.T <= 16) return launch_experts<DT, NW, STAGED, 1>(m, s, stream);
    if (m.T <= 32) return launch_experts<DT, NW, STAGED, 2>(m, s, stream);
    return launch_experts<DT, NW, STAGED, 4>(m, s, stream);
}

template <int DT>
hipError_t launch_dt(const Moe &m, const MoeWs &s, hipStream_t stream) {
    constexpr int E = (int)sizeof(typename Type<DT>::T);
    // few (token, expert) products: a wave for each; many: four for each
    if ((long long)m.T * m.E < 2048)
        hipLaunchKernelGGL((router_kernel<DT, 1>), dim3((m.E + kWaves - 1) / kWaves, m.T),
                           dim3(kThreads), 0, stream, m, s);
    else
        hipLaunchKernelGGL((router_kernel<DT, 4>), dim3((m.E + 4 * kWaves - 1) / (4 * kWaves), m.T),
                           dim3(kThreads), 0, stream, m, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool staged = stage_ok(m.X, m.ldx, m.D, E) && stage_ok(m.W1, m.ld1, m.D, E) &&
                        stage_ok(m.W2, m.ld2, m.F, E) && m.stride1 * E % 16 == 0 &&
                        m.stride2 * E % 16 == 0 && (m.F + 32) * m.ld1 * E < 0x7fff0000LL &&
                        (long long)m.T * m.k * s.fp * 4 < 0x7fff0000LL;
    if (!staged) return launch_tokens<DT, 4, false>(m, s, stream);
    // with strips for every wave the CUs hold, a wave takes a whole strip;
    // with fewer, four share one
    const long long active = m.T * m.k < m.E ? m.T * m.k : m.E;
    const long long strips = active * ((m.F + 15) / 16 + (m.D + 31) / 32) / 2;
    if (strips >= 2048) return launch_tokens<DT, 1, true>(m, s, stream);
    return launch_tokens<DT, 4, true>(m, s, stream);
}

}  // namespace

size_t moe_workspace(const Moe &m) {
    MoeWs s;
    return lay_out(m, nullptr, s);
}

hipError_t launch_moe(int dtype, const Moe &m, const Workspace &ws, hipStream_t stream) {
    MoeWs s;
    lay_out(m, &ws, s);
    switch (dtype) {
    case SGEMM_DTYPE_BF16: return launch_dt<SGEMM_DTYPE_BF16>(m, s, stream);
    case SGEMM_DTYPE_F16: return launch_dt<SGEMM_DTYPE_F16>(m, s, stream);
    default: return launch_dt<SGEMM_DTYPE_F32>(m, s, stream);
    }
}

}  // namespace sg
