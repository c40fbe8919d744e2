// linear_rows.hip -- products of a linear layer with at most 64 rows, the
// shapes of decoding and of small batches' gradients:
//     rows_kernel   Y = act(X W^T + b) + R   W's rows run along k
//     cols_kernel   dX = G W                 k runs over W's rows
//     outer_kernel  dW = G^T X               k runs over the few rows
// The first two are bound by reading W once: at M = 16 a weight value of two bytes is
// used for 32 operations, far below the ~300 operations per byte at which the
// matrix cores would be the limit.
#include "stream_rows.hpp"

namespace sg {
namespace {

struct RowsGrid {
    int strips, slices, kslice;   // column strips, k slices, k per slice
    int width;                    // columns per strip
    float *part;                  // slices x strips x the strip's accumulators
    unsigned *count;              // one arrival counter per strip, zero between launches
};

constexpr int kWaves = 4, kThreads = 64 * kWaves;

// The sum over slices of the partial sums at(s), in order, eight loads in flight
// at a time (one after another each would wait for memory by itself).
template <class F>
__device__ __forceinline__ floatx4 sum_slices(int slices, F &&at) {
    floatx4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < slices; s += 8) {
        floatx4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = s + q < slices ? load_partial(at(s + q)) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (s + q < slices)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += v[q][e];
    }
    return sum;
}

// One strip of 16 rows of W per workgroup, the four waves taking contiguous
// quarters of the slice's k and meeting in LDS.
template <int DT, int TB, int U>
__global__ void __launch_bounds__(kThreads) rows_kernel(Prod p, RowsGrid gr) {
    using T = typename Type<DT>::T;
    constexpr int KS = Step<DT>::K;
    __shared__ floatx4 red[kWaves][TB][64];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x % gr.strips, slice = blockIdx.x / gr.strips;
    const int n0 = strip * 16;

    // rows past the edge repeat the last one: their results are not stored
    const T *w[1] = {static_cast<const T *>(p.B) + (long long)min(n0 + i, p.N - 1) * p.ldb};
    const T *x[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
        x[t] = static_cast<const T *>(p.A) + (long long)min(16 * t + i, p.M - 1) * p.lda;
    const int ks = slice * gr.kslice, ke = min(ks + gr.kslice, p.K);
    const int per = ((ke - ks + kWaves - 1) / kWaves + KS - 1) / KS * KS;
    const int k0 = ks + wave * per, k1 = min(k0 + per, ke);
    floatx4 acc[1][TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[0][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    stream_dot<DT, 1, TB, U>(w, x, k0, k1, lane, acc);

#pragma unroll
    for (int t = 0; t < TB; ++t) red[wave][t][lane] = acc[0][t];
    __syncthreads();
    const int t = wave;   // wave t finishes token block t
    floatx4 sum = {0.f, 0.f, 0.f, 0.f};
    if (t < TB) {
#pragma unroll
        for (int z = 0; z < kWaves; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += red[z][t][lane][e];
    }
    if (gr.slices > 1) {
        auto at = [&](int s) {
            return gr.part + ((((long long)s * gr.strips + strip) * TB + t) * 64 + lane) * 4;
        };
        if (t < TB) store_partial(at(slice), sum);
        if (!arrive_last(gr.count + strip, gr.slices, &last)) return;
        if (t < TB) sum = sum_slices(gr.slices, at);
        if (tid == 0)
            __hip_atomic_store(gr.count + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const int m = 16 * t + i;
    if (t >= TB || m >= p.M) return;
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    with_act(p.act, [&](auto tag) {
        finish_run<DT, decltype(tag)::value>(p, m, n0 + 4 * g, v);
    });
}

// Strips of `width` rows of W (at most 16 RB), staged (stream_rows.hpp), the
// eight waves taking the stages of a slice in turn and meeting in LDS.
template <int DT, int RB, int TB>
__global__ void __launch_bounds__(512) rows_staged_kernel(Prod p, RowsGrid gr) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    using T = typename Type<DT>::T;
    constexpr int NW = 8;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NW * 2 * kStageBytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x % gr.strips, slice = blockIdx.x / gr.strips;
    const int n0 = strip * gr.width, rows = min(gr.width, p.N - n0);
    int xoff[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) xoff[t] = min(16 * t + i, p.M - 1) * (int)p.lda * (int)sizeof(T);
    const int ks = slice * gr.kslice, ke = min(ks + gr.kslice, p.K);
    floatx4 acc[RB][TB];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[r][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    staged_dot<DT, RB, TB>(static_cast<const T *>(p.B) + (long long)n0 * p.ldb,
                           [&](int r) { return r < rows ? r * (int)p.ldb * (int)sizeof(T) : kOut; },
                           static_cast<const T *>(p.A), xoff, ks, ke, wave, NW,
                           smem + wave * 2 * kStageBytes, lane, acc);
    // the ring is this wave's own up to here; now every wave leaves its sums
    static_assert(NW * RB * TB * 1024 <= (int)sizeof(smem), "the waves' sums fit the ring");
    floatx4 *red = reinterpret_cast<floatx4 *>(smem);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) red[((r * TB + t) * NW + wave) * 64 + lane] = acc[r][t];
    __syncthreads();
    // wave v finishes blocks v, v + 8, ... of the strip's RB x TB
    auto sum_of = [&](int b) {
        floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int z = 0; z < NW; ++z) {
            const floatx4 v = red[(b * NW + z) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += v[e];
        }
        return s;
    };
    auto finish = [&](int b, const floatx4 &s) {
        const int m = 16 * (b % TB) + i, c = 16 * (b / TB) + 4 * g;
        if (m >= p.M || c >= rows) return;
        const float v[4] = {s[0], s[1], s[2], s[3]};
        with_act(p.act, [&](auto tag) { finish_run<DT, decltype(tag)::value>(p, m, n0 + c, v); });
    };
    if (gr.slices == 1) {
        for (int b = wave; b < RB * TB; b += NW) finish(b, sum_of(b));
        return;
    }
    auto at = [&](int s, int b) {
        return gr.part + ((((long long)s * gr.strips + strip) * (RB * TB) + b) * 64 + lane) * 4;
    };
    for (int b = wave; b < RB * TB; b += NW) store_partial(at(slice, b), sum_of(b));
    __syncthreads();   // red is read: its first word takes the flag
    if (!arrive_last(gr.count + strip, gr.slices, reinterpret_cast<int *>(smem))) return;
    for (int b = wave; b < RB * TB; b += NW)
        finish(b, sum_slices(gr.slices, [&](int s) { return at(s, b); }));
    if (tid == 0)
        __hip_atomic_store(gr.count + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#endif
}

// A lane's V x V block of an operand whose own index is contiguous: it loads 16
// bytes of each of V rows of k, which is V columns of V k values: fragments of V
// products, once the block is turned (16-bit types: pairs of rows are
// interleaved, 4 V byte permutes; fp32 needs none, a product step taking one
// row).  Fragment c stands for column V i + c.
template <int DT>
__device__ __forceinline__ uintx4 turned(const uintx4 (&w)[Step<DT>::V], int c) {
    uintx4 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (DT == SGEMM_DTYPE_F32)
            f[q] = w[q][c];
        else   // halves c % 2 of dword c / 2 of rows 2q and 2q + 1
            f[q] = __builtin_amdgcn_perm(w[2 * q + 1][c / 2], w[2 * q][c / 2],
                                         (c & 1) ? 0x07060302u : 0x05040100u);
    }
    return f;
}

// v without its first d values (d < V), zeros behind the rest: what a lane does
// whose columns end inside its 16 bytes, which it loads so that they end with the
// row (37 x 429 x 921 bf16: dX 20 us and dW 11; value by value 33 and 17).
template <int DT>
__device__ __forceinline__ uintx4 without(uintx4 v, int d) {
    const int dwords = DT == SGEMM_DTYPE_F32 ? d : d >> 1;
    const bool one = dwords & 1, two = dwords & 2, half = DT != SGEMM_DTYPE_F32 && (d & 1);
    unsigned u[5];
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = one ? (q < 3 ? v[q + 1] : 0u) : v[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = two ? (q < 2 ? u[q + 2] : 0u) : u[q];
    u[4] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        v[q] = half ? __builtin_amdgcn_perm(u[q + 1], u[q], 0x05040302u) : u[q];
    return v;
}

// dX = G W: a strip of 16 V columns of W per workgroup (V values to 16
// bytes), k walking W's rows, turned in registers.  LO: G in two parts.
template <int DT, int TB, bool LO, int NW>
__global__ void __launch_bounds__(64 * NW) cols_kernel(Prod p, RowsGrid gr) {
    using T = typename Type<DT>::T;
    constexpr int V = Step<DT>::V, KS = Step<DT>::K, COLS = 16 * V;
    __shared__ floatx4 red[NW / 2][V * TB][64];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x % gr.strips, slice = blockIdx.x / gr.strips;
    const int n0 = strip * COLS, col = n0 + V * i, cols = p.N - col;
    const T *B = static_cast<const T *>(p.B) + (cols > 0 ? col : 0);
    const int ks = slice * gr.kslice, ke = min(ks + gr.kslice, p.K);

    struct Round {
        uintx4 w[V], x[TB], l[LO ? TB : 1];
    } a, b;
    // 16-byte loads throughout unless the strip ends inside a lane's columns;
    // lanes past the end read the strip's first columns (not stored)
    const bool even = n0 + COLS <= p.N || (p.N % V == 0 && p.N - n0 >= V);
    const T *Bf = static_cast<const T *>(p.B) + (cols >= V ? col : n0);
    // in a strip that does, the lane's load ends with the row at the latest; only
    // rows of fewer than V columns are read value by value
    const bool wide = p.N >= V;
    const int at_end = even ? 0 : min(col, p.N - V), beyond = even ? 0 : min(col - at_end, V - 1);
    const T *Be = even ? Bf : static_cast<const T *>(p.B) + at_end;
    auto load = [&](Round &r, int k) {
        const int kg = k + V * g;
        if (even && k + KS <= ke) {
#pragma unroll
            for (int e = 0; e < V; ++e) r.w[e] = load_whole<DT>(Bf + (long long)(kg + e) * p.ldb);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const long long at = (long long)min(16 * t + i, p.M - 1) * p.lda + kg;
                r.x[t] = load_whole<DT>(static_cast<const T *>(p.A) + at);
                if constexpr (LO) r.l[t] = load_whole<DT>(static_cast<const T *>(p.lo) + at);
            }
            return;
        }
        if (wide) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = kg + e < ke;
                r.w[e] = load_whole<DT>(Be + (long long)(in ? kg + e : ke - 1) * p.ldb, in);
            }
            if (!even)
#pragma unroll
                for (int e = 0; e < V; ++e) r.w[e] = without<DT>(r.w[e], beyond);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                r.w[e] = load_frag<DT>(B + (long long)(kg + e) * p.ldb, kg + e < ke ? cols : 0, Bf);
        }
        if (k + KS <= ke) {
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const long long at = (long long)min(16 * t + i, p.M - 1) * p.lda + kg;
                r.x[t] = load_whole<DT>(static_cast<const T *>(p.A) + at);
                if constexpr (LO) r.l[t] = load_whole<DT>(static_cast<const T *>(p.lo) + at);
            }
            return;
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const long long at = (long long)min(16 * t + i, p.M - 1) * p.lda + kg;
            r.x[t] = load_frag<DT>(static_cast<const T *>(p.A) + at, ke - kg,
                                   static_cast<const T *>(p.A));
            if constexpr (LO)
                r.l[t] = load_frag<DT>(static_cast<const T *>(p.lo) + at, ke - kg,
                                       static_cast<const T *>(p.lo));
        }
    };
    floatx4 acc[V][TB];
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[c][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto products = [&](const Round &r) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const uintx4 f = turned<DT>(r.w, c);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                acc[c][t] = mfma_step<DT>(f, r.x[t], acc[c][t]);
                if constexpr (LO) acc[c][t] = mfma_step<DT>(f, r.l[t], acc[c][t]);
            }
        }
    };
    // the waves take the steps of the slice in turn
    constexpr int ST = NW * KS;
    const int k0 = ks + wave * KS;
    if (k0 < ke) {
        load(a, k0);
        for (int k = k0; k < ke; k += 2 * ST) {
            if (k + ST < ke) load(b, k + ST);
            pipeline_fence();
            products(a);
            pipeline_fence();
            if (k + ST >= ke) break;
            if (k + 2 * ST < ke) load(a, k + 2 * ST);
            pipeline_fence();
            products(b);
            pipeline_fence();
        }
    }
    // the upper half of the waves hand their sums to the lower, down to the
    // first wave, which leaves the workgroup's in red[0]
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int j = 0; j < V * TB; ++j) red[wave - half][j][lane] = acc[j / TB][j % TB];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int j = 0; j < V * TB; ++j) {
                const floatx4 v = red[wave][j][lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j / TB][j % TB][e] += v[e];
            }
    }
    if (wave == 0)
#pragma unroll
        for (int j = 0; j < V * TB; ++j) red[0][j][lane] = acc[j / TB][j % TB];
    __syncthreads();
    if (gr.slices > 1) {
        // every wave takes a share of the accumulators, eight slices' loads in
        // flight at a time
        auto at = [&](int s, int j) {
            return gr.part + ((((long long)s * gr.strips + strip) * (V * TB) + j) * 64 + lane) * 4;
        };
        for (int j = wave; j < V * TB; j += NW) store_partial(at(slice, j), red[0][j][lane]);
        if (!arrive_last(gr.count + strip, gr.slices, &last)) return;
        for (int j = wave; j < V * TB; j += NW) red[0][j][lane] = sum_slices(gr.slices, [&](int s) { return at(s, j); });
        if (tid == 0)
            __hip_atomic_store(gr.count + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
    }
    // result element r of row block t: V adjacent columns of row 16 t + i
    for (int u = wave; u < 4 * TB; u += NW) {
        const int t = u >> 2, r = u & 3, m = 16 * t + i;
        float v[V];
#pragma unroll
        for (int c = 0; c < V; ++c)
            v[c] = reinterpret_cast<const float *>(&red[0][c * TB + t][lane])[r];
        if (m < p.M) finish_run<DT, SGEMM_ACT_NONE>(p, m, n0 + V * (4 * g + r), v);
    }
}

// dW = G^T X with at most 64 rows of G and X (LO: G in two parts): bound by
// writing dW.  A wave computes 16 V x 16 V of it from S steps of k, and each lane
// stores 16 bytes of a row at a time: no ring and no barriers.  With few blocks
// the four waves of a workgroup share one, each taking some of its columns of G
// (SPLIT 4: 16 rows, 1024 x 1024 14 -> 9 us; with many, the repeated loads cost
// more: 16 rows, 14336 x 4096 49 -> 57 us).  X is turned in
// registers; G waits in LDS, from where a lane takes one column of its block at
// a time (so the walk over the columns is a loop).  Product (c, c') of the wave is rows V i + c of dW (lane i)
// and columns V (4r + g) + c' (result element r).
template <int DT, int S, bool LO, int SPLIT>
__global__ void __launch_bounds__(kThreads) outer_kernel(Prod p, int blocks_n) {
    using T = typename Type<DT>::T;
    constexpr int V = Step<DT>::V, KS = Step<DT>::K, B = 16 * V, PARTS = LO ? 2 : 1;
    __shared__ uintx4 held[kWaves][PARTS][S][V][64];
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    static_assert(V % SPLIT == 0 && (SPLIT == 1 || SPLIT == kWaves), "whole columns");
    const int block = SPLIT == 1 ? blockIdx.x * kWaves + wave : blockIdx.x;
    const int m0 = block / blocks_n * B, n0 = block % blocks_n * B;
    if (m0 >= p.M) return;
    // (X's lanes are dealt so that the four lanes that store one row side by
    // side store 64 bytes in a row)
    const int am = m0 + V * i, bn = n0 + V * (4 * (i & 3) + (i >> 2));
    // 16-byte loads throughout: where the block ends inside a lane's values they
    // end with the row and are moved; lanes past an end read values that are not
    // stored, rows past K the last one (zeroed)
    auto even = [&](int at0, int n) { return at0 + B <= n || (n % V == 0 && n - at0 >= V); };
    const bool fast_m = even(m0, p.M), fast_n = even(n0, p.N);
    // K == 0: no row to read; fewer than V values: value by value
    const bool fast = p.K > 0 && p.M >= V && p.N >= V;
    const int amf = fast_m ? (am + V <= p.M ? am : m0) : min(am, p.M - V);
    const int bnf = fast_n ? (bn + V <= p.N ? bn : n0) : min(bn, p.N - V);
    const int beyond_m = fast_m ? 0 : min(am - amf, V - 1);
    const int beyond_n = fast_n ? 0 : min(bn - bnf, V - 1);
    uintx4 fb[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        uintx4 a[PARTS][V], b[V];
        if (fast) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int k = s * KS + V * g + e;
                const bool in = k < p.K;
                const long long kc = in ? k : p.K - 1;
                b[e] = load_whole<DT>(static_cast<const T *>(p.B) + kc * p.ldb + bnf, in);
                a[0][e] = load_whole<DT>(static_cast<const T *>(p.A) + kc * p.lda + amf, in);
                if constexpr (LO)
                    a[1][e] = load_whole<DT>(static_cast<const T *>(p.lo) + kc * p.lda + amf, in);
            }
            if (!fast_n)
#pragma unroll
                for (int e = 0; e < V; ++e) b[e] = without<DT>(b[e], beyond_n);
            if (!fast_m)
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) a[q][e] = without<DT>(a[q][e], beyond_m);
        } else if (p.K == 0) {   // no row to read: dW is zero
#pragma unroll
            for (int e = 0; e < V; ++e) {
                b[e] = uintx4{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < PARTS; ++q) a[q][e] = uintx4{0, 0, 0, 0};
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int k = s * KS + V * g + e;
                const bool in = k < p.K;
                const long long at = (long long)k * p.lda + am;
                b[e] = load_frag<DT>(static_cast<const T *>(p.B) + (long long)k * p.ldb + bn,
                                     in ? p.N - bn : 0, static_cast<const T *>(p.B));
                a[0][e] = load_frag<DT>(static_cast<const T *>(p.A) + at, in ? p.M - am : 0,
                                        static_cast<const T *>(p.A));
                if constexpr (LO)
                    a[1][e] = load_frag<DT>(static_cast<const T *>(p.lo) + at, in ? p.M - am : 0,
                                            static_cast<const T *>(p.lo));
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) held[wave][q][s][e][lane] = a[q][e];
#pragma unroll
        for (int c = 0; c < V; ++c) fb[s][c] = turned<DT>(b, c);
    }
    const int rows = min(V, p.M - am);   // rows of this lane inside dW
#pragma unroll 1
    for (int q = 0; q < V / SPLIT; ++q) {
        const int c = SPLIT == 1 ? q : wave * (V / SPLIT) + q;
        floatx4 acc[V];
#pragma unroll
        for (int d = 0; d < V; ++d) acc[d] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                T col[V];   // column c of this lane's block (a lane reads its own values)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    col[e] = reinterpret_cast<const T *>(&held[wave][q][s][e][lane])[c];
                uintx4 fa;
                __builtin_memcpy(&fa, col, 16);
#pragma unroll
                for (int d = 0; d < V; ++d) acc[d] = mfma_step<DT>(fb[s][d], fa, acc[d]);
            }
        if (c >= rows) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v[V];
#pragma unroll
            for (int d = 0; d < V; ++d) v[d] = acc[d][r];
            finish_run<DT, SGEMM_ACT_NONE>(p, am + c, n0 + V * (4 * r + g), v);
        }
    }
}

struct PlanRows {
    int strips, slices, kslice, width, tb, rb, acc;
    bool staged;
};

constexpr int kCUs = 256;

PlanRows plan_rows(int dtype, const Prod &p) {
    const int elem = dtype == SGEMM_DTYPE_F32 ? 4 : 2, v = 16 / elem, step = 4 * v;
    PlanRows q{};
    q.tb = p.M > 32 ? 4 : p.M > 16 ? 2 : 1;
    q.staged = !p.b_mc && stage_ok(p.B, p.ldb, p.K, elem) && stage_ok(p.A, p.lda, p.K, elem);
    int s = 1, unit = step;
    if (q.staged) {
        // one strip per CU where N reaches for it: as wide as it has to be, up
        // to 64 columns (then several strips per CU)
        const int rounds = (p.N + 64 * kCUs - 1) / (64 * kCUs);
        q.width = ((p.N + rounds * kCUs - 1) / (rounds * kCUs) + 3) / 4 * 4;
        // (and at least as wide as there are rows: every strip reads all rows of X;
        // 64 x 4096 x 4096 bf16 22 us with 16 columns, 16 with 64 and k split)
        if (q.width < 16 * q.tb) q.width = 16 * q.tb;
        q.rb = q.width > 32 ? 4 : q.width > 16 ? 2 : 1;
        q.acc = q.rb * q.tb;
        q.strips = (p.N + q.width - 1) / q.width;
        unit = 512 / q.rb / elem;
        // a slice keeps one stage for every wave
        if (q.strips <= kCUs / 2) {
            s = kCUs / q.strips;
            const int most = p.K / (8 * unit);
            if (s > most) s = most;
        }
    } else {
        q.width = p.b_mc ? 16 * v : 16;
        q.acc = (p.b_mc ? v : 1) * q.tb;   // 16-byte accumulators per lane of a strip
        q.strips = (p.N + q.width - 1) / q.width;
        // split k until two workgroups per CU are in flight, each wave keeping
        // four steps at least (with one, 64 x 2048 x 512 dX 18 -> 24 us: the join)
        if (q.strips < kCUs && q.strips <= kWorkspaceCounters) {
            s = (2 * kCUs + q.strips - 1) / q.strips;
            const int most = p.K / (kWaves * 4 * step);   // (or two for each of eight waves)
            if (s > most) s = most;
            if (s > 64) s = 64;
        }
    }
    if (s < 1) s = 1;
    q.kslice = ((p.K + s - 1) / s + unit - 1) / unit * unit;
    if (q.kslice < unit) q.kslice = unit;
    q.slices = (p.K + q.kslice - 1) / q.kslice;
    if (q.slices < 1) q.slices = 1;
    return q;
}

template <int DT, int TB>
hipError_t launch_tb(const Prod &p, const PlanRows &q, const RowsGrid &gr, hipStream_t stream) {
    constexpr int CW = TB == 1 ? 8 : 4;   // the sums of eight waves fit LDS for one block of rows
    const dim3 grid((unsigned)gr.strips * gr.slices), block(kThreads);
    if (q.staged && q.rb == 1)
        hipLaunchKernelGGL((rows_staged_kernel<DT, 1, TB>), grid, dim3(512), 0, stream, p, gr);
    else if (q.staged && q.rb == 2)
        hipLaunchKernelGGL((rows_staged_kernel<DT, 2, TB>), grid, dim3(512), 0, stream, p, gr);
    else if (q.staged)
        hipLaunchKernelGGL((rows_staged_kernel<DT, 4, TB>), grid, dim3(512), 0, stream, p, gr);
    else if (!p.b_mc)
        hipLaunchKernelGGL((rows_kernel<DT, TB, TB == 1 ? 8 : 4>), grid, block, 0, stream, p, gr);
    else if (DT != SGEMM_DTYPE_F32 && p.lo)
        hipLaunchKernelGGL((cols_kernel<DT, TB, DT != SGEMM_DTYPE_F32, CW>), grid, dim3(64 * CW), 0,
                           stream, p, gr);
    else
        hipLaunchKernelGGL((cols_kernel<DT, TB, false, CW>), grid, dim3(64 * CW), 0, stream, p, gr);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(Prod p, const Workspace &ws, hipStream_t stream) {
    const PlanRows q = plan_rows(DT, p);
    const RowsGrid gr{q.strips, q.slices, q.kslice, q.width, static_cast<float *>(ws.ptr),
                      ws.counters};
    switch (q.tb) {
    case 1: return launch_tb<DT, 1>(p, q, gr, stream);
    case 2: return launch_tb<DT, 2>(p, q, gr, stream);
    default: return launch_tb<DT, 4>(p, q, gr, stream);
    }
}

template <int DT, int S, int SPLIT>
hipError_t launch_steps(const Prod &p, long long blocks, int bn, hipStream_t stream) {
    const dim3 grid((unsigned)(SPLIT == 1 ? (blocks + kWaves - 1) / kWaves : blocks));
    if (DT != SGEMM_DTYPE_F32 && p.lo)
        hipLaunchKernelGGL((outer_kernel<DT, S, DT != SGEMM_DTYPE_F32, SPLIT>), grid, dim3(kThreads),
                           0, stream, p, bn);
    else
        hipLaunchKernelGGL((outer_kernel<DT, S, false, SPLIT>), grid, dim3(kThreads), 0, stream, p, bn);
    return hipGetLastError();
}

template <int DT, int S>
hipError_t launch_split(const Prod &p, hipStream_t stream) {
    constexpr int B = 16 * Step<DT>::V;
    const int bn = (p.N + B - 1) / B;
    const long long blocks = (long long)((p.M + B - 1) / B) * bn;
    return blocks <= 2 * kCUs ? launch_steps<DT, S, kWaves>(p, blocks, bn, stream)
                              : launch_steps<DT, S, 1>(p, blocks, bn, stream);
}

template <int DT>
hipError_t launch_outer_dt(Prod p, hipStream_t stream) {
    constexpr int KS = Step<DT>::K;
    if (p.K <= KS) return launch_split<DT, 1>(p, stream);
    if (DT != SGEMM_DTYPE_F32 || p.K <= 2 * KS) return launch_split<DT, 2>(p, stream);
    return launch_split<DT, DT == SGEMM_DTYPE_F32 ? 4 : 2>(p, stream);
}

}  // namespace

hipError_t launch_outer(int dtype, const Prod &p, hipStream_t stream) {
    switch (dtype) {
    case SGEMM_DTYPE_BF16: return launch_outer_dt<SGEMM_DTYPE_BF16>(p, stream);
    case SGEMM_DTYPE_F16: return launch_outer_dt<SGEMM_DTYPE_F16>(p, stream);
    default: return launch_outer_dt<SGEMM_DTYPE_F32>(p, stream);
    }
}

size_t rows_workspace(int dtype, const Prod &p) {
    const PlanRows q = plan_rows(dtype, p);
    return q.slices == 1 ? 0 : (size_t)q.slices * q.strips * q.acc * 64 * 16;
}

hipError_t launch_rows(int dtype, const Prod &p, const Workspace &ws, hipStream_t stream) {
    switch (dtype) {
    case SGEMM_DTYPE_BF16: return launch_dt<SGEMM_DTYPE_BF16>(p, ws, stream);
    case SGEMM_DTYPE_F16: return launch_dt<SGEMM_DTYPE_F16>(p, ws, stream);
    default: return launch_dt<SGEMM_DTYPE_F32>(p, ws, stream);
    }
}

}  // namespace sg
