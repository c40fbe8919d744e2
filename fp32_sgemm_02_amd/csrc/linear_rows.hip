// linear_rows.hip -- products of a linear layer with at most 64 rows, the
// shapes of decoding and of small batches' gradients:
//     rows_kernel   Y = act(X W^T + b) + R   W's rows run along k
//     cols_kernel   dX = G W                 k runs over W's rows
// Both are bound by reading W once: at M = 16 a weight value of two bytes is
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
        if (t < TB) {
            sum = floatx4{0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < gr.slices; s += 8) {
                floatx4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = s + q < gr.slices ? load_partial(at(s + q)) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (s + q < gr.slices)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[e] += v[q][e];
            }
        }
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
    for (int b = wave; b < RB * TB; b += NW) {
        floatx4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < gr.slices; s += 8) {
            floatx4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = s + q < gr.slices ? load_partial(at(s + q, b)) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (s + q < gr.slices)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] += v[q][e];
        }
        finish(b, sum);
    }
    if (tid == 0)
        __hip_atomic_store(gr.count + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#endif
}

// dX = G W: a strip of 16 V columns of W per workgroup (V values to 16
// bytes), k walking W's rows.  A lane loads 16 bytes of each of V rows, which
// is V columns of V k values: the fragments of V products, once the V x V
// block is turned (16-bit types: pairs of rows are interleaved, 4 V byte
// permutes per step; fp32 needs none, a product step taking one row).
// Product c of the block stands for column V i + c of the strip.  LO: G in two
// parts.
template <int DT, int TB, bool LO>
__global__ void __launch_bounds__(kThreads) cols_kernel(Prod p, RowsGrid gr) {
    using T = typename Type<DT>::T;
    constexpr int V = Step<DT>::V, KS = Step<DT>::K, COLS = 16 * V;
    __shared__ floatx4 red[2][V][TB][64];
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
    auto load = [&](Round &r, int k) {
        const int kg = k + V * g;
#pragma unroll
        for (int e = 0; e < V; ++e)
            r.w[e] = load_frag<DT>(B + (long long)(kg + e) * p.ldb, kg + e < ke ? cols : 0);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const long long at = (long long)min(16 * t + i, p.M - 1) * p.lda + kg;
            r.x[t] = load_frag<DT>(static_cast<const T *>(p.A) + at, ke - kg);
            if constexpr (LO) r.l[t] = load_frag<DT>(static_cast<const T *>(p.lo) + at, ke - kg);
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
            uintx4 f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (DT == SGEMM_DTYPE_F32)
                    f[q] = r.w[q][c];
                else   // halves c % 2 of dword c / 2 of rows 2q and 2q + 1
                    f[q] = __builtin_amdgcn_perm(r.w[2 * q + 1][c / 2], r.w[2 * q][c / 2],
                                                 (c & 1) ? 0x07060302u : 0x05040100u);
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                acc[c][t] = mfma_step<DT>(f, r.x[t], acc[c][t]);
                if constexpr (LO) acc[c][t] = mfma_step<DT>(f, r.l[t], acc[c][t]);
            }
        }
    };
    // the waves take the steps of the slice in turn
    constexpr int ST = kWaves * KS;
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
    // waves 2 and 3 hand their sums to 0 and 1, then 1 to 0: a fixed order
#pragma unroll
    for (int half = 2; half >= 1; half /= 2) {
        __syncthreads();
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int t = 0; t < TB; ++t) red[wave - half][c][t][lane] = acc[c][t];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int c = 0; c < V; ++c)
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[c][t][e] += red[wave][c][t][lane][e];
    }
    if (gr.slices > 1) {
        auto at = [&](int s, int j) {
            return gr.part + ((((long long)s * gr.strips + strip) * (V * TB) + j) * 64 + lane) * 4;
        };
        if (wave == 0)
#pragma unroll
            for (int j = 0; j < V * TB; ++j) store_partial(at(slice, j), acc[j / TB][j % TB]);
        if (!arrive_last(gr.count + strip, gr.slices, &last)) return;
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < V * TB; ++j) acc[j / TB][j % TB] = load_partial(at(0, j));
            for (int s = 1; s < gr.slices; ++s)
#pragma unroll
                for (int j = 0; j < V * TB; ++j) {
                    const floatx4 v = load_partial(at(s, j));
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j / TB][j % TB][e] += v[e];
                }
        }
        if (tid == 0)
            __hip_atomic_store(gr.count + strip, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (wave != 0) return;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int m = 16 * t + i;
        if (m >= p.M) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v[V];
#pragma unroll
            for (int c = 0; c < V; ++c) v[c] = acc[c][t][r];
            finish_run<DT, SGEMM_ACT_NONE>(p, m, n0 + V * (4 * g + r), v);
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
        if (q.width < 16) q.width = 16;
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
        // four steps at least
        if (q.strips < kCUs && q.strips <= kWorkspaceCounters) {
            s = (2 * kCUs + q.strips - 1) / q.strips;
            const int most = p.K / (kWaves * 4 * step);
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
        hipLaunchKernelGGL((cols_kernel<DT, TB, DT != SGEMM_DTYPE_F32>), grid, block, 0, stream, p,
                           gr);
    else
        hipLaunchKernelGGL((cols_kernel<DT, TB, false>), grid, block, 0, stream, p, gr);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(Prod p, const Workspace &ws, hipStream_t stream) {
    const PlanRows q = plan_rows(DT, p);
    p.cvec = epilogue_vec(p, (int)sizeof(typename Type<DT>::T));
    const RowsGrid gr{q.strips, q.slices, q.kslice, q.width, static_cast<float *>(ws.ptr),
                      ws.counters};
    switch (q.tb) {
    case 1: return launch_tb<DT, 1>(p, q, gr, stream);
    case 2: return launch_tb<DT, 2>(p, q, gr, stream);
    default: return launch_tb<DT, 4>(p, q, gr, stream);
    }
}

}  // namespace

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
