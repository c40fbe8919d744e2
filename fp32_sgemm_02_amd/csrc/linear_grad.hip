// linear_grad.hip -- the elementwise half of a linear layer's backward pass:
//     G = dY * act'(Z),   db = column sums of G,
// and the last step of an fp32 linear layer, Y = act(Z) + R.
//
// Memory-bound: dY and Z are read once and G written once, 16 bytes per lane
// where the rows allow it, and the column sums are taken from the fp32 values
// on the way.  A workgroup owns a block of columns (16 lanes of 16 bytes) and
// a band of rows (16 row lanes); the bands' partial sums go to memory as
// device-coherent stores and the workgroup of a column block that counts last
// adds them in band order.
#include "linear_internal.hpp"

namespace sg {
namespace {

constexpr int kF32 = SGEMM_DTYPE_F32;
constexpr int kColLanes = 16, kRowLanes = 16;   // lanes of a workgroup

struct GradArgs {
    int M, N;
    const void *dY, *Z;
    void *G, *lo, *db;
    long long lddy, ldz, ldg;
    int band;       // rows per band
    int bands;
    float *part;    // bands x N
    unsigned *count;
};

template <int DT, int ACT>
__global__ void __launch_bounds__(256) grad_kernel(GradArgs a) {
    using Ty = Type<DT>;
    using T = typename Ty::T;
    constexpr int V = Ty::V, COLS = kColLanes * V;
    __shared__ float red[kRowLanes][COLS];
    __shared__ int last;
    const int tid = threadIdx.x, cl = tid % kColLanes, rl = tid / kColLanes;
    const int n0 = blockIdx.x * COLS, n = n0 + cl * V;
    const int r0 = blockIdx.y * a.band, r1 = min(r0 + a.band, a.M);
    const int cols = min(V, a.N - n);
    float sum[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    if (cols > 0) {
        // 16 bytes at a time (from any address; those of G are aligned) unless N
        // ends inside a lane's; the same for the whole block, so that the loads of
        // several rows run together
        const bool vec = n0 + COLS <= a.N || a.N % V == 0;
#pragma unroll 2
        for (int r = r0 + rl; r < r1; r += kRowLanes) {
            const T *dy = static_cast<const T *>(a.dY) + (long long)r * a.lddy + n;
            const T *z = static_cast<const T *>(a.Z) + (long long)r * a.ldz + n;
            T *g = a.G ? static_cast<T *>(a.G) + (long long)r * a.ldg + n : nullptr;
            T *lo = a.lo ? static_cast<T *>(a.lo) + (long long)r * a.ldg + n : nullptr;
            T y[V], x[V], o[V], l[V];
            if (vec) {
                __builtin_memcpy(y, dy, 16);
                if (ACT != SGEMM_ACT_NONE)
                    __builtin_memcpy(x, z, 16);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    y[e] = e < cols ? dy[e] : T(0);
                    if (ACT != SGEMM_ACT_NONE) x[e] = e < cols ? z[e] : T(0);
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = Ty::load(y[e]);
                if (ACT != SGEMM_ACT_NONE) v *= slope_for<DT, ACT>(Ty::load(x[e]));
                sum[e] += v;
                o[e] = Ty::store(v);
                // what the rounding of G left over; 0 where G overflowed
                const float d = v - Ty::load(o[e]);
                l[e] = Ty::store(fabsf(d) < INFINITY ? d : 0.f);
            }
            if (g) {   // past N: zeros, up to the end of the 16 bytes
                __builtin_memcpy(__builtin_assume_aligned(g, 16), o, 16);
                if (lo) __builtin_memcpy(__builtin_assume_aligned(lo, 16), l, 16);
            }
        }
    }
    if (!a.db) return;
#pragma unroll
    for (int e = 0; e < V; ++e) red[rl][cl * V + e] = sum[e];
    __syncthreads();
    T *db = static_cast<T *>(a.db);
    for (int c = tid; c < COLS && n0 + c < a.N; c += 256) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRowLanes; ++r) s += red[r][c];
        if (a.bands == 1)
            db[n0 + c] = Ty::store(s);
        else
            __hip_atomic_store(a.part + (long long)blockIdx.y * a.N + n0 + c, s, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (a.bands == 1) return;
    __builtin_amdgcn_s_waitcnt(0);   // this wave's partial sums are in memory
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(a.count + blockIdx.x, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(a.bands - 1);
    __syncthreads();
    if (!last) return;
    for (int c = tid; c < COLS && n0 + c < a.N; c += 256) {
        const float *src = a.part + n0 + c;
        float s = 0.f;
        for (int z = 0; z < a.bands; z += 16) {
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; ++x)
                v[x] = z + x < a.bands ? __hip_atomic_load(src + (long long)(z + x) * a.N,
                                                           __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT)
                                       : 0.f;
#pragma unroll
            for (int x = 0; x < 16; ++x)
                if (z + x < a.bands) s += v[x];
        }
        db[n0 + c] = Ty::store(s);
    }
    if (tid == 0)
        __hip_atomic_store(a.count + blockIdx.x, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ void __launch_bounds__(256) finish32_kernel(int M, int N, const float *Z, long long ldz,
                                                       int act, const float *R, long long ldr,
                                                       float *Y, long long ldy) {
    for (int i = blockIdx.y; i < M; i += gridDim.y) {
        const float *z = Z + (long long)i * ldz, *r = R ? R + (long long)i * ldr : nullptr;
        float *y = Y + (long long)i * ldy;
        for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < N; j += gridDim.x * blockDim.x) {
            const float v = activate(act, z[j]);
            y[j] = r ? v + r[j] : v;
        }
    }
}

__global__ void __launch_bounds__(256) sum32_kernel(int M, int N, const float *parts, long long ldp,
                                                    long long step, int count, float *C,
                                                    long long ldc) {
    for (int i = blockIdx.y; i < M; i += gridDim.y)
        for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < N; j += gridDim.x * blockDim.x) {
            const float *p = parts + (long long)i * ldp + j;
            float s = 0.f;
            for (int q = 0; q < count; ++q) s += p[q * step];
            C[(long long)i * ldc + j] = s;
        }
}

struct Bands {
    int blocks, band, bands;
};

Bands bands_of(int dtype, int M, int N) {
    const int cols = kColLanes * (dtype == kF32 ? 4 : 8);
    Bands b;
    b.blocks = (N + cols - 1) / cols;
    // at most 32 bands, whose sums the last workgroup of a column block adds up
    // with two round trips to memory; one band where the column blocks
    // outnumber the arrival counters
    b.band = ((M + 31) / 32 + kRowLanes - 1) / kRowLanes * kRowLanes;
    if (b.blocks > kWorkspaceCounters) b.band = M;
    if (b.band < 1) b.band = 1;
    b.bands = M > 0 ? (M + b.band - 1) / b.band : 1;
    return b;
}

template <int DT>
hipError_t launch_dt(const GradArgs &a, int act, int blocks, hipStream_t stream) {
    const dim3 grid(blocks, a.bands), block(256);
    switch (act) {
    case SGEMM_ACT_RELU:
        hipLaunchKernelGGL((grad_kernel<DT, SGEMM_ACT_RELU>), grid, block, 0, stream, a);
        break;
    case SGEMM_ACT_SILU:
        hipLaunchKernelGGL((grad_kernel<DT, SGEMM_ACT_SILU>), grid, block, 0, stream, a);
        break;
    case SGEMM_ACT_GELU_ERF:
        hipLaunchKernelGGL((grad_kernel<DT, SGEMM_ACT_GELU_ERF>), grid, block, 0, stream, a);
        break;
    case SGEMM_ACT_GELU_TANH:
        hipLaunchKernelGGL((grad_kernel<DT, SGEMM_ACT_GELU_TANH>), grid, block, 0, stream, a);
        break;
    default:
        hipLaunchKernelGGL((grad_kernel<DT, SGEMM_ACT_NONE>), grid, block, 0, stream, a);
        break;
    }
    return hipGetLastError();
}

}  // namespace

size_t grad_workspace(int dtype, int M, int N) {
    const Bands b = bands_of(dtype, M, N);
    return b.bands == 1 ? 0 : (size_t)b.bands * N * sizeof(float);
}

hipError_t launch_grad(int dtype, int M, int N, const void *dY, long long lddy, const void *Z,
                       long long ldz, int act, void *G, void *lo, long long ldg, void *db,
                       float *part, unsigned *count, hipStream_t stream) {
    const Bands b = bands_of(dtype, M, N);
    const GradArgs a{M, N, dY, Z, G, lo, db, lddy, ldz, ldg, b.band, b.bands, part, count};
    switch (dtype) {
    case SGEMM_DTYPE_BF16: return launch_dt<SGEMM_DTYPE_BF16>(a, act, b.blocks, stream);
    case SGEMM_DTYPE_F16: return launch_dt<SGEMM_DTYPE_F16>(a, act, b.blocks, stream);
    default: return launch_dt<kF32>(a, act, b.blocks, stream);
    }
}

hipError_t launch_sum32(int M, int N, const float *parts, long long ldp, long long step, int count,
                        float *C, long long ldc, hipStream_t stream) {
    const int bx = (N + 255) / 256 < 64 ? (N + 255) / 256 : 64, by = M < 65535 ? M : 65535;
    hipLaunchKernelGGL(sum32_kernel, dim3(bx, by), dim3(256), 0, stream, M, N, parts, ldp, step, count,
                       C, ldc);
    return hipGetLastError();
}

hipError_t launch_finish32(int M, int N, const float *Z, long long ldz, int act, const float *R,
                           long long ldr, float *Y, long long ldy, hipStream_t stream) {
    const int bx = (N + 255) / 256 < 64 ? (N + 255) / 256 : 64, by = M < 65535 ? M : 65535;
    hipLaunchKernelGGL(finish32_kernel, dim3(bx, by), dim3(256), 0, stream, M, N, Z, ldz, act, R,
                       ldr, Y, ldy);
    return hipGetLastError();
}

}  // namespace sg
