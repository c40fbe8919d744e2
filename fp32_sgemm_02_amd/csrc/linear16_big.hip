// linear16_big.hip -- the tile kernel of large 16-bit products: 256 x 256 of C
// per workgroup of 8 waves, the waves of a SIMD taking turns between the
// matrix cores and the memory pipelines.
//
// Operands, images, row order and epilogue as in linear16.hip (k-contiguous
// operands as swizzled rows, the others read transposed); what differs is the
// schedule.  A wave owns 128 x 64 of C (64 rows of
// each half of the tile's, 32 columns of each half).  One stage (64 of k) of it is four
// phases of 16 MFMAs, a quadrant each: with the halves A0, A1 of its rows and
// B0, B1 of its columns,
//     phase 0: A0 B0    1: A0 B1    2: A1 B1    3: A1 B0
// A phase is a load section (the LDS reads of the one half the phase lacks,
// two direct loads for a later stage, waits, barrier) and a compute section
// (16 MFMAs, barrier).  Waves 4-7 run one barrier behind waves 0-3, and waves
// w and w + 4 share a SIMD: while one computes, the other loads, so the matrix
// cores always have a wave to serve and no wave waits for a stage as a whole.
//
// A half is read from LDS in one phase (B0 for the next stage in phase 3, where
// nothing else is needed) and its place is refilled, with the stage after
// next, in the phase after: seven phases pass before those values are read.
// At the end of a load section a wave has waited for its own LDS reads (so the
// refill may start) and for all but its last 12 direct loads (so the half that
// the next phase reads is complete once the barrier is passed).  Stages past
// the end are loaded as zeros, which touch no memory and keep the counts.
#include "linear_internal.hpp"

namespace sg {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBK = 64, kTile = 256;
constexpr int kHalf = kTile / 2 * kBK * 2;          // bytes of one half of an operand's stage
constexpr int kStage = 4 * kHalf;                   // A0 A1 B0 B1
constexpr int kOutOfRange = (int)0x80000000u;

// One operand.  Its halves are rows 0 .. 127 and 128 .. 255 of the tile; of
// each, a wave tile takes 64 rows (IS_A, two wave tiles) or 32 (four).  An
// image half holds its rows (k-contiguous) or, own index
// contiguous, 64 rows of k of 16 chunks of 8 tile rows (256 bytes, which are
// contiguous in memory too).
template <int MC, bool IS_A>
struct Half {
    int off[2][2], kk[2];
    const u16 *base;
    long long ld;

    // see mc_swz in linear16.hip
    static __device__ __forceinline__ int swz(int k) { return 2 * ((k & 3) | ((k >> 1) & 4)); }

    __device__ __forceinline__ void init(const u16 *P, long long ld_, int row0, int rows, int wave,
                                         int lane) {
        ld = ld_;
        const int lim = rows - row0;
        base = MC ? P + row0 : P + (long long)row0 * ld;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int q = (j * 8 + wave) * 64 + lane;   // chunk of the half
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (MC) {
                    const int k = q >> 4, row = 128 * h + 8 * ((q & 15) ^ swz(k));
                    kk[j] = k;
                    off[h][j] = row >= lim ? kOutOfRange : (k * (int)ld + row) * 2;
                } else {
                    const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7), row = 128 * h + r;
                    kk[j] = 8 * c;
                    off[h][j] = row >= lim ? kOutOfRange : (row * (int)ld + 8 * c) * 2;
                }
            }
        }
    }
    __device__ __forceinline__ void issue(int h, int t, int krem, unsigned char *img, int wave) const {
        const u16 *src = MC ? base + (long long)t * kBK * ld : base + (long long)t * kBK;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void *)src, (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (lds_void *)(img + (j * 8 + wave) * 1024), 16,
                kk[j] >= krem ? kOutOfRange : off[h][j], 0, 0, 0);
    }
    // Fragments of wave tile w's BLOCKS blocks of a half, both 32-k steps.
    template <int BLOCKS>
    static __device__ __forceinline__ void read(const unsigned char *img, int w, int lane,
                                                uintx4 (&f)[BLOCKS][2]) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (MC) {
            const int k = 8 * g + (i >> 2);   // and k + 4, k + 32, k + 36: the same swizzle
            unsigned at[BLOCKS];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int chunk = 2 * (BLOCKS * w + b) + ((i >> 1) & 1);
                at[b] = lds_address(img) + k * 256 + ((chunk ^ swz(k)) << 4) + ((i & 1) << 3);
            }
            read_transposed<BLOCKS, 2, 1024, 8192>(at, f);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    const int r = 16 * (BLOCKS * w + b) + i;
                    f[b][s] = *reinterpret_cast<const uintx4 *>(
                        img + r * 128 + (((4 * s + g) ^ ((r >> 1) & 7)) << 4));
                }
        }
    }
};

struct GridBig {
    int tiles_m, tiles_n, group_m;
};

template <int DT, int AMC, int BMC>
__global__ void __launch_bounds__(512, 2) prod16_big_kernel(Prod p, GridBig gr) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    using OpA = Half<AMC, true>;
    using OpB = Half<BMC, false>;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * kStage];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // waves w and w + 4 share a SIMD and are on opposite sides of the turn;
    // they hold the two row halves of one column strip
    const int wm = wave >> 2, wn = wave & 3;
    int tm, tn;
    tile_coords(xcd_remap(blockIdx.x, gr.tiles_m * gr.tiles_n), gr.tiles_m, gr.tiles_n, gr.group_m,
                tm, tn);
    const int m0 = tm * kTile, n0 = tn * kTile;
    const int stages = (p.K + kBK - 1) / kBK;

    OpA a;
    OpB b;
    a.init(static_cast<const u16 *>(p.A), p.lda, m0, p.M, wave, lane);
    b.init(static_cast<const u16 *>(p.B), p.ldb, n0, p.N, wave, lane);

    floatx4 acc[4][8];   // [column block][row block]
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[y][x] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto fence = []() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto barrier = [&]() {
        fence();
        __builtin_amdgcn_s_barrier();
        fence();
    };
    // all but the last N direct loads and every LDS access of this wave done
    auto wait = [&](auto n) {
        constexpr int N = decltype(n)::value;
        fence();
        __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
        fence();
    };
    using Twelve = std::integral_constant<int, 12>;
    using Zero = std::integral_constant<int, 0>;
    auto image = [&](int t, int part) { return smem + (t & 1) * kStage + part * kHalf; };
    auto load_a = [&](int h, int t) { a.issue(h, t, p.K - t * kBK, image(t, h), wave); };
    auto load_b = [&](int h, int t) { b.issue(h, t, p.K - t * kBK, image(t, 2 + h), wave); };

    uintx4 fa[4][2], f0[2][2], f1[2][2], g0[2][2];
    auto read_a = [&](int h, int t) { OpA::template read<4>(image(t, h), wm, lane, fa); };
    auto read_b = [&](int h, int t, uintx4 (&f)[2][2]) {
        OpB::template read<2>(image(t, 2 + h), wn, lane, f);
    };
    auto compute = [&](int ha, int hb, const uintx4 (&f)[2][2]) {
        barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    acc[2 * hb + y][4 * ha + x] =
                        mfma16<DT>(f[y][s], fa[x][s], acc[2 * hb + y][4 * ha + x]);
        __builtin_amdgcn_s_setprio(0);
        barrier();
    };
    // stage t with B0 in f; leaves B0 of stage t + 1 in g
    auto stage = [&](int t, const uintx4 (&f)[2][2], uintx4 (&g)[2][2]) {
        load_b(0, t + 2);
        read_a(0, t);
        wait(Twelve{});
        compute(0, 0, f);
        load_a(0, t + 2);
        read_b(1, t, f1);
        wait(Twelve{});
        compute(0, 1, f1);
        load_b(1, t + 2);
        read_a(1, t);
        wait(Twelve{});
        compute(1, 1, f1);
        load_a(1, t + 2);
        read_b(0, t + 1, g);
        wait(Twelve{});
        compute(1, 0, f);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        load_b(0, t);
        load_a(0, t);
        load_b(1, t);
        load_a(1, t);
    }
    wait(Twelve{});
    barrier();   // A0 and B0 of stage 0 are complete
    read_b(0, 0, f0);
    wait(Twelve{});
    barrier();   // and B0 read by every wave
    if (wave >= 4) barrier();
    for (int t = 0; t < stages; t += 2) {
        stage(t, f0, g0);
        if (t + 1 < stages) stage(t + 1, g0, f0);
    }
    if (wave < 4) barrier();
    wait(Zero{});   // no load of a stage past the end is left in flight

    barrier();   // no wave reads the ring any more
    float *box = reinterpret_cast<float *>(smem) + wave * (kStage / 16);   // 16 KB a wave
    each<4>([&](auto c) __attribute__((always_inline)) {
        constexpr int h = c / 2, v = c % 2;   // column half, row half
        finish_wave<DT, 4, 2>(p, m0 + 128 * v + 64 * wm, n0 + 128 * h + 32 * wn, lane, box + v * 2048,
                              [&](auto y, auto x) __attribute__((always_inline)) {
                                  return acc[2 * h + y][4 * v + x];
                              });
    });
#endif
}

template <int DT, int AMC, int BMC>
hipError_t launch(const Prod &p, const GridBig &gr, hipStream_t stream) {
    hipLaunchKernelGGL((prod16_big_kernel<DT, AMC, BMC>), dim3(gr.tiles_m * gr.tiles_n), dim3(512), 0,
                       stream, p, gr);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const Prod &p, hipStream_t stream) {
    const GridBig gr{(p.M + kTile - 1) / kTile, (p.N + kTile - 1) / kTile, 8};
    if (!p.b_mc) return launch<DT, 0, 0>(p, gr, stream);
    if (!p.a_mc) return launch<DT, 0, 1>(p, gr, stream);
    return launch<DT, 1, 1>(p, gr, stream);
}

}  // namespace

hipError_t launch_prod16_big(int dtype, const Prod &p, hipStream_t stream) {
    return dtype == SGEMM_DTYPE_BF16 ? launch_dt<SGEMM_DTYPE_BF16>(p, stream)
                                     : launch_dt<SGEMM_DTYPE_F16>(p, stream);
}

}  // namespace sg
