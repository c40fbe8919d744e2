// linear16.hip -- products of 16-bit operands with a 16-bit result and the
// whole epilogue of a linear layer in the kernel.
//
//     C(m, n) = act(sum_k A(m, k) B(n, k) + bias(n)) + R(m, n)
//
// The three products of a linear layer are this one with different storage:
//     Y  = X W^T    A = X (k contiguous),  B = W (k contiguous)
//     dX = G W      A = G (k contiguous),  B = W read with its own index
//                   contiguous (k walks the rows of W)
//     dW = G^T X    A = G and B = X, both with their own index contiguous
//
// Operand images in LDS.  A stage is 64 values of k.  A k-contiguous operand
// is held as rows of 128 bytes, the eight 16-byte chunks of a row swizzled
// (chunk c of row r in slot c ^ (r >> 1 & 7)), and a lane's MFMA fragment is
// one 16-byte read.  The other kind is held as 64 rows (one per k) of the
// tile's width and read with the transposing LDS read: in a group of 16 lanes,
// lane j fetches four values of row j / 4 and receives, as its four results,
// value i = j of those four rows, so two reads give the 8 k values of a
// fragment.  The chunks of those rows are swizzled by k (mc_swz) so that the
// 32 lanes served at a time touch all banks once.
#include "linear_internal.hpp"

namespace sg {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBK = 64;                            // k per stage
constexpr int kOutOfRange = (int)0x80000000u;      // a buffer offset that reads zero

// Waits for this wave's LDS accesses and for all but its last N vector loads.
template <int N>
__device__ __forceinline__ void wait_loads() {
    pipeline_fence();
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Swizzle of the 16-byte chunks of row k of an own-index-contiguous image of
// BT columns.  32 lanes of a transposing read (two groups of 16) fetch 32
// bytes of each of the rows k, k+1, k+2, k+3 and k+8 .. k+11: the swizzle moves
// these to eight different 32-byte places of the 256 bytes of the banks.
// (Moving only the four rows of one group apart cost as many cycles again:
// SQ_LDS_BANK_CONFLICT 2 per read, 0 with this one.)
template <int BT>
__device__ __forceinline__ int mc_swz(int k) {
    if constexpr (BT >= 128)
        return 2 * ((k & 3) | ((k >> 1) & 4));
    else   // rows of 128 bytes: every other row is 128 bytes apart already
        return 2 * (((k >> 1) & 1) | ((k >> 2) & 2));
}

// One operand's tile: BT rows, stored k-contiguous (MC = 0) or with its own
// index contiguous (MC = 1), loaded by NW waves.
// DIRECT: 16-byte rows throughout, copied to LDS by direct loads (a chunk
// outside the matrix reads as zero: its buffer offset is out of range).
// Otherwise the chunks pass through registers, from any 2-byte alignment
// (the target loads 16 bytes from any address), those that straddle an edge
// value by value.
template <int BT, int MC, bool DIRECT, int NW>
struct Operand {
    static constexpr int BYTES = BT * kBK * 2;
    static constexpr int L = BT * 8 / (64 * NW);   // 16-byte chunks per lane and stage
    static_assert(L * 64 * NW == BT * 8, "chunks divide evenly");

    int off[L];   // DIRECT: byte offset from the stage's origin; else row of the chunk
    int kk[L];    // k of the chunk within the stage
    int cc[L];    // !DIRECT, MC: first tile column of the chunk
    const u16 *base;
    long long ld;
    int lim;   // rows of the tile inside the matrix
    uintx4 reg[DIRECT ? 1 : L];

    __device__ __forceinline__ void init(const u16 *P, long long ld_, int row0, int rows, int wave,
                                         int lane) {
        ld = ld_;
        lim = rows - row0;
        base = MC ? P + row0 : P + (long long)row0 * ld;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int q = (j * NW + wave) * 64 + lane;   // chunk of the image
            if constexpr (MC) {
                const int k = q / (BT / 8), c = (q % (BT / 8)) ^ mc_swz<BT>(k);
                kk[j] = k;
                cc[j] = 8 * c;
                off[j] = 8 * c >= lim ? kOutOfRange : (k * (int)ld + 8 * c) * 2;
            } else {
                const int r = q / 8, c = (q % 8) ^ ((r >> 1) & 7), row = r;
                kk[j] = 8 * c;
                cc[j] = row;
                off[j] = row >= lim ? kOutOfRange : (row * (int)ld + 8 * c) * 2;
            }
        }
    }

    // Copy of stage t into the image (DIRECT) or into registers; krem: k values
    // of the stage inside the matrix.
    __device__ __forceinline__ void issue(int t, int krem, unsigned char *img, int wave) {
        const u16 *src = MC ? base + (long long)t * kBK * ld : base + (long long)t * kBK;
        if constexpr (DIRECT) {
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                (void *)src, (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
            for (int j = 0; j < L; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    r, (lds_void *)(img + (j * NW + wave) * 1024), 16,
                    kk[j] >= krem ? kOutOfRange : off[j], 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int n = MC ? (kk[j] < krem ? lim - cc[j] : 0)
                                 : (cc[j] < lim ? krem - kk[j] : 0);   // values inside
                const u16 *s = MC ? src + (long long)kk[j] * ld + cc[j]
                                  : src + (long long)cc[j] * ld + kk[j];
                uintx4 v = {0, 0, 0, 0};
                if (n >= 8) {
                    __builtin_memcpy(&v, s, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n) v[e / 2] |= (unsigned)s[e] << (16 * (e & 1));
                }
                reg[j] = v;
            }
        }
    }
    __device__ __forceinline__ void commit(unsigned char *img, int wave, int lane) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int j = 0; j < L; ++j)
                *reinterpret_cast<uintx4 *>(img + ((j * NW + wave) * 64 + lane) * 16) = reg[j];
        }
    }

    // Fragments of the BLOCKS 16-row blocks from `blk` on (counted from the
    // tile's first row), 32-k step s.
    template <int BLOCKS>
    static __device__ __forceinline__ void read(const unsigned char *img, int blk, int s, int lane,
                                                uintx4 (&f)[BLOCKS]) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (MC) {
            const int k = 32 * s + 8 * g + (i >> 2);   // and k + 4: the same swizzle
            unsigned at[BLOCKS];
            uintx4 r[BLOCKS][1];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int chunk = 2 * (blk + b) + ((i >> 1) & 1);
                at[b] = lds_address(img) + k * (BT * 2) + ((chunk ^ mc_swz<BT>(k)) << 4) + ((i & 1) << 3);
            }
            read_transposed<BLOCKS, 1, 4 * BT * 2, 0>(at, r);
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) f[b] = r[b][0];
        } else {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int r = 16 * (blk + b) + i;
                f[b] = *reinterpret_cast<const uintx4 *>(img + r * 128 +
                                                         (((4 * s + g) ^ ((r >> 1) & 7)) << 4));
            }
        }
    }
};

// Copies of operands whose rows do not take direct loads, with rows of whole
// 16-byte chunks (the fill is zeros): one launch for both operands, blockIdx.y.
struct Pack {
    const u16 *src[2];
    u16 *dst[2];
    long long ld[2];
    int rows[2], cols[2], chunks[2];   // chunks: 8-value chunks of a row
};

__global__ void __launch_bounds__(256) pack_kernel(Pack p) {
    const int o = blockIdx.y, chunks = p.chunks[o];
    const long long total = (long long)p.rows[o] * chunks;
    for (long long q = blockIdx.x * 256ll + threadIdx.x; q < total; q += gridDim.x * 256ll) {
        const int r = (int)(q / chunks), c = 8 * (int)(q % chunks), n = p.cols[o] - c;
        const u16 *s = p.src[o] + r * p.ld[o] + c;
        uintx4 v = {0, 0, 0, 0};
        if (n >= 8)
            __builtin_memcpy(&v, s, 16);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) v[e / 2] |= (unsigned)s[e] << (16 * (e & 1));
        *reinterpret_cast<uintx4 *>(p.dst[o] + q * 8) = v;
    }
}

struct Grid16 {
    int tiles_m, tiles_n, group_m;
    int slices, per;     // k slices, stages per slice
    float *part;         // slices x tiles x the tile's accumulators
    unsigned *count;     // one arrival counter per tile, zero between launches
};

// Split over k: the workgroup leaves its accumulators in memory and the one
// that counts last adds the slices in order.  Returns whether this workgroup
// finishes the tile (its acc then holds the whole sum).
template <int NB, int MB, int NT>
__device__ __forceinline__ bool join_slices(const Grid16 &gr, int tile, int tiles, int slice,
                                            int tid, int *last, floatx4 (&acc)[NB][MB]) {
    auto at = [&](int s, int j) {
        return gr.part + ((((long long)s * tiles + tile) * (NB * MB) + j) * NT + tid) * 4;
    };
#pragma unroll
    for (int j = 0; j < NB * MB; ++j) store_partial(at(slice, j), acc[j / MB][j % MB]);
    if (!arrive_last(gr.count + tile, gr.slices, last)) return false;
#pragma unroll
    for (int j = 0; j < NB * MB; ++j) acc[j / MB][j % MB] = floatx4{0.f, 0.f, 0.f, 0.f};
    // two slices' loads in flight at a time
    for (int s = 0; s < gr.slices; s += 2) {
        floatx4 v[2][NB * MB];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < NB * MB; ++j)
                v[q][j] = s + q < gr.slices ? load_partial(at(s + q, j)) : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (s + q < gr.slices)
#pragma unroll
                for (int j = 0; j < NB * MB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j / MB][j % MB][e] += v[q][j][e];
    }
    if (tid == 0) __hip_atomic_store(gr.count + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// The tile kernel: BM x BN of C per workgroup, WM x WN per wave, NBUF stages in
// LDS, one barrier per stage.  With direct loads NBUF - 1 stages are in flight
// (those past the end read zeros, which touch no memory and keep the count of
// outstanding loads); operands that pass through registers have two.
// KG: k-groups.  With two, two sets of waves own the same tile and each takes
// one 32-k step of every stage, so that a SIMD has a second wave whose LDS
// reads and loads run under the first one's products; at the end each set
// hands half of its sums to the other through LDS and finishes the other half.
template <int DT, int BM, int BN, int WM, int WN, int NBUF_, int KG, int AMC, int BMC, bool ADIR,
          bool BDIR>
struct Tile16 {
    static constexpr int WAVES_N = BN / WN, WAVES = (BM / WM) * WAVES_N, NW = WAVES * KG, NT = 64 * NW;
    static constexpr int MB = WM / 16, NB = WN / 16;
    using OpA = Operand<BM, AMC, ADIR, NW>;
    using OpB = Operand<BN, BMC, BDIR, NW>;
    static constexpr int NBUF = ADIR && BDIR ? NBUF_ : 2;
    static constexpr int AHEAD = NBUF - 1;   // stages in flight
    static constexpr int STAGE = OpA::BYTES + OpB::BYTES, LDS = NBUF * STAGE;

// Workgroup `block` of the tiles' slices; smem: LDS bytes.
static __device__ __forceinline__ void run(const Prod &p, const Grid16 &gr, int block, int slice,
                                           unsigned char *smem) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wave / WAVES, wm = wave % WAVES / WAVES_N, wn = wave % WAVES_N;
    const int tiles = gr.tiles_m * gr.tiles_n;
    int tm, tn;
    const int tile = xcd_remap(block, tiles);
    tile_coords(tile, gr.tiles_m, gr.tiles_n, gr.group_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int stages = (p.K + kBK - 1) / kBK;
    const int t0 = slice * gr.per, t1 = min(t0 + gr.per, stages);

    OpA a;
    OpB b;
    a.init(static_cast<const u16 *>(p.A), p.lda, m0, p.M, wave, lane);
    b.init(static_cast<const u16 *>(p.B), p.ldb, n0, p.N, wave, lane);

    floatx4 acc[NB][MB];
#pragma unroll
    for (int y = 0; y < NB; ++y)
#pragma unroll
        for (int x = 0; x < MB; ++x) acc[y][x] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto issue = [&](int t, unsigned char *img) {
        // stages past the slice's end read zeros
        const int krem = t >= t1 ? 0 : p.K - t * kBK;
        a.issue(t, krem, img, wave);
        b.issue(t, krem, img + OpA::BYTES, wave);
    };
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) issue(t0 + q, smem + q * STAGE);
    int slot = 0;
    for (int t = t0; t < t1; ++t) {
        unsigned char *cur = smem + slot * STAGE;
        unsigned char *nxt = smem + (slot == 0 ? NBUF - 1 : slot - 1) * STAGE;
        a.commit(cur, wave, lane);
        b.commit(cur + OpA::BYTES, wave, lane);
        wait_loads<(ADIR && BDIR) ? (AHEAD - 1) * (OpA::L + OpB::L) : 0>();
        if constexpr (ADIR && BDIR) {
            // a barrier that leaves the direct loads in flight (the reads of the
            // stage before ended with its products)
            pipeline_fence();
            __builtin_amdgcn_s_barrier();
        } else {
            __syncthreads();
        }
        // stage t is in LDS, and no wave reads buffer nxt
        pipeline_fence();
        issue(t + AHEAD, nxt);
#pragma unroll
        for (int q = 0; q < 2 / KG; ++q) {
            const int s = KG == 2 ? kg : q;
            uintx4 fa[MB], fb[NB];
            OpA::template read<MB>(cur, wm * MB, s, lane, fa);
            OpB::template read<NB>(cur + OpA::BYTES, wn * NB, s, lane, fb);
#pragma unroll
            for (int y = 0; y < NB; ++y)
#pragma unroll
                for (int x = 0; x < MB; ++x) acc[y][x] = mfma16<DT>(fb[y], fa[x], acc[y][x]);
        }
        slot = slot + 1 == NBUF ? 0 : slot + 1;
    }
    wait_loads<0>();   // no load of a stage past the end is left in flight
    // Row blocks [x0, x0 + XB) are this wave's to finish.
    constexpr int XB = MB / KG;
    const int x0 = KG == 2 ? kg * XB : 0;
    floatx4 sum[NB][XB];
    if constexpr (KG == 2) {
        static_assert(NT / 2 * NB * XB * 16 <= LDS / 2, "both halves fit the ring");
        __syncthreads();
        // the other set's blocks, as [set][block][thread of the set]
        floatx4 *box = reinterpret_cast<floatx4 *>(smem);
        const int th = tid % (NT / 2);
        each<NB * XB>([&](auto j) __attribute__((always_inline)) {
            const floatx4 lo = acc[j / XB][j % XB], hi = acc[j / XB][XB + j % XB];
            box[(kg * NB * XB + j) * (NT / 2) + th] = kg ? lo : hi;
            sum[j / XB][j % XB] = kg ? hi : lo;
        });
        __syncthreads();
        each<NB * XB>([&](auto j) __attribute__((always_inline)) {
            const floatx4 v = box[((1 - kg) * NB * XB + j) * (NT / 2) + th];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[j / XB][j % XB][e] += v[e];
        });
    } else {
#pragma unroll
        for (int y = 0; y < NB; ++y)
#pragma unroll
            for (int x = 0; x < XB; ++x) sum[y][x] = acc[y][x];
    }
    // (the flag of the join is in the free ring: with a second LDS object the
    // compiler has the fragment reads wait for every direct load)
    if (gr.slices > 1 &&
        !join_slices<NB, XB, NT>(gr, tile, tiles, slice, tid, reinterpret_cast<int *>(smem), sum))
        return;

    __syncthreads();   // the ring is free
    finish_wave<DT, XB, NB>(p, m0 + wm * WM + 16 * x0, n0 + wn * WN, lane,
                            reinterpret_cast<float *>(smem) + wave * XB * NB * 256,
                            [&](auto y, auto x) __attribute__((always_inline)) { return sum[y][x]; });
}
};

template <int DT, int BM, int BN, int WM, int WN, int NBUF, int KG, int AMC, int BMC, bool ADIR,
          bool BDIR>
__global__ void __launch_bounds__(512)   // at most 256 registers a lane: with more the compiler
                                         // keeps moving the accumulators between register files
prod16_kernel(Prod p, Grid16 gr) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    using Tile = Tile16<DT, BM, BN, WM, WN, NBUF, KG, AMC, BMC, ADIR, BDIR>;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[Tile::LDS];
    Tile::run(p, gr, blockIdx.x, blockIdx.y, smem);
#endif
}

// Both products of a backward pass in one launch, dX's workgroups first: neither
// fills the card by itself, and a launch is saved (515 x 1000 x 776 f16 with SiLU 23.4 -> 17.9 us).  G takes direct
// loads, W and X both do or both do not (DIR).
template <int DT, int BM, int BN, int WM, int WN, int NBUF, int KG, bool DIR>
__global__ void __launch_bounds__(512)
prod16_pair_kernel(Prod x, Grid16 gx, Prod w, Grid16 gw) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass needs the launch stub only
    using X = Tile16<DT, BM, BN, WM, WN, NBUF, KG, 0, 1, true, DIR>;
    using W = Tile16<DT, BM, BN, WM, WN, NBUF, KG, 1, 1, true, DIR>;
    static_assert(X::LDS == W::LDS, "one ring");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[X::LDS];
    const int tiles_x = gx.tiles_m * gx.tiles_n, tiles_w = gw.tiles_m * gw.tiles_n;
    const int b = blockIdx.x, first = tiles_x * gx.slices;
    if (b < first)
        X::run(x, gx, b % tiles_x, b / tiles_x, smem);
    else
        W::run(w, gw, (b - first) % tiles_w, (b - first) / tiles_w, smem);
#endif
}

// ---- host: tile and split --------------------------------------------------

// Whether an operand's rows take direct 16-byte loads: 16-byte rows whose
// stored length is whole chunks, and a tile whose byte offsets fit 31 bits.
bool direct_ok(const void *q, long long ld, int row_len, int bt, int mc) {
    return rows16(q, ld, 2) && row_len % 8 == 0 && (mc ? kBK : bt) * ld * 2 < 0x7fff0000LL;
}

// Whether p's operands are loaded directly by tiles of bt rows.
bool a_direct(const Prod &p, int bt) {
    return direct_ok(p.A, p.lda, p.a_pad ? 0 : p.a_mc ? p.M : p.K, bt, p.a_mc);
}
bool b_direct(const Prod &p, int bt) {
    return direct_ok(p.B, p.ldb, p.b_pad ? 0 : p.b_mc ? p.N : p.K, bt, p.b_mc);
}

struct Plan16 {
    int bm, bn, slices, per;
    bool brief;   // one or two stages: a ring of two, so that more tiles share a CU
    bool big;     // linear16_big.hip
};

constexpr int kCUs = 256;

Plan16 plan16(const Prod &p) {
    auto tiles = [&](int b) { return (long long)((p.M + b - 1) / b) * ((p.N + b - 1) / b); };
    Plan16 q{};
    q.big = tiles(256) >= kCUs / 2 && a_direct(p, 256) && b_direct(p, 256);
    // 128 x 128 where they give more than half the CUs a tile each (6113 x 560 x
    // 4408, 240 tiles: 53 us, 83 with 64 x 64; 2048 x 1536 x 2048, 192 tiles: 23.3 us
    // and 24.7; with 144 tiles both take 14.3; with fewer the split costs more:
    // 2048 x 1024 x 4096, 128 tiles: 36 us and 28)
    q.bm = q.bn = tiles(128) > kCUs / 2 ? 128 : 64;
    const long long t = tiles(q.bm);
    const int stages = (p.K + kBK - 1) / kBK;
    int s = 1;
    // split k where tiles leave half the CUs without work (with more tiles the
    // partial sums' way through memory costs more than it gains: 2048^3 24 us
    // whole, 42 in two)
    if (!q.big && t <= kCUs / 2) {
        s = (int)(kCUs / t);
        const int most = stages / 4;
        if (s > most) s = most;
        if (s > 32) s = 32;
        if (s < 1) s = 1;
    }
    q.brief = stages <= 2;
    q.per = (stages + s - 1) / s;
    if (q.per < 1) q.per = 1;
    q.slices = stages ? (stages + q.per - 1) / q.per : 1;
    return q;
}

// Operands that the tiles cannot load directly are copied first where the
// product is large enough to pay for it (the register path reaches a third of
// the rate: 4096 x 4096 x 4097 bf16 284 us, 135 with the copies; smaller ones
// lose more by the copies' launch than they gain: 1000 x 3001 x 777 18 us without
// and 23 with them, but 44 and 30 where W is read transposed).  Returns p as the tiles see it, with the copies in `at`, and the
// bytes they take.
Prod packed(const Prod &p, unsigned char *at, Pack *pack, size_t *bytes) {
    Prod q = p;
    *bytes = 0;
    if (pack) *pack = Pack{};
    if (2.0 * p.M * p.N * p.K < (p.b_mc ? 2e9 : 8e9)) return q;
    auto take = [&](int o, const void *&X, long long &ld, int rows, int cols) {
        const int chunks = (cols + 7) / 8;
        u16 *dst = reinterpret_cast<u16 *>(at + *bytes);
        if (pack) {
            pack->src[o] = static_cast<const u16 *>(X);
            pack->dst[o] = dst;
            pack->ld[o] = ld;
            pack->rows[o] = rows;
            pack->cols[o] = cols;
            pack->chunks[o] = chunks;
        }
        X = dst;
        ld = 8ll * chunks;
        *bytes += ((size_t)rows * chunks * 16 + 255) / 256 * 256;
    };
    if (!a_direct(p, 256)) {
        take(0, q.A, q.lda, p.a_mc ? p.K : p.M, p.a_mc ? p.M : p.K);
        q.a_pad = 1;
    }
    if (!b_direct(p, 256)) {
        take(1, q.B, q.ldb, p.b_mc ? p.K : p.N, p.b_mc ? p.N : p.K);
        q.b_pad = 1;
    }
    return q;
}

template <int DT, int BM, int BN, int WM, int WN, int NBUF, int KG, int AMC, int BMC>
hipError_t launch_tile(const Prod &p, const Grid16 &gr, bool ad, bool bd, hipStream_t stream) {
    // (operands that are not loaded directly have two stages whatever NBUF is)
    constexpr int NT = 64 * (BM / WM) * (BN / WN) * KG;
    const dim3 grid(gr.tiles_m * gr.tiles_n, gr.slices);
    if (ad && bd)
        hipLaunchKernelGGL((prod16_kernel<DT, BM, BN, WM, WN, NBUF, KG, AMC, BMC, true, true>), grid,
                           dim3(NT), 0, stream, p, gr);
    else if (ad && BMC)   // the backward products: G is laid out for direct loads, B may not be
        hipLaunchKernelGGL((prod16_kernel<DT, BM, BN, WM, WN, 2, KG, AMC, BMC, BMC != 0, false>), grid,
                           dim3(NT), 0, stream, p, gr);
    else
        hipLaunchKernelGGL((prod16_kernel<DT, BM, BN, WM, WN, 2, KG, AMC, BMC, false, false>), grid,
                           dim3(NT), 0, stream, p, gr);
    return hipGetLastError();
}

template <int DT, int BM, int BN, int WM, int WN, int NBUF, int KG>
hipError_t launch_layout(const Prod &p, const Grid16 &gr, bool ad, bool bd, hipStream_t stream) {
    if (!p.b_mc) return launch_tile<DT, BM, BN, WM, WN, NBUF, KG, 0, 0>(p, gr, ad, bd, stream);
    if (!p.a_mc) return launch_tile<DT, BM, BN, WM, WN, NBUF, KG, 0, 1>(p, gr, ad, bd, stream);
    return launch_tile<DT, BM, BN, WM, WN, NBUF, KG, 1, 1>(p, gr, ad, bd, stream);
}

Grid16 grid_of(const Prod &p, const Plan16 &q) {
    Grid16 gr{};
    gr.tiles_m = (p.M + q.bm - 1) / q.bm;
    gr.tiles_n = (p.N + q.bn - 1) / q.bn;
    gr.group_m = 8;
    gr.slices = q.slices;
    gr.per = q.per;
    return gr;
}

size_t sums_of(const Prod &p, const Plan16 &q) {
    const Grid16 gr = grid_of(p, q);
    return q.slices == 1 ? 0 : (size_t)gr.tiles_m * gr.tiles_n * q.slices * q.bm * q.bn * sizeof(float);
}

template <int DT>
hipError_t launch_dt(const Prod &given, const Workspace &ws, hipStream_t stream) {
    Pack pack;
    size_t bytes = 0;
    const Prod p = packed(given, static_cast<unsigned char *>(ws.ptr), &pack, &bytes);
    if (bytes) {
        hipLaunchKernelGGL(pack_kernel, dim3(2 * kCUs, 2), dim3(256), 0, stream, pack);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const Plan16 q = plan16(p);
    if (q.big) return launch_prod16_big(DT, p, stream);
    Grid16 gr = grid_of(p, q);
    gr.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws.ptr) + bytes);
    gr.count = ws.counters;
    const bool ad = a_direct(p, q.bm), bd = b_direct(p, q.bm);
    if (q.bm == 128)
        return q.brief ? launch_layout<DT, 128, 128, 64, 64, 2, 2>(p, gr, ad, bd, stream)
                       : launch_layout<DT, 128, 128, 64, 64, 4, 2>(p, gr, ad, bd, stream);
    return q.brief ? launch_layout<DT, 64, 64, 32, 32, 2, 2>(p, gr, ad, bd, stream)
                   : launch_layout<DT, 64, 64, 32, 32, 4, 2>(p, gr, ad, bd, stream);
}

// Whether dX and dW run as one launch: the same small tile, no copies, operands
// of one kind, and not so many tiles that a launch no longer matters.
bool pairs(const Prod &x, const Prod &w, const Plan16 &qx, const Plan16 &qw) {
    size_t cx, cw;
    (void)packed(x, nullptr, nullptr, &cx);
    (void)packed(w, nullptr, nullptr, &cw);
    const Grid16 gx = grid_of(x, qx), gw = grid_of(w, qw);
    return !qx.big && !qw.big && qx.bm == 64 && qw.bm == 64 && cx == 0 && cw == 0 &&
           a_direct(x, 64) && a_direct(w, 64) && b_direct(x, 64) == b_direct(w, 64) &&
           gx.tiles_m * gx.tiles_n * gx.slices + gw.tiles_m * gw.tiles_n * gw.slices <= 8 * kCUs;
}

template <int DT>
hipError_t launch_pair(const Prod &x, Grid16 gx, const Prod &w, Grid16 gw, bool dir,
                       hipStream_t stream) {
    const dim3 grid(gx.tiles_m * gx.tiles_n * gx.slices + gw.tiles_m * gw.tiles_n * gw.slices);
    if (dir)
        hipLaunchKernelGGL((prod16_pair_kernel<DT, 64, 64, 32, 32, 4, 2, true>), grid, dim3(512), 0,
                           stream, x, gx, w, gw);
    else
        hipLaunchKernelGGL((prod16_pair_kernel<DT, 64, 64, 32, 32, 2, 2, false>), grid, dim3(512), 0,
                           stream, x, gx, w, gw);
    return hipGetLastError();
}

}  // namespace

size_t prod16_pair_workspace(const Prod &x, const Prod &w) {
    const Plan16 qx = plan16(x), qw = plan16(w);
    if (pairs(x, w, qx, qw)) return sums_of(x, qx) + sums_of(w, qw);
    const size_t a = prod16_workspace(0, x), b = prod16_workspace(0, w);
    return a > b ? a : b;
}

hipError_t launch_prod16_pair(int dtype, const Prod &x, const Prod &w, const Workspace &ws,
                              hipStream_t stream) {
    const Plan16 qx = plan16(x), qw = plan16(w);
    if (!pairs(x, w, qx, qw)) {
        const hipError_t e = launch_prod16(dtype, x, ws, stream);
        return e != hipSuccess ? e : launch_prod16(dtype, w, ws, stream);
    }
    Grid16 gx = grid_of(x, qx), gw = grid_of(w, qw);
    gx.part = static_cast<float *>(ws.ptr);
    gx.count = ws.counters;
    gw.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws.ptr) + sums_of(x, qx));
    gw.count = ws.counters + kWorkspaceCounters / 2;   // (split products have at most 128 tiles)
    const bool dir = b_direct(x, 64);
    return dtype == SGEMM_DTYPE_BF16
               ? launch_pair<SGEMM_DTYPE_BF16>(x, gx, w, gw, dir, stream)
               : launch_pair<SGEMM_DTYPE_F16>(x, gx, w, gw, dir, stream);
}

size_t prod16_workspace(int, const Prod &given) {
    size_t bytes = 0;
    // (copies lie on 256-byte boundaries, as at this address)
    const Prod p = packed(given, reinterpret_cast<unsigned char *>(4096), nullptr, &bytes);
    const Plan16 q = plan16(p);
    return bytes + sums_of(p, q);
}

hipError_t launch_prod16(int dtype, const Prod &p, const Workspace &ws, hipStream_t stream) {
    return dtype == SGEMM_DTYPE_BF16 ? launch_dt<SGEMM_DTYPE_BF16>(p, ws, stream)
                                     : launch_dt<SGEMM_DTYPE_F16>(p, ws, stream);
}

}  // namespace sg
