// linear.cpp -- the C ABI of the feed-forward operators: linear layers with
// their whole epilogue, their backward pass, and the mixture-of-experts layer.
// Argument checks, empty cases, the choice of kernels, and their launches.
//
// A call makes up to three launches that hand data to each other through the
// workspace of its stream, and calls of several host threads may meet on one
// stream: the launches of a call are made under a lock, so that they stay
// together in the stream's order.
#include <cstdint>
#include <mutex>
#include <new>

#include "linear_internal.hpp"

namespace sg {
namespace {

constexpr int bad(int argument) { return -100 - argument; }

int to_status(hipError_t e) { return (int)e; }

int elem_of(int dtype) { return dtype == SGEMM_DTYPE_F32 ? 4 : 2; }
bool known(int dtype) {
    return dtype == SGEMM_DTYPE_F32 || dtype == SGEMM_DTYPE_BF16 || dtype == SGEMM_DTYPE_F16;
}
bool aligned(const void *q, int to) { return reinterpret_cast<uintptr_t>(q) % to == 0; }
bool usable(const void *q, int elem) { return q && aligned(q, elem); }
size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

std::mutex &launch_mutex() {
    static std::mutex m;
    return m;
}

// f's status; a C++ exception (host memory, a mutex) becomes one, since none may
// cross the C interface.
template <class F>
int guarded(F &&f) {
    try {
        return f();
    } catch (const std::bad_alloc &) {
        return to_status(hipErrorOutOfMemory);
    } catch (...) {
        return to_status(hipErrorUnknown);
    }
}

// The feed-forward workspace of a call: acquired (where bytes are needed),
// used by the launches of f, and released.
template <class F>
int with_workspace(size_t bytes, bool counters, hipStream_t stream, F &&f) {
    std::lock_guard<std::mutex> lock(launch_mutex());
    Workspace ws;
    if (bytes || counters) {
        const hipError_t e = workspace_acquire(bytes, stream, Problem{}, ws, 1);
        if (e != hipSuccess) return to_status(e);
    }
    int st = f(ws);
    const hipError_t e = workspace_release(ws, stream);
    return st != 0 ? st : to_status(e);
}

// An fp32 product with its partial sums at the front of the workspace.
int run_in(Problem p, const Workspace &ws, size_t bytes, hipStream_t stream) {
    if (bytes) {
        p.scratch = ws.base;
        p.scratch_bytes = bytes;
    }
    return run_product(p, stream);
}

size_t ours_workspace(int dtype, const Prod &p, bool rows) {
    return rows ? rows_workspace(dtype, p) : prod16_workspace(dtype, p);
}
hipError_t launch_product(int dtype, const Prod &p, bool rows, const Workspace &ws,
                          hipStream_t stream) {
    return rows ? launch_rows(dtype, p, ws, stream) : launch_prod16(dtype, p, ws, stream);
}

int run_linear(int dtype, const Prod &p, hipStream_t stream) {
    const bool rows = p.M <= kFewRows;
    if (dtype != SGEMM_DTYPE_F32 || rows) {
        const size_t bytes = ours_workspace(dtype, p, rows);
        return with_workspace(bytes, false, stream, [&](const Workspace &ws) {
            return to_status(launch_product(dtype, p, rows, ws, stream));
        });
    }
    // fp32: the library's product with its fused epilogue where the tile has one
    // that serves these operands; otherwise with the bias in the product's
    // epilogue and one elementwise pass for what comes after
    const float *A = static_cast<const float *>(p.A), *B = static_cast<const float *>(p.B);
    const float *bias = static_cast<const float *>(p.bias), *R = static_cast<const float *>(p.R);
    float *Y = static_cast<float *>(p.C), *Z = static_cast<float *>(p.Z);
    Problem q{p.M, p.N, p.K, 1.f, 0.f, A, p.lda, B, p.ldb, Y, p.ldc};
    q.trans_b = 1;
    q.bias = bias;
    q.act = p.act;
    if ((R || Z) && p.K > 0) {
        Problem f = q;
        f.R = R;
        f.ldr = p.ldr;
        f.Z = Z;
        f.ldz = p.ldz;
        const int st = run_fused_linear(f, stream);
        if (st != kNotFused) return st;
    }
    // R may be Y, so the sum goes elsewhere first: to Z, or to the workspace
    const bool temp = R && !Z;
    const long long ld = (long long)round_up(p.N, 4);
    if (Z) {
        q.C = Z;
        q.ldc = p.ldz;
        q.act = SGEMM_ACT_NONE;
    } else if (temp) {
        q.C = reinterpret_cast<float *>(uintptr_t{4096});   // (for the plan: an aligned place)
        q.ldc = ld;
    }
    const size_t sums = round_up(product_workspace(q), 256);
    return with_workspace(sums + (temp ? (size_t)ld * p.M * 4 : 0), false, stream,
                          [&](const Workspace &ws) -> int {
        if (temp) q.C = reinterpret_cast<float *>(static_cast<unsigned char *>(ws.ptr) + sums);
        const int st = run_in(q, ws, sums, stream);
        if (st != 0 || (!R && !Z)) return st;
        return to_status(launch_finish32(p.M, p.N, q.C, q.ldc, temp ? SGEMM_ACT_NONE : p.act, R,
                                         p.ldr, Y, p.ldc, stream));
    });
}

// An fp32 product of the backward pass with few tiles of C and a long inner
// length leaves most CUs idle in the plans of single products: its inner
// length is cut into equal chunks, run as one batch (and one product for what is
// left over), and the partial products are added in order (7600 x 136 x 589: dX and
// dW take 29 and 54 us, the two uncut 331; beyond 128 tiles of 128 x 128 one
// product fills the card by itself).
struct Chunks {
    int count = 0, k = 0, rest = 0;   // 0: not cut
    long long ld = 0, step = 0;       // of the partial products
    size_t bytes = 0, sums = 0;       // the partial products, and the batch's own sums
};

Problem chunk_of(const Problem &p, const Chunks &c, float *parts) {
    Problem q = p;
    q.K = c.k;
    q.batch = c.count;
    q.stride_a = p.trans_a ? (long long)c.k * p.lda : c.k;
    q.stride_b = (long long)c.k * p.ldb;   // (B is never transposed here)
    q.C = parts;
    q.ldc = c.ld;
    q.stride_c = c.step;
    return q;
}
Problem rest_of(const Problem &p, const Chunks &c, float *parts) {
    Problem q = p;
    const long long k = (long long)c.k * c.count;
    q.K = c.rest;
    q.A = p.trans_a ? p.A + k * p.lda : p.A + k;
    q.B = p.B + k * p.ldb;
    q.C = parts + c.count * c.step;
    q.ldc = c.ld;
    return q;
}

Chunks chunks_of(const Problem &p) {
    Chunks c;
    if (p.M == 0 || p.N == 0) return c;
    const long long tiles = (long long)((p.M + 127) / 128) * ((p.N + 127) / 128);
    // a chunk of 256 at least: enough to pay for writing and adding its result
    long long n = tiles > 128 ? 1 : 512 / tiles;
    if (n > p.K / 256) n = p.K / 256;
    if (n > 32) n = 32;
    if (n < 2) return c;
    c.k = (int)(p.K / n / 16 * 16);
    c.count = p.K / c.k;
    c.rest = p.K - c.count * c.k;
    c.ld = (long long)round_up(p.N, 4);
    c.step = c.ld * p.M;
    c.bytes = round_up((size_t)c.step * (c.count + 1) * 4, 256);
    float *at = reinterpret_cast<float *>(uintptr_t{4096});   // (for the plans: an aligned place)
    c.sums = product_workspace(chunk_of(p, c, at));
    const size_t r = c.rest ? product_workspace(rest_of(p, c, at)) : 0;
    if (r > c.sums) c.sums = r;
    c.sums = round_up(c.sums, 256);
    return c;
}

size_t chunked_workspace(const Problem &p) {
    const Chunks c = chunks_of(p);
    return c.count ? c.sums + c.bytes : product_workspace(p);
}

// p with its partial sums (`bytes` as chunked_workspace) at the front of the
// workspace.
int run_chunked(const Problem &p, const Workspace &ws, hipStream_t stream) {
    const Chunks c = chunks_of(p);
    if (!c.count) return run_in(p, ws, product_workspace(p), stream);
    float *parts = reinterpret_cast<float *>(static_cast<unsigned char *>(ws.ptr) + c.sums);
    int st = run_in(chunk_of(p, c, parts), ws, c.sums, stream);
    if (st == 0 && c.rest) st = run_in(rest_of(p, c, parts), ws, c.sums, stream);
    if (st != 0) return st;
    return to_status(launch_sum32(p.M, p.N, parts, c.ld, c.step, c.count + (c.rest ? 1 : 0), p.C,
                                  p.ldc, stream));
}

struct Backward {
    int M, N, K;
    const void *dY;
    int lddy;
    const void *Z;
    int ldz, act;
    const void *X;
    int ldx;
    const void *W;
    int ldw;
    void *dX;
    int lddx;
    void *dW;
    int lddw;
    void *db;
};

int run_backward(int dtype, const Backward &b, hipStream_t stream) {
    const int elem = elem_of(dtype), v = 16 / elem;
    const bool f32 = dtype == SGEMM_DTYPE_F32;
    const bool want_dx = b.dX && b.M > 0 && b.K > 0, want_dw = b.dW && b.N > 0 && b.K > 0;
    const bool want_db = b.db && b.N > 0;
    const bool few = b.M <= kFewRows;
    // G is dY itself without an activation, as long as the 16-bit tiles can
    // load its rows directly (the few-rows kernels load any)
    const bool g_is_dy = b.act == SGEMM_ACT_NONE &&
                         (f32 || few || (rows16(b.dY, b.lddy, elem) && b.N % v == 0));
    const bool make_g = !g_is_dy && (want_dx || want_dw) && b.M > 0 && b.N > 0;
    // few rows: both products are bound by W and dW, so G is kept in two parts
    // (as exact as fp32) at no cost; otherwise its rounding adds an error of
    // the size of the results' own rounding (ReLU's slope is 0 or 1: nothing to
    // round)
    const bool two = make_g && few && !f32 && b.act != SGEMM_ACT_NONE && b.act != SGEMM_ACT_RELU;
    const long long ldg = make_g ? (long long)round_up(b.N, v) : b.lddy;
    const size_t g_bytes =
        make_g ? round_up((size_t)(two ? 2 : 1) * b.M * ldg * elem, 256) : 0;

    // (plans are made before G has its place: as well aligned as this)
    const void *g_at = make_g ? reinterpret_cast<const void *>(uintptr_t{4096}) : b.dY;
    Prod dx{b.M, b.K, b.N, g_at, ldg, b.W, b.ldw, b.dX, b.lddx};
    dx.b_mc = 1;
    Prod dw{b.N, b.K, b.M, g_at, ldg, b.X, b.ldx, b.dW, b.lddw};
    dw.a_mc = dw.b_mc = 1;
    dx.a_pad = dw.a_pad = make_g;
    const bool dx_ours = want_dx && (!f32 || few), dw_ours = want_dw && (!f32 || few);
    auto op32 = [&](int ta, int M, int N, int K, const void *A, long long lda, const void *B, int ldb,
                    void *C, int ldc) {
        Problem q{M, N, K, 1.f, 0.f, static_cast<const float *>(A), lda, static_cast<const float *>(B),
                  ldb, static_cast<float *>(C), ldc};
        q.trans_a = ta;
        return q;
    };
    // fp32 products of more than a few rows run as the library's own
    Problem dx32 = op32(0, b.M, b.K, b.N, g_at, ldg, b.W, b.ldw, b.dX, b.lddx);
    Problem dw32 = op32(1, b.N, b.K, b.M, g_at, ldg, b.X, b.ldx, b.dW, b.lddw);
    const bool dx_lib = want_dx && !dx_ours, dw_lib = want_dw && !dw_ours;
    size_t scratch = want_db ? grad_workspace(dtype, b.M, b.N) : 0;
    if (dx_lib && chunked_workspace(dx32) > scratch) scratch = chunked_workspace(dx32);
    if (dw_lib && chunked_workspace(dw32) > scratch) scratch = chunked_workspace(dw32);
    if (dx_ours) {
        const size_t s = ours_workspace(dtype, dx, few);
        if (s > scratch) scratch = s;
    }
    if (dw_ours && !few) {
        const size_t s = ours_workspace(dtype, dw, false);
        if (s > scratch) scratch = s;
    }
    const bool pair = dx_ours && dw_ours && !few;   // 16-bit, more than a few rows
    if (pair && prod16_pair_workspace(dx, dw) > scratch) scratch = prod16_pair_workspace(dx, dw);
    // the workspace: the launches' partial sums, one after another's, then G
    scratch = round_up(scratch, 256);
    return with_workspace(scratch + g_bytes, false, stream, [&](const Workspace &ws) -> int {
        if (make_g || want_db) {
            unsigned char *G = make_g ? static_cast<unsigned char *>(ws.ptr) + scratch : nullptr;
            void *lo = two ? G + (size_t)b.M * ldg * elem : nullptr;
            const hipError_t e =
                launch_grad(dtype, b.M, b.N, b.dY, b.lddy, b.Z, b.ldz, b.act, G, lo, ldg,
                            want_db ? b.db : nullptr, static_cast<float *>(ws.ptr), ws.counters,
                            stream);
            if (e != hipSuccess) return to_status(e);
            if (make_g) {
                dx.A = dw.A = G;
                dx32.A = dw32.A = reinterpret_cast<const float *>(G);
            }
            dx.lo = dw.lo = lo;
        }
        if (pair) return to_status(launch_prod16_pair(dtype, dx, dw, ws, stream));
        if (want_dx) {
            const int st = dx_lib ? run_chunked(dx32, ws, stream)
                                  : to_status(launch_product(dtype, dx, few, ws, stream));
            if (st != 0) return st;
        }
        if (!want_dw) return 0;
        if (dw_lib) return run_chunked(dw32, ws, stream);
        return to_status(few ? launch_outer(dtype, dw, stream)
                             : launch_product(dtype, dw, false, ws, stream));
    });
}

}  // namespace
}  // namespace sg

extern "C" {

int sgemm_linear(int dtype, int M, int N, int K, const void *X, int ldx, const void *W, int ldw,
                 const void *bias, const void *R, int ldr, int act, void *Y, int ldy, void *Z,
                 int ldz, hipStream_t stream) {
    using namespace sg;
    if (!known(dtype)) return bad(1);
    const int elem = elem_of(dtype);
    if (M < 0) return bad(2);
    if (N < 0) return bad(3);
    if (K < 0) return bad(4);
    if (ldx < (K > 1 ? K : 1)) return bad(6);
    if (ldw < (K > 1 ? K : 1)) return bad(8);
    if (bias && !aligned(bias, elem)) return bad(9);
    if (R && !aligned(R, elem)) return bad(10);
    if (R && ldr < (N > 1 ? N : 1)) return bad(11);
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_GELU_TANH) return bad(12);
    if (ldy < (N > 1 ? N : 1)) return bad(14);
    if (Z && !aligned(Z, elem)) return bad(15);
    if (Z && ldz < (N > 1 ? N : 1)) return bad(16);
    if (M == 0 || N == 0) return 0;
    if (K > 0 && !usable(X, elem)) return bad(5);
    if (K > 0 && !usable(W, elem)) return bad(7);
    if (!usable(Y, elem)) return bad(13);
    Prod p{M, N, K, X, ldx, W, ldw, Y, ldy};
    p.bias = bias;
    p.R = R;
    p.ldr = ldr;
    p.Z = Z;
    p.ldz = ldz;
    p.act = act;
    return guarded([&] { return run_linear(dtype, p, stream); });
}

int sgemm_linear_backward(int dtype, int M, int N, int K, const void *dY, int lddy, const void *Z,
                          int ldz, int act, const void *X, int ldx, const void *W, int ldw,
                          void *dX, int lddx, void *dW, int lddw, void *db, hipStream_t stream) {
    using namespace sg;
    if (!known(dtype)) return bad(1);
    const int elem = elem_of(dtype);
    if (M < 0) return bad(2);
    if (N < 0) return bad(3);
    if (K < 0) return bad(4);
    const int n1 = N > 1 ? N : 1, k1 = K > 1 ? K : 1;
    if (lddy < n1) return bad(6);
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_GELU_TANH) return bad(9);
    const bool cells = M > 0 && N > 0;
    if (cells && !usable(dY, elem)) return bad(5);
    if (cells && act != SGEMM_ACT_NONE && !usable(Z, elem)) return bad(7);
    if (act != SGEMM_ACT_NONE && ldz < n1) return bad(8);
    if (dW && ldx < k1) return bad(11);
    if (dW && cells && K > 0 && !usable(X, elem)) return bad(10);
    if (dX && ldw < k1) return bad(13);
    if (dX && cells && K > 0 && !usable(W, elem)) return bad(12);
    if (dX && !aligned(dX, elem)) return bad(14);
    if (dX && lddx < k1) return bad(15);
    if (dW && !aligned(dW, elem)) return bad(16);
    if (dW && lddw < k1) return bad(17);
    if (db && !aligned(db, elem)) return bad(18);
    const Backward b{M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX, lddx, dW, lddw, db};
    return guarded([&] { return run_backward(dtype, b, stream); });
}

int sgemm_moe(int dtype, int T, int D, int F, int E, int top_k, int gated, int renormalize, int act,
              const void *X, int ldx, const void *Wr, int ldr, const void *W1, int ld1,
              long long stride1, const void *W2, int ld2, long long stride2, void *Y, int ldy,
              int *ids, float *weights, hipStream_t stream) {
    using namespace sg;
    if (!known(dtype)) return bad(1);
    const int elem = elem_of(dtype);
    if (T < 0 || T > kMoeTokens) return bad(2);
    if (D < 1 || D > kMoeWidth) return bad(3);
    if (F < 1 || F > (1 << 20)) return bad(4);
    if (E < 1 || E > kMoeExperts) return bad(5);
    if (top_k < 1 || top_k > kMoeChoices || top_k > E) return bad(6);
    if (gated != 0 && gated != 1) return bad(7);
    if (renormalize != 0 && renormalize != 1) return bad(8);
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_GELU_TANH) return bad(9);
    if (ldx < D) return bad(11);
    if (ldr < D) return bad(13);
    if (ld1 < D) return bad(15);
    if (stride1 < 0) return bad(16);
    if (ld2 < F) return bad(18);
    if (stride2 < 0) return bad(19);
    if (ldy < D) return bad(21);
    if (ids && !aligned(ids, 4)) return bad(22);
    if (weights && !aligned(weights, 4)) return bad(23);
    if (T == 0) return 0;
    if (!usable(X, elem)) return bad(10);
    if (!usable(Wr, elem)) return bad(12);
    if (!usable(W1, elem)) return bad(14);
    if (!usable(W2, elem)) return bad(17);
    if (!usable(Y, elem)) return bad(20);
    const Moe m{T,  D,   F,   E,       top_k, gated, renormalize, act,     X, ldx, Wr, ldr,
                W1, ld1, stride1, W2,  ld2,   stride2, Y,         ldy, ids, weights};
    return guarded([&] {
        return with_workspace(moe_workspace(m), true, stream, [&](const Workspace &ws) {
            return to_status(launch_moe(dtype, m, ws, stream));
        });
    });
}

}  // extern "C"
