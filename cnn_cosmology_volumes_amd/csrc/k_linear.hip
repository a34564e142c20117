// Linear layers over rows (a dense layer, or a 1^3 convolution over voxels):
//   pre = X W + bias,  Y = act(pre) + R            X [rows][in], W [in][out]
// and backward, with D = dY act'(pre):
//   dX = D W^T,  dW = X^T D,  db = column sums of D.
//
// One product kernel serves all three, C [M][N] = sum_k A(m, k) B(k, n), for
// operands whose values lie along k (X and D in the first two, W in W^T) or
// across it (W forward, both operands of dW).
#include "cf_internal.h"

#include <math.h>

namespace cf {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int LIN_T = 256;

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf2f(v); }

struct LinAct {
    int act;
    float slope;
};
__device__ __forceinline__ float lin_act(const LinAct& a, float z)
{
    if (a.act == CF_ACT_SILU) return z * __builtin_amdgcn_rcpf(1.f + __expf(-z));
    return z > 0.f ? z : a.slope * z;
}
__device__ __forceinline__ float lin_dact(const LinAct& a, float z)
{
    if (a.act == CF_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
        return s * fmaf(z, 1.f - s, 1.f);
    }
    return z > 0.f ? 1.f : a.slope;
}

// What becomes of the product.
enum LinMode {
    LIN_FWD,        // bias, pre, activation, residual
    LIN_PLAIN,      // rounded to TO
};

template <typename T> struct LinProduct {
    const T* A;
    const T* B;
    const T* B2;            // k >= K: B2(k - K, n) with A(m, k - K), or null
    int64_t M, K;
    int N;
    int64_t lda, ldb;
    int64_t tiles_m;
    int tiles_n;
    int splits;             // of the reduction
    int kb, kb_split;       // pieces of the reduction, and of a split
    float* part;            // [splits][M][N], where splits > 1
    float* db_part;         // [db_parts][N], column sums of B
    int db_parts;
    void* C;
    const float* bias;
    const T* R;
    T* pre;
    LinAct act;
    float* db;
};

template <typename T> struct LinTile;
template <> struct LinTile<uint16_t> {
    static constexpr int V = 8, BK = 64;
};
template <> struct LinTile<float> {
    static constexpr int V = 4, BK = 32;
};

// Values from p on, of which n are inside; zeros for the others.
template <typename T> __device__ __forceinline__ uint4 lin_chunk(const T* p, int64_t n)
{
    constexpr int V = LinTile<T>::V;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n >= V) {
        __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
        T t[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) t[i] = p[i];
        __builtin_memcpy(&v, t, 16);
    }
    return v;
}

// An operand's piece in LDS: along k [ROWS][BK], across it [BK][ROWS], rows a
// few banks apart.
template <typename T, bool ALONG, int ROWS> struct LinOperand {
    static constexpr int V = LinTile<T>::V, BK = LinTile<T>::BK;
    static constexpr int PITCH = ALONG ? BK + V : ROWS + (sizeof(T) == 2 ? 32 : 8);
    static constexpr int SIZE = (ALONG ? ROWS : BK) * PITCH;
    static constexpr int CHUNKS = ROWS * BK / V / LIN_T;        // a thread's
    static_assert(ROWS * BK / V % LIN_T == 0, "whole rounds");

    __device__ static __forceinline__ void fetch(uint4 (&reg)[CHUNKS], const T* p, int64_t ld, int64_t r0, int64_t rows,
                                                 int64_t k0, int64_t K)
    {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = i * LIN_T + (int)threadIdx.x;
            if (ALONG) {
                const int64_t r = r0 + c / (BK / V), k = k0 + c % (BK / V) * V;
                reg[i] = lin_chunk<T>(p + r * ld + k, r < rows ? K - k : 0);
            } else {
                const int64_t k = k0 + c / (ROWS / V), r = r0 + c % (ROWS / V) * V;
                reg[i] = lin_chunk<T>(p + k * ld + r, k < K ? rows - r : 0);
            }
        }
    }
    __device__ static __forceinline__ void put(T* s, const uint4 (&reg)[CHUNKS])
    {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = i * LIN_T + (int)threadIdx.x;
            const int at = ALONG ? c / (BK / V) * PITCH + c % (BK / V) * V : c / (ROWS / V) * PITCH + c % (ROWS / V) * V;
            *reinterpret_cast<uint4*>(s + at) = reg[i];
        }
    }
    // bf16: the fragment of a 32 x 32 x 16 product at row r, step ks of the piece:
    // row r + lane % 32, k = 16 ks + 8 (lane / 32) + 0..7.
    __device__ static __forceinline__ bf16x8 frag(const uint16_t* s, int r, int ks)
    {
        const int lane = (int)threadIdx.x & 63;
        if (ALONG) return *reinterpret_cast<const bf16x8*>(s + (r + lane % 32) * PITCH + ks * 16 + lane / 32 * 8);
        // Sixteen lanes read four values of four rows of k each; lane i gets
        // column i of these 4 x 16 values.
        const int i = lane & 15, row = r + (lane & 16) + 4 * (i & 3), k = ks * 16 + lane / 32 * 8 + (i >> 2);
        typedef __attribute__((address_space(3))) s16x4* lds4;
        union {
            s16x4 h[2];
            bf16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + k * PITCH + row));
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + (k + 4) * PITCH + row));
        return u.v;
    }
    // fp32: values of row r + lane % 32 at k = 8 ks + 4 (lane / 32) + 0..3, one for
    // each of four 32 x 32 x 2 products.
    __device__ static __forceinline__ f32x4 frag(const float* s, int r, int ks)
    {
        const int lane = (int)threadIdx.x & 63, k = ks * 8 + lane / 32 * 4;
        if (ALONG) return *reinterpret_cast<const f32x4*>(s + (r + lane % 32) * PITCH + k);
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = s[(k + j) * PITCH + r + lane % 32];
        return v;
    }
};

__device__ __forceinline__ void lin_mma(const bf16x8& a, const bf16x8& b, f32x16& c)
{
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void lin_mma(const f32x4& a, const f32x4& b, f32x16& c)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 ones(const bf16x8&)
{
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (__bf16)1.f;
    return v;
}
__device__ __forceinline__ f32x4 ones(const f32x4&) { return f32x4{1.f, 1.f, 1.f, 1.f}; }

// One value of the result.
template <typename T, typename TO, int MODE>
__device__ __forceinline__ void lin_result(const LinProduct<T>& q, int64_t m, int n, float v)
{
    const int64_t at = m * q.N + n;
    if (MODE == LIN_FWD) {
        if (q.bias) v += q.bias[n];
        if (q.pre) Elem<T>::store(q.pre, at, v);
        v = lin_act(q.act, v);
        if (q.R) v += widen(q.R[at]);
    }
    Elem<TO>::store((TO*)q.C, at, v);
}

// TILE x TILE of the result a block, four waves of TILE/2 x TILE/2.
template <typename T, typename TO, bool AA, bool BA, int TILE, int MODE, bool DB>
__global__ __launch_bounds__(LIN_T) void lin_product_kernel(LinProduct<T> q)
{
    using OA = LinOperand<T, AA, TILE>;
    using OB = LinOperand<T, BA, TILE>;
    constexpr int BK = LinTile<T>::BK, STEPS = BK / (sizeof(T) == 2 ? 16 : 8), B = TILE / 64;
    __shared__ __attribute__((aligned(16))) T sa[OA::SIZE];
    __shared__ __attribute__((aligned(16))) T sb[OB::SIZE];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int wi = wave / 2 * (TILE / 2), wj = wave % 2 * (TILE / 2);
    const int64_t units = q.tiles_m * q.tiles_n * q.splits;
    for (int64_t u = xcd_remap(blockIdx.x, gridDim.x); u < units; u += gridDim.x) {
        const int split = (int)(u % q.splits);
        const int64_t t = u / q.splits, ti = t / q.tiles_n;
        const int tj = (int)(t % q.tiles_n);
        const int64_t i0 = ti * TILE;
        const int j0 = tj * TILE;
        const int b0 = split * q.kb_split, total = q.B2 ? 2 * q.kb : q.kb;
        const int b1 = min(b0 + q.kb_split, total);
        f32x16 acc[B][B] = {};
        f32x16 col[B] = {};
        const bool sums = DB && ti == 0 && wi == 0;
        uint4 ra[OA::CHUNKS], rb[OB::CHUNKS];
        auto fetch = [&](int b) {
            const bool second = b >= q.kb;
            const int64_t k0 = (int64_t)(second ? b - q.kb : b) * BK;
            OA::fetch(ra, q.A, q.lda, i0, q.M, k0, q.K);
            OB::fetch(rb, second ? q.B2 : q.B, q.ldb, j0, q.N, k0, q.K);
        };
        if (b0 < b1) fetch(b0);
        for (int b = b0; b < b1; ++b) {
            __syncthreads();
            OA::put(sa, ra);
            OB::put(sb, rb);
            __syncthreads();
            if (b + 1 < b1) fetch(b + 1);
#pragma unroll
            for (int ks = 0; ks < STEPS; ++ks) {
                decltype(OA::frag(sa, 0, 0)) fa[B], fb[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    fa[i] = OA::frag(sa, wi + i * 32, ks);
                    fb[i] = OB::frag(sb, wj + i * 32, ks);
                }
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int j = 0; j < B; ++j) lin_mma(fa[i], fb[j], acc[i][j]);
                if (DB && sums)
#pragma unroll
                    for (int j = 0; j < B; ++j) lin_mma(ones(fb[j]), fb[j], col[j]);
            }
        }
        // register r of a lane: row 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int n = j0 + wj + j * 32 + lane % 32;
            if (n >= q.N) continue;
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t m = i0 + wi + i * 32 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
                    if (m >= q.M) continue;
                    if (q.splits > 1) q.part[((int64_t)split * q.M + m) * q.N + n] = acc[i][j][r];
                    else lin_result<T, TO, MODE>(q, m, n, acc[i][j][r]);
                }
            if (DB && sums && lane < 32 && q.db) {
                if (q.splits > 1) q.db_part[(int64_t)split * q.N + n] = col[j][0];
                else q.db[n] = col[j][0];
            }
        }
    }
}

// Adds the splits' sums in order, and in the blocks past `main` those of db, 16
// columns a block and 16 threads to a column.
template <typename T, typename TO, int MODE>
__global__ __launch_bounds__(256) void lin_join_kernel(LinProduct<T> q, int main)
{
    __shared__ double sh[16][17];
    if ((int)blockIdx.x >= main) {
        const int c = ((int)blockIdx.x - main) * 16 + (int)threadIdx.x % 16, k = (int)threadIdx.x / 16;
        double sum = 0.0;
        if (c < q.N)
            for (int i = k; i < q.db_parts; i += 16) sum += (double)q.db_part[(int64_t)i * q.N + c];
        sh[k][threadIdx.x % 16] = sum;
        __syncthreads();
        if (k == 0 && c < q.N) {
            for (int i = 1; i < 16; ++i) sum += sh[i][threadIdx.x];
            q.db[c] = (float)sum;
        }
        return;
    }
    const int64_t total = q.M * q.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)main * 256) {
        float v = 0.f;
        for (int s = 0; s < q.splits; ++s) v += q.part[s * total + i];
        lin_result<T, TO, MODE>(q, i / q.N, (int)(i % q.N), v);
    }
}

// D = dY act'(pre): fp32, or as bf16 hi and lo = D - hi, which together keep 16
// bits or more: dW is fp32 and would show the rounding of hi alone (2^-9 of every
// term).  dX, rounded to bf16 itself, takes hi alone.
// A block takes a range of rows, 2^lg lanes to a row, and leaves the column sums of D.
template <typename T>
__global__ __launch_bounds__(256) void lin_gate_kernel(const T* __restrict__ pre, const T* __restrict__ dY, T* hi, T* lo,
                                                       int64_t rows, int N, int lg, LinAct act, float* db_part)
{
    constexpr int V = LinTile<T>::V;
    __shared__ float sh[256 * V];
    const int lane = (int)threadIdx.x & ((1 << lg) - 1), c = (((int)blockIdx.y << lg) + lane) * V;
    const int64_t r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
    float sum[V] = {};
    if (c < N)
        for (int64_t r = r0 + ((int)threadIdx.x >> lg); r < r1; r += 256 >> lg) {
            const int64_t at = r * N + c;
            T z[V] = {}, d[V] = {}, h[V], l[V];
            const bool whole = c + V <= N;
            if (whole) {
                __builtin_memcpy(z, pre + at, 16);
                __builtin_memcpy(d, dY + at, 16);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < N) {
                        z[j] = pre[at + j];
                        d[j] = dY[at + j];
                    }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = widen(d[j]) * lin_dact(act, widen(z[j]));
                sum[j] += v;
                Elem<T>::store(h, j, v);
                // (an infinite hi stands for itself: inf - inf would make NaN of it)
                const float rest = v - widen(h[j]);
                if (sizeof(T) == 2) Elem<T>::store(l, j, __builtin_isfinite(widen(h[j])) ? rest : 0.f);
            }
            if (whole) {
                __builtin_memcpy(hi + at, h, 16);
                if (sizeof(T) == 2) __builtin_memcpy(lo + at, l, 16);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < N) {
                        hi[at + j] = h[j];
                        if (sizeof(T) == 2) lo[at + j] = l[j];
                    }
            }
        }
    if (!db_part) return;
#pragma unroll
    for (int j = 0; j < V; ++j) sh[j * 256 + (int)threadIdx.x] = sum[j];
    __syncthreads();
    // sum j of the lanes of one column lies at j 256 + lane, 2^lg apart
    for (int i = (int)threadIdx.x; i < V << lg; i += 256) {
        const int j = i >> lg, k = i & ((1 << lg) - 1), col = (((int)blockIdx.y << lg) + k) * V + j;
        if (col >= N) continue;
        float v = 0.f;
        for (int g = 0; g < 256 >> lg; ++g) v += sh[j * 256 + (g << lg) + k];
        db_part[(int64_t)blockIdx.x * N + col] = v;
    }
}

size_t up256l(size_t b) { return (b + 255) & ~(size_t)255; }

// Tiles and splits of a product.
struct LinPlan {
    int tile;
    int64_t tiles_m;
    int tiles_n, kb, kb_split, splits;
    size_t part_bytes, db_bytes;
};
LinPlan lin_plan(int64_t M, int N, int64_t K, int size, int passes)
{
    LinPlan p;
    const int bk = size == 2 ? 64 : 32;
    const int64_t t128 = (M + 127) / 128 * ((N + 127) / 128);
    p.tile = t128 >= 256 ? 128 : 64;
    p.tiles_m = (M + p.tile - 1) / p.tile;
    p.tiles_n = (N + p.tile - 1) / p.tile;
    p.kb = (int)((K + bk - 1) / bk);
    const int64_t tiles = p.tiles_m * p.tiles_n, total = (int64_t)p.kb * passes;
    int64_t want = tiles >= 256 ? 1 : (512 + tiles - 1) / tiles;
    want = want < (total + 3) / 4 ? want : (total + 3) / 4;
    p.kb_split = (int)((total + want - 1) / want);
    p.splits = (int)((total + p.kb_split - 1) / p.kb_split);
    p.part_bytes = p.splits > 1 ? up256l((size_t)p.splits * (size_t)M * N * 4) : 0;
    p.db_bytes = p.splits > 1 ? up256l((size_t)p.splits * N * 4) : 0;
    return p;
}

// Lanes of a row (log2), columns of blocks and parts of the rows of lin_gate_kernel.
struct LinGate {
    int lg, cols, parts;
    size_t bytes, db_bytes;      // of hi or lo, of the column sums
};
LinGate lin_gate(int64_t rows, int N, int size)
{
    const int V = 16 / size, vecs = (N + V - 1) / V;
    LinGate g;
    g.lg = 0;
    while (g.lg < 8 && 1 << g.lg < vecs) ++g.lg;
    g.cols = (vecs + (1 << g.lg) - 1) >> g.lg;
    const int64_t most = (1024 + g.cols - 1) / g.cols, each = 4 * (256 >> g.lg), want = (rows + each - 1) / each;
    g.parts = (int)(want < most ? want : most);
    g.bytes = up256l((size_t)rows * N * size);
    g.db_bytes = up256l((size_t)g.parts * N * 4);
    return g;
}

// The product over K of B (and then of B2, if there is one).  DB: q.db is formed
// with it; else q.db_part already holds its parts, if q.db is not null.
template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t lin_run(LinProduct<T> q, int64_t M, int N, int64_t K, const T* A, int64_t lda, const T* B, const T* B2,
                   int64_t ldb, void* ws, hipStream_t s)
{
    const LinPlan p = lin_plan(M, N, K, (int)sizeof(T), B2 ? 2 : 1);
    q.A = A;
    q.B = B;
    q.B2 = B2;
    q.M = M;
    q.N = N;
    q.K = K;
    q.lda = lda;
    q.ldb = ldb;
    q.tiles_m = p.tiles_m;
    q.tiles_n = p.tiles_n;
    q.splits = p.splits;
    q.kb = p.kb;
    q.kb_split = p.kb_split;
    q.part = (float*)ws;
    if (DB) {
        q.db_part = (float*)((char*)ws + p.part_bytes);
        q.db_parts = p.splits;
    }
    const int64_t units = p.tiles_m * p.tiles_n * p.splits, most = 1 << 20;
    const unsigned grid = (unsigned)(units < most ? units : most);
    if (p.tile == 128) lin_product_kernel<T, TO, AA, BA, 128, MODE, DB><<<grid, LIN_T, 0, s>>>(q);
    else lin_product_kernel<T, TO, AA, BA, 64, MODE, DB><<<grid, LIN_T, 0, s>>>(q);
    hipError_t e = hipGetLastError();
    const bool join_db = q.db && (!DB || p.splits > 1);
    if (e != hipSuccess || (p.splits == 1 && !join_db)) return e;
    const int64_t blocks = p.splits > 1 ? (M * N + 255) / 256 : 0;
    const int main = (int)(blocks < 4096 ? blocks : 4096);
    lin_join_kernel<T, TO, MODE><<<(unsigned)(main + (join_db ? (N + 15) / 16 : 0)), 256, 0, s>>>(q, main);
    return hipGetLastError();
}

}  // namespace

size_t linear_ws_bytes(cf_dtype dt, int64_t rows, int in, int out, bool bwd)
{
    const int size = dt == CF_F32 ? 4 : 2;
    if (!bwd) return lin_plan(rows, out, in, size, 1).part_bytes;
    const LinGate g = lin_gate(rows, out, size);
    const LinPlan x = lin_plan(rows, in, out, size, 1), w = lin_plan(in, out, rows, size, size == 2 ? 2 : 1),
                  one = lin_plan(in, out, rows, size, 1);
    const size_t gated = g.bytes * (size == 2 ? 2 : 1) + g.db_bytes, plain = one.part_bytes + one.db_bytes;
    const size_t most = gated + (w.part_bytes > x.part_bytes ? w.part_bytes : x.part_bytes);
    return most > plain ? most : plain;
}

template <typename T>
hipError_t launch_linear_fwd(int64_t rows, int in, int out, const T* X, const T* W, const float* bias, cf_act act,
                             float slope, const T* R, T* pre, T* Y, void* ws, hipStream_t s)
{
    LinProduct<T> q{};
    q.C = Y;
    q.bias = bias;
    q.R = R;
    q.pre = pre;
    q.act = LinAct{(int)act, slope};
    return lin_run<T, T, true, false, LIN_FWD, false>(q, rows, out, in, X, in, W, nullptr, out, ws, s);
}

template <typename T>
hipError_t launch_linear_bwd(int64_t rows, int in, int out, const T* X, const T* W, const T* pre, const T* dY,
                             cf_act act, float slope, T* dX, float* dW, float* db, void* ws, hipStream_t s)
{
    const bool gated = act == CF_ACT_SILU || slope != 1.f;
    const T* D = dY;
    const T* lo = nullptr;
    char* at = (char*)ws;
    LinProduct<T> w{};
    w.C = dW;
    w.db = db;
    if (gated) {
        const LinGate g = lin_gate(rows, out, (int)sizeof(T));
        T* hi = (T*)at;
        at += g.bytes;
        T* rest = (T*)at;
        if (sizeof(T) == 2) at += g.bytes;
        w.db_part = (float*)at;
        w.db_parts = g.parts;
        at += g.db_bytes;
        lin_gate_kernel<T><<<dim3((unsigned)g.parts, (unsigned)g.cols), 256, 0, s>>>(
            pre, dY, hi, rest, rows, out, g.lg, LinAct{(int)act, slope}, db ? w.db_part : nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        D = hi;
        if (sizeof(T) == 2) lo = rest;
    }
    if (dX) {
        LinProduct<T> q{};
        q.C = dX;
        const hipError_t e = lin_run<T, T, true, true, LIN_PLAIN, false>(q, rows, in, out, D, out, W, nullptr, out, at, s);
        if (e != hipSuccess) return e;
    }
    if (gated) return lin_run<T, float, false, false, LIN_PLAIN, false>(w, in, out, rows, X, in, D, lo, out, at, s);
    return lin_run<T, float, false, false, LIN_PLAIN, true>(w, in, out, rows, X, in, D, nullptr, out, at, s);
}

template hipError_t launch_linear_fwd<float>(int64_t, int, int, const float*, const float*, const float*, cf_act, float,
                                             const float*, float*, float*, void*, hipStream_t);
template hipError_t launch_linear_fwd<uint16_t>(int64_t, int, int, const uint16_t*, const uint16_t*, const float*, cf_act,
                                                float, const uint16_t*, uint16_t*, uint16_t*, void*, hipStream_t);
template hipError_t launch_linear_bwd<float>(int64_t, int, int, const float*, const float*, const float*, const float*,
                                             cf_act, float, float*, float*, float*, void*, hipStream_t);
template hipError_t launch_linear_bwd<uint16_t>(int64_t, int, int, const uint16_t*, const uint16_t*, const uint16_t*,
                                                const uint16_t*, cf_act, float, uint16_t*, float*, float*, void*,
                                                hipStream_t);

}  // namespace cf
