// Linear layers over rows (a dense layer, or a 1^3 convolution over voxels):
//   pre = X W + bias,  Y = act(pre) + R            X [rows][in], W [in][out]
// and backward, with D = dY act'(pre):
//   dX = D W^T,  dW = X^T D,  db = column sums of D.
//
// One product kernel serves all three, C [M][N] = sum_k A(m, k) B(k, n), for
// operands whose values lie along k (X and D in the first two, W in W^T) or
// across it (W forward, both operands of dW).
#include "linear_common.h"

namespace cf {
namespace {

constexpr int LIN_T = 256;

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

// TILE x TILE of the result a block, four waves of TILE/2 x TILE/2.
template <typename T, typename TO, bool AA, bool BA, int TILE, int MODE, bool DB>
__global__ __launch_bounds__(LIN_T) void lin_product_kernel(LinProduct<T> q)
{
    using OA = LinOperand<T, AA, TILE>;
    using OB = LinOperand<T, BA, TILE>;
    constexpr int BK = LinTile<T>::BK, STEPS = BK / (sizeof(T) == 2 ? 16 : 8), B = TILE / 64;
    constexpr int STAGE = (OA::SIZE + OB::SIZE) * (int)sizeof(T), OUT = 4 * 32 * (32 * B + 4) * 4;
    __shared__ __attribute__((aligned(16))) char raw[STAGE > OUT ? STAGE : OUT];
    T* const sa = (T*)raw;
    T* const sb = sa + OA::SIZE;
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
        if (DB && sums && lane < 32 && q.db)
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int n = j0 + wj + j * 32 + lane;
                if (n >= q.N) continue;
                if (q.splits > 1) q.db_part[(int64_t)split * q.N + n] = col[j][0];
                else q.db[n] = col[j][0];
            }
        const int n = j0 + wj + lane % (4 * B) * 8;
        float bias[8] = {};
        if (MODE == LIN_FWD && q.bias && n < q.N) load8(q.bias + n, q.N - n, bias);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < B; ++i)
            lin_rows<T, TO, MODE, B>(acc[i], (float*)raw + wave * 32 * (32 * B + 4), q, split, i0 + wi + i * 32, j0 + wj, bias);
        __syncthreads();
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
    const int vecs = (q.N + 7) / 8;
    const int64_t total = q.M * vecs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)main * 256) {
        const int64_t m = i / vecs;
        const int n = (int)(i - m * vecs) * 8;
        float v[8] = {}, bias[8] = {}, res[8] = {};
        if (MODE == LIN_FWD && q.bias) load8(q.bias + n, q.N - n, bias);
        if (MODE == LIN_FWD && q.R) load8(q.R + m * q.N + n, q.N - n, res);
#pragma unroll 4
        for (int s = 0; s < q.splits; ++s) {
            float p[8];
            load8(q.part + (s * q.M + m) * q.N + n, q.N - n, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += p[j];
        }
        lin_result<T, TO, MODE>(q, m, n, v, bias, res);
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

// Whether all rows of X, W, D and their gradients start at multiples of 16 bytes.
bool lin_aligned(int in, int out, int size) { return in * size % 16 == 0 && out * size % 16 == 0; }

size_t up256l(size_t b) { return (b + 255) & ~(size_t)255; }

LinPlan lin_plan(int64_t M, int N, int64_t K, int size, int passes, bool aligned)
{
    LinPlan p;
    p.aligned = aligned;
    const int bk = size == 2 ? 64 : 32;
    const int64_t t128 = (M + 127) / 128 * ((N + 127) / 128);
    p.tile = t128 >= 256 ? 128 : 64;
    if (aligned && M >= 4096 && N >= 512 && K >= 512) p.tile = 256;
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
                   int64_t ldb, bool aligned, void* ws, hipStream_t s)
{
    const LinPlan p = lin_plan(M, N, K, (int)sizeof(T), B2 ? 2 : 1, aligned);
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
    hipError_t e;
    if (p.aligned) {
        e = launch_lin_mm<T, TO, AA, BA, MODE, DB>(p, q, s);
    } else {
        if (p.tile == 128) lin_product_kernel<T, TO, AA, BA, 128, MODE, DB><<<grid, LIN_T, 0, s>>>(q);
        else lin_product_kernel<T, TO, AA, BA, 64, MODE, DB><<<grid, LIN_T, 0, s>>>(q);
        e = hipGetLastError();
    }
    const bool join_db = q.db && (!DB || p.splits > 1);
    if (e != hipSuccess || (p.splits == 1 && !join_db)) return e;
    const int64_t blocks = p.splits > 1 ? (M * ((N + 7) / 8) + 255) / 256 : 0;
    const int main = (int)(blocks < 4096 ? blocks : 4096);
    lin_join_kernel<T, TO, MODE><<<(unsigned)(main + (join_db ? (N + 15) / 16 : 0)), 256, 0, s>>>(q, main);
    return hipGetLastError();
}

}  // namespace

size_t linear_ws_bytes(cf_dtype dt, int64_t rows, int in, int out, bool bwd)
{
    const int size = dt == CF_F32 ? 4 : 2;
    const bool al = lin_aligned(in, out, size);
    if (!bwd) return lin_plan(rows, out, in, size, 1, al).part_bytes;
    const LinGate g = lin_gate(rows, out, size);
    const LinPlan x = lin_plan(rows, in, out, size, 1, al),
                  w = lin_plan(in, out, rows, size, size == 2 ? 2 : 1, al), one = lin_plan(in, out, rows, size, 1, al);
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
    return lin_run<T, T, true, false, LIN_FWD, false>(q, rows, out, in, X, in, W, nullptr, out,
                                                 lin_aligned(in, out, sizeof(T)), ws, s);
}

template <typename T>
hipError_t launch_linear_bwd(int64_t rows, int in, int out, const T* X, const T* W, const T* pre, const T* dY,
                             cf_act act, float slope, T* dX, float* dW, float* db, void* ws, hipStream_t s)
{
    const bool gated = act == CF_ACT_SILU || slope != 1.f, al = lin_aligned(in, out, sizeof(T));
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
        const hipError_t e = lin_run<T, T, true, true, LIN_PLAIN, false>(q, rows, in, out, D, out, W, nullptr, out,
                                                                              al, at, s);
        if (e != hipSuccess) return e;
    }
    if (gated) return lin_run<T, float, false, false, LIN_PLAIN, false>(w, in, out, rows, X, in, D, lo, out, al, at, s);
    return lin_run<T, float, false, false, LIN_PLAIN, true>(w, in, out, rows, X, in, D, nullptr, out, al, at, s);
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
