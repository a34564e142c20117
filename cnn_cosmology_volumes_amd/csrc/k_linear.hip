// Linear layers over rows (a dense layer, or a 1^3 convolution over voxels):
//   pre = X W + bias,  Y = act(pre) + R            X [rows][in], W [in][out]
// and backward, with D = dY act'(pre):
//   dX = D W^T,  dW = X^T D,  db = column sums of D.
//
// Three products C [M][N] = sum_k A(m, k) B(k, n) (k_linear_mm.hip), whose operands
// lie along the reduction (X and D in the first two, W in W^T) or across it (W
// forward, both operands of dW); few rows have kernels of their own
// (k_linear_few.hip).  Here: what goes before and after a product, which tile and
// split it takes, and the calls.
#include "linear_common.h"

namespace cf {
namespace {

// a / b, b below 2^31: 64-bit division is some hundred instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int b)
{
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

size_t up256l(size_t b) { return (b + 255) & ~(size_t)255; }
int up_vec(int n, int size) { return (n + 16 / size - 1) / (16 / size) * (16 / size); }

// Adds the splits' sums, and in the blocks past `main` those of db, 16 columns a
// block and 16 threads to a column.  Results are taken as vectors of eight columns,
// 2^lg threads to each, which take every 2^lg-th split: the few results of a long
// reduction are bound by the latency of a thread's loads, so several of them are
// under way.
// (dW and db of 380581 x 2 x 1 bf16, 992 splits: 54 us with eight threads and a load
// at a time.)
union LinJoinShared {
    double col[16][17];
    float part[256][8];
};
template <typename T, typename TO, int MODE>
__device__ __forceinline__ void lin_join(const LinProduct<T>& q, int block, int main, int lg, LinJoinShared& sh)
{
    if (block >= main) {
        const int c = (block - main) * 16 + (int)threadIdx.x % 16, k = (int)threadIdx.x / 16;
        double sum = 0.0;
        if (c < q.N)
            for (int i = k; i < q.db_parts; i += 256) {
                float t[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int at = i + u * 16 < q.db_parts ? i + u * 16 : q.db_parts - 1;
                    t[u] = q.db_part[(int64_t)at * q.N + c];
                }
#pragma unroll
                for (int u = 0; u < 16; ++u) sum += i + u * 16 < q.db_parts ? (double)t[u] : 0.0;
            }
        sh.col[k][threadIdx.x % 16] = sum;
        __syncthreads();
        if (k == 0 && c < q.N) {
            for (int i = 1; i < 16; ++i) sum += sh.col[i][threadIdx.x];
            q.db[c] = (float)sum;
        }
        return;
    }
    const int groups = 1 << lg, each = 256 >> lg;
    const int vecs = (q.N + 7) / 8, mine = (int)threadIdx.x & (each - 1), group = (int)threadIdx.x >> (8 - lg);
    const int64_t total = q.M * vecs;
    for (int64_t i0 = (int64_t)block * each; i0 < total; i0 += (int64_t)main * each) {
        const int64_t i = i0 + mine, m = quotient(i, vecs);
        const int n = (int)(i - m * vecs) * 8;
        float v[8] = {};
        if (i < total) {
            const float* p = q.part + m * q.N + n;
            const int64_t step = q.M * q.N;
            const bool whole = q.N - n >= 8;
            for (int s = group; s < q.splits; s += 4 * groups) {
                Lin8<float> t[4] = {};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (s + u * groups >= q.splits) continue;
                    if (whole) t[u].load(p + (s + u * groups) * step);
                    else t[u].load(p + (s + u * groups) * step, q.N - n);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float w[8];
                    t[u].get(w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += w[j];
                }
            }
        }
        if (lg) {
            __syncthreads();
            __builtin_memcpy(sh.part[threadIdx.x], v, 32);
            __syncthreads();
            if (group) continue;
#pragma unroll 4
            for (int g = 1; g < groups; ++g)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += sh.part[g * each + mine][j];
        }
        if (i >= total) continue;
        float bias[8] = {};
        Lin8<T> res = {};
        if (MODE != LIN_PLAIN && q.bias) load8<false>(q.bias + n, q.N - n, bias);
        if (MODE == LIN_FWD_RES) {
            if (q.N - n >= 8) res.load(q.R + m * q.N + n);
            else res.load(q.R + m * q.N + n, q.N - n);
        }
        lin_result<false, T, TO, MODE>(q, m * q.N + n, n, v, bias, res);
    }
}

template <typename T, typename TO, int MODE>
__global__ __launch_bounds__(256) void lin_join_kernel(LinProduct<T> q, int main, int lg)
{
    __shared__ LinJoinShared sh;
    lin_join<T, TO, MODE>(q, (int)blockIdx.x, main, lg, sh);
}
// Those of dX in the first blocks, and of dW and db: a launch less.
template <typename T>
__global__ __launch_bounds__(256) void lin_join_bwd_kernel(LinProduct<T> x, int main_x, int lg_x, LinProduct<T> w, int main_w,
                                                           int lg_w)
{
    __shared__ LinJoinShared sh;
    if ((int)blockIdx.x < main_x) lin_join<T, T, LIN_PLAIN>(x, (int)blockIdx.x, main_x, lg_x, sh);
    else lin_join<T, float, LIN_PLAIN>(w, (int)blockIdx.x - main_x, main_w, lg_w, sh);
}

// Copies of matrices whose rows are not whole vectors, with rows that are: the
// products' loads take 16 bytes at multiples of 16.  (Reading such rows as they are,
// value by value at their ends and through registers, took 7429 x 333 x 1001 82 us
// in fp32 and 32 in bf16.)
struct LinPack {
    const void* from[3];
    void* to[3];
    int64_t vecs[3];        // of a copy
    int cols[3];
    int blocks[3];
};
template <typename T> __device__ __forceinline__ void lin_pack(const LinPack& q, int block)
{
    constexpr int V = LinTile<T>::V;
    int job = 0;
    while (block >= q.blocks[job]) block -= q.blocks[job++];
    const int cols = q.cols[job], each = (cols + V - 1) / V;
    const T* from = (const T*)q.from[job];
    for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < q.vecs[job]; i += (int64_t)q.blocks[job] * 256) {
        const int64_t r = quotient(i, each);
        const int c = (int)(i - r * each) * V;
        const uint4 v = lin_chunk<T>(from + r * cols + c, cols - c, cols >= V);
        __builtin_memcpy((T*)q.to[job] + i * V, &v, 16);
    }
}

// D = dY act'(pre) with rows of `ld` values: fp32, or as bf16 hi and lo = D - hi,
// which together keep 16 bits or more: dW is fp32 and would show the rounding of hi
// alone (2^-9 of every term), and dX, whose own rounding is no larger, would be off by
// 2.4e-3 for 1.7e-3.  A slope of 0 or a power of two leaves no lo (null).
// A block takes a range of rows, 2^lg lanes to a row, and leaves the column sums of D.
template <typename T> struct LinGated {
    const T *pre, *dY;
    T *hi, *lo;
    int64_t rows;
    int N, ld, lg, parts, blocks;
    LinAct act;
    float* db_part;
};
template <typename T> __device__ __forceinline__ void lin_gate_rows(const LinGated<T>& q, int block)
{
    constexpr int V = LinTile<T>::V;
    __shared__ float sh[256 * V];
    const int part = block % q.parts, column = block / q.parts;
    const int lane = (int)threadIdx.x & ((1 << q.lg) - 1), c = ((column << q.lg) + lane) * V;
    const int64_t r0 = q.rows * part / q.parts, r1 = q.rows * (part + 1) / q.parts;
    float sum[V] = {};
    if (c < q.N)
        for (int64_t r = r0 + ((int)threadIdx.x >> q.lg); r < r1; r += 256 >> q.lg) {
            const uint4 zv = lin_chunk<T>(q.pre + r * q.N + c, q.N - c, q.N >= V);
            const uint4 dv = lin_chunk<T>(q.dY + r * q.N + c, q.N - c, q.N >= V);
            T z[V], d[V], h[V], l[V];
            __builtin_memcpy(z, &zv, 16);
            __builtin_memcpy(d, &dv, 16);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = widen(d[j]) * lin_dact<T>(q.act, widen(z[j]));
                sum[j] += v;
                Elem<T>::store(h, j, v);
                // (an infinite hi stands for itself: inf - inf would make NaN of it)
                const float rest = v - widen(h[j]);
                if (sizeof(T) == 2) Elem<T>::store(l, j, __builtin_isfinite(widen(h[j])) ? rest : 0.f);
            }
            __builtin_memcpy(q.hi + r * q.ld + c, h, 16);
            if (sizeof(T) == 2 && q.lo) __builtin_memcpy(q.lo + r * q.ld + c, l, 16);
        }
    if (!q.db_part) return;
#pragma unroll
    for (int j = 0; j < V; ++j) sh[j * 256 + (int)threadIdx.x] = sum[j];
    __syncthreads();
    // sum j of the lanes of one column lies at j 256 + lane, 2^lg apart
    for (int i = (int)threadIdx.x; i < V << q.lg; i += 256) {
        const int j = i >> q.lg, k = i & ((1 << q.lg) - 1), col = ((column << q.lg) + k) * V + j;
        if (col >= q.N) continue;
        float v = 0.f;
        for (int g = 0; g < 256 >> q.lg; ++g) v += sh[j * 256 + (g << q.lg) + k];
        q.db_part[(int64_t)part * q.N + col] = v;
    }
}

// What a product needs beforehand: D, if there is an activation, and the copies.
template <typename T> __global__ __launch_bounds__(256) void lin_before_kernel(LinGated<T> g, LinPack p)
{
    if ((int)blockIdx.x < g.blocks) lin_gate_rows<T>(g, (int)blockIdx.x);
    else lin_pack<T>(p, (int)blockIdx.x - g.blocks);
}

// Lanes of a row (log2), columns of blocks and parts of the rows of lin_gate_rows.
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
    const int64_t most = (1024 + g.cols - 1) / g.cols, each = 256 >> g.lg, want = (rows + each - 1) / each;
    g.parts = (int)(want < most ? want : most);
    g.bytes = up256l((size_t)rows * up_vec(N, size) * size);
    g.db_bytes = up256l((size_t)g.parts * N * 4);
    return g;
}

// Tile and splits of a product by estimated time, in us: a block's pieces of the
// reduction and what it does besides (first loads, results), in as many rounds as the
// blocks that the chip holds at once leave, and the joining of splits (their bytes at
// 4.5 TB/s, a launch).  Fitted to these, tiles of 64 x 64 / 128 x 128 / 256 x 128 / 256 x 256:
//   bf16  32768 x 2048 x 2048 - / 352 / 307 / 264 us   32768 x 512 x 1024 81 / 54 / 49 / 52
//         262144 x 128 x 512 223 / 166 / 144 / 135     8192 x 1024 x 1024 38 / 27 / 26 / 33
//         262144 x 64 x 64 23 / 33 / - / -
//         dW of 32768 x 512 x 1024 in two parts, 8 / 8 / 16 / 32 splits: - / 103 / 94 / 92
//   fp32  32768 x 2048 x 2048 2158 / 2005 / 1929 us    4096 x 2048 x 2048 276 / 257 / 255
//         40102 x 128 x 1456 218 / 205 / 205           8192 x 1024 x 1024 148 / 135 / 136
//         416890 x 32 x 176 191 / 191 / 185            16640 x 512 x 256 52 / 72 / 84
//         262144 x 64 x 64 45 / 74 / 71                7429 x 333 x 1001 65 / 66 / 69
//         3000 x 1500 x 1500 134 / 190 / -             32768 x 1024 x 128 90 / 81 / -
//         dW of 32768 x 512 x 1024, 8 / 16 / 16 splits: 342 / 339 / 340, with db 392 / 374 / -
//         with residuals 40102 x 128 x 1456 234 / 244 / 286, 65536 x 256 x 256 94 / 91 / 98
// In fp32 a piece is bound by the matrix cores, so that the CU with the most blocks
// counts; in bf16 by its loads, and the chip's mean does.  256 x 256 is for bf16: in
// fp32 it was not ahead by 2% anywhere (32768 x 2048 x 2048 1953, 8192 x 1024 x 1024
// 158).  Over 40 fp32 sizes, these among them, the tile taken is 2% slower than the
// fastest one by geometric mean, 14% at most (5000 x 1024 x 1024 dW with db).
// sums: with db, whose sums take the registers that the largest tiles would need, and
// matrix instructions of their own.  residual: fp32 residuals on their way take
// registers too (of tiles of 256 x 128 some go through scratch memory).
LinPlan lin_plan(int64_t M, int N, int64_t K, int size, int passes, bool sums, bool residual)
{
    struct Tile {
        int tm, tn, slots;
        double alone;                    // bf16: a piece's time where a CU has a block for itself, of that with its full share
        double crowd[5];                 // fp32: a piece's time with so many blocks on a CU, of that with all
        double piece[2], rest[2];        // bf16, fp32
        double sums, residual;           // fp32: a piece with db's sums, of that without; more for residuals
    };
    static const Tile tiles[4] = {{64, 64, 1280, 0.4, {0.28, 0.43, 0.7, 0.95, 1.0}, {0.61, 1.27}, {5.5, 9.0}, 1.25, 1.5},
                                  {128, 128, 512, 0.5, {0.53, 1.0}, {0.64, 1.92}, {6.5, 12.0}, 1.1, 5.0},
                                  {256, 128, 512, 0.5, {0.53, 1.0}, {1.09, 3.62}, {10.5, 22.0}, 1.0, 20.0},
                                  {256, 256, 256, 1.0, {}, {0.85, 0.0}, {11.0, 0.0}, 1.0, 0.0}};
    const int bk = LIN_PIECE / size, kb = (int)((K + bk - 1) / bk), f32 = size == 4;
    const int64_t total = (int64_t)kb * passes;
    LinPlan best{};
    double least = 0.0;
    for (const Tile& t : tiles) {
        if ((sums && t.tm == 256) || (f32 && t.tn == 256)) break;
        const int64_t tm = (M + t.tm - 1) / t.tm;
        const int tn = (N + t.tn - 1) / t.tn;
        for (int64_t want = 1; want <= 1024 && (want == 1 || total / want >= 4); want *= 2) {
            const int64_t each = (total + want - 1) / want, splits = (total + each - 1) / each, units = tm * tn * splits;
            const double full = (double)units / t.slots;
            double share = full >= 1.0 ? 1.0 : full > t.alone ? full : t.alone;
            if (f32 && full < 1.0) share = t.crowd[(units - 1) / 256];
            // (many small blocks: one begins as another ends)
            const double rounds = full <= 1.0  ? 1.0
                                  : t.tm == 64 ? full + (f32 ? 0.0 : 0.5)
                                               : (double)((units + t.slots - 1) / t.slots);
            const double piece = t.piece[f32] * share * (f32 && sums ? t.sums : 1.0);
            double us = rounds * (each * piece + t.rest[f32] + (f32 && residual ? t.residual : 0.0));
            if (splits > 1) us += 4.0 + (double)M * N * 8.0 * splits / 4.5e6;
            if (!best.tm || us < least) {
                least = us;
                best = LinPlan{t.tm, t.tn, tm, tn, kb, (int)each, (int)splits, 0, 0};
            }
            if (full > 4.0) break;
        }
    }
    if (best.splits > 1) {
        best.part_bytes = up256l((size_t)best.splits * (size_t)M * N * 4);
        best.db_bytes = up256l((size_t)best.splits * N * 4);
    }
    return best;
}

// A product whose sums, or whose db, are still to be joined: blocks of the join for the
// sums and of all, threads to a vector (log2).
template <typename T> struct LinJoin {
    LinProduct<T> q{};
    int main = 0, all = 0, lg = 0;
};

// The product over K (and then over K again, of A2 and B2, if there are), and what is
// to be joined after it.  DB: q.db is formed with it; else q.db_part already holds its parts, if
// q.db is not null.
template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t lin_run(LinJoin<T>& join, int64_t M, int N, int64_t K, const T* A, const T* A2, int64_t lda, const T* B,
                   const T* B2, int64_t ldb, void* ws, hipStream_t s)
{
    // (a dX in two passes takes the tiles and the number of splits of one)
    LinPlan p = lin_plan(M, N, K, (int)sizeof(T), B2 ? 2 : 1, DB, MODE == LIN_FWD_RES);
    if (A2) p.kb_split *= 2;
    LinProduct<T>& q = join.q;
    q.A = A;
    q.B = B;
    q.A2 = A2 ? A2 : A;
    q.B2 = B2 ? B2 : B;
    q.passes = A2 || B2 ? 2 : 1;
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
    if (p.splits >= 16)
        for (join.lg = 3; join.lg < 6 && 4 << join.lg < p.splits;) ++join.lg;
    const int64_t vecs = p.splits > 1 ? M * ((N + 7) / 8) : 0, blocks = (vecs + (255 >> join.lg)) >> (8 - join.lg);
    join.main = (int)(blocks < 4096 ? blocks : 4096);
    join.all = join.main + (q.db && (!DB || p.splits > 1) ? (N + 15) / 16 : 0);
    return launch_lin_mm<T, TO, AA, BA, MODE, DB>(p, q, s);
}

template <typename T, typename TO, int MODE> hipError_t run_join(const LinJoin<T>& j, hipStream_t s)
{
    if (!j.all) return hipSuccess;
    lin_join_kernel<T, TO, MODE><<<(unsigned)j.all, 256, 0, s>>>(j.q, j.main, j.lg);
    return hipGetLastError();
}
template <typename T> hipError_t run_join_bwd(const LinJoin<T>& x, const LinJoin<T>& w, hipStream_t s)
{
    if (!x.all) return run_join<T, float, LIN_PLAIN>(w, s);
    if (!w.all) return run_join<T, T, LIN_PLAIN>(x, s);
    lin_join_bwd_kernel<T><<<(unsigned)(x.all + w.all), 256, 0, s>>>(x.q, x.main, x.lg, w.q, w.main, w.lg);
    return hipGetLastError();
}

// Takes copies of matrices in turn from the workspace.
template <typename T> struct LinCopies {
    LinPack pack{};
    int count = 0, blocks = 0;
    char* at;
    // The matrix, or where its copy will be.
    const T* take(const T* m, int64_t rows, int cols)
    {
        const int ld = up_vec(cols, (int)sizeof(T));
        if (ld == cols) return m;
        const int64_t vecs = rows * (ld * (int)sizeof(T) / 16), want = (vecs + 255) / 256;
        pack.from[count] = m;
        pack.to[count] = at;
        pack.vecs[count] = vecs;
        pack.cols[count] = cols;
        blocks += pack.blocks[count++] = (int)(want < 8192 ? want : 8192);
        T* to = (T*)at;
        at += up256l((size_t)vecs * 16);
        return to;
    }
    hipError_t run(const LinGated<T>& g, hipStream_t s)
    {
        if (!g.blocks && !blocks) return hipSuccess;
        lin_before_kernel<T><<<(unsigned)(g.blocks + blocks), 256, 0, s>>>(g, pack);
        return hipGetLastError();
    }
};
size_t copy_bytes(int64_t rows, int cols, int size)
{
    const int ld = up_vec(cols, size);
    return ld == cols ? 0 : up256l((size_t)rows * ld * size);
}

// Whether the forward of few rows is one launch of lin_few_fwd_kernel: its blocks
// take a whole reduction each, which is too long for long rows of X.  One launch / a
// product, in us, captured into a graph (a call by itself takes 10 and 15 at least):
//   1 row, bf16    2048 x 1024  6.4 / 7.8   4096 x 2048 11.2 / 10.6  8192 x 2048 19 / 13  65536 x 1024 199 / 34
//   8 rows, fp32   2048 x 256     9 / 11    4096 x 1024 14.5 / 13.8  8192 x 1024 25 / 18  65536 x 512 242 / 48
// Rows of W that are not whole vectors would be copied for the product; up to 4
// rows of X and where its columns leave blocks enough, the launch goes on for less:
//   1 row, bf16    8192 x 1537    20 / 27    16384 x 2047  54 / 42   16384 x 4095  62 / 75
//   1 row, fp32    8192 x 515     19 / 29    16384 x 1537  53 / 73   65536 x 2047 229 / 336
//   8 rows, fp32   8192 x 515     52 / 28    16384 x 2047 130 / 87
bool lin_few_fwd(int64_t rows, int in, int out, int size)
{
    if (rows > LIN_FEW) return false;
    return in <= 4096 || (rows <= 4 && out * size % 16 && out * size >= (in <= 8192 ? 1024 : 6144));
}
// And the backward: a block takes 8 or 16 rows of W over all columns, which is too
// long where there are few rows of W and many columns; very many rows of W leave each
// block little beside its own start.  One launch / products, in us, captured into a
// graph (a call by itself takes 10 and 20 at least):
//   1 row, bf16    2048 x 1024  9.2 / 17   1024 x 4096 24 / 24   512 x 16384 79 / 29   16 x 65536 319 / 22
//   8 rows, fp32   2047 x 2047   20 / 30   1024 x 4096 31 / 26   512 x 16384 106 / 33  16 x 65536 422 / 26
//   8 rows         bf16 4096 x 16384 121 / 125, 65536 x 128 68 / 26; fp32 3001 x 4097 35 / 58, 65536 x 512 ahead
// More than 8 rows have longer sums, and their products are no longer:
//   16 rows        bf16 2048 x 1024 11 / 17, 4096 x 4096 67 / 39, 16384 x 128 41 / 15; fp32 1024 x 2048 28 / 19
bool lin_few_bwd(int64_t rows, int in, int out, int size)
{
    if (rows > LIN_FEW) return false;
    if (rows > 8) return in <= 4096 && out * size <= 4096 && (int64_t)in * out <= 1 << 22;
    return (out <= 2048 || 4 * in >= out) && (in <= 16384 || (size == 4 && out >= 512));
}

bool lin_gated(cf_act act, float slope) { return act == CF_ACT_SILU || slope != 1.f; }

}  // namespace

size_t linear_ws_bytes(cf_dtype dt, int64_t rows, int in, int out, bool bwd)
{
    const int size = dt == CF_F32 ? 4 : 2;
    if (bwd ? lin_few_bwd(rows, in, out, size) : lin_few_fwd(rows, in, out, size)) return 0;
    const size_t copies = copy_bytes(rows, in, size) + copy_bytes(in, out, size);
    if (!bwd) {
        const size_t with = lin_plan(rows, out, in, size, 1, false, true).part_bytes,
                     without = lin_plan(rows, out, in, size, 1, false, false).part_bytes;
        return copies + (with > without ? with : without);
    }
    const LinGate g = lin_gate(rows, out, size);
    const LinPlan x = lin_plan(rows, in, out, size, 1, false, false),
                  w = lin_plan(in, out, rows, size, size == 2 ? 2 : 1, false, false),
                  one = lin_plan(in, out, rows, size, 1, true, false);
    const LinPlan exact = lin_plan(in, out, rows, size, 1, false, false);
    const size_t parts = w.part_bytes > exact.part_bytes ? w.part_bytes : exact.part_bytes;
    const size_t gated = g.bytes * (size == 2 ? 2 : 1) + g.db_bytes + parts;
    const size_t plain = copy_bytes(rows, out, size) + one.part_bytes + one.db_bytes;
    return copies + x.part_bytes + (gated > plain ? gated : plain);
}

// product 0: forward, 1: dX, 2: dW without an activation, 3: dW with D in one part, 4: with D in two, 5: forward with
// a residual
LinTiles linear_tiles(cf_dtype dt, int64_t rows, int in, int out, int product)
{
    const int size = dt == CF_F32 ? 4 : 2;
    const bool forward = product == 0 || product == 5;
    if (forward ? lin_few_fwd(rows, in, out, size) : lin_few_bwd(rows, in, out, size)) return LinTiles{0, 0, 0};
    const LinPlan p = forward        ? lin_plan(rows, out, in, size, 1, false, product == 5)
                      : product == 1 ? lin_plan(rows, in, out, size, 1, false, false)
                                     : lin_plan(in, out, rows, size, product == 4 && size == 2 ? 2 : 1, product == 2, false);
    return LinTiles{p.tm, p.tn, p.splits};
}

template <typename T>
hipError_t launch_linear_fwd(int64_t rows, int in, int out, const T* X, const T* W, const float* bias, cf_act act,
                             float slope, const T* R, T* pre, T* Y, void* ws, hipStream_t s)
{
    LinJoin<T> y;
    LinProduct<T>& q = y.q;
    q.C = Y;
    q.bias = bias;
    q.R = R;
    q.pre = pre;
    q.act = LinAct{(int)act, slope};
    if (lin_few_fwd(rows, in, out, (int)sizeof(T))) {
        q.A = X;
        q.B = W;
        q.M = rows;
        q.N = out;
        q.K = in;
        return launch_lin_few_fwd(q, s);
    }
    LinCopies<T> copies;
    copies.at = (char*)ws;
    X = copies.take(X, rows, in);
    W = copies.take(W, in, out);
    hipError_t e = copies.run(LinGated<T>{}, s);
    if (e != hipSuccess) return e;
    const int ldi = up_vec(in, sizeof(T)), ldo = up_vec(out, sizeof(T));
    if (R) {
        e = lin_run<T, T, true, false, LIN_FWD_RES, false>(y, rows, out, in, X, nullptr, ldi, W, nullptr, ldo, copies.at, s);
        return e != hipSuccess ? e : run_join<T, T, LIN_FWD_RES>(y, s);
    }
    e = lin_run<T, T, true, false, LIN_FWD, false>(y, rows, out, in, X, nullptr, ldi, W, nullptr, ldo, copies.at, s);
    return e != hipSuccess ? e : run_join<T, T, LIN_FWD>(y, s);
}

template <typename T>
hipError_t launch_linear_bwd(int64_t rows, int in, int out, const T* X, const T* W, const T* pre, const T* dY,
                             cf_act act, float slope, T* dX, float* dW, float* db, void* ws, hipStream_t s)
{
    const bool gated = lin_gated(act, slope);
    const LinAct a = {(int)act, slope};
    if (lin_few_bwd(rows, in, out, (int)sizeof(T)))
        return launch_lin_few_bwd((int)rows, in, out, X, W, pre, dY, a, gated, dX, dW, db, s);
    const int ldi = up_vec(in, sizeof(T)), ldo = up_vec(out, sizeof(T));
    LinCopies<T> copies;
    copies.at = (char*)ws;
    X = copies.take(X, rows, in);
    if (dX) W = copies.take(W, in, out);
    const T* D = gated ? nullptr : copies.take(dY, rows, out);
    const T* lo = nullptr;
    char* at = copies.at;
    LinJoin<T> x, w;
    x.q.C = dX;
    w.q.C = dW;
    w.q.db = db;
    LinGated<T> gate{};
    if (gated) {
        // (dY times 0 or a power of two is a bf16 value itself)
        int exponent;
        const bool exact = act == CF_ACT_LRELU && (slope == 0.f || frexpf(slope, &exponent) == 0.5f);
        const LinGate g = lin_gate(rows, out, (int)sizeof(T));
        T* hi = (T*)at;
        at += g.bytes;
        T* rest = nullptr;
        if (sizeof(T) == 2 && !exact) {
            rest = (T*)at;
            at += g.bytes;
        }
        w.q.db_part = (float*)at;
        w.q.db_parts = g.parts;
        at += g.db_bytes;
        gate = LinGated<T>{pre, dY, hi, rest, rows, out, ldo, g.lg, g.parts, g.parts * g.cols, a, db ? w.q.db_part : nullptr};
        D = hi;
        lo = rest;
    }
    hipError_t e = copies.run(gate, s);
    if (e != hipSuccess) return e;
    if (dX) {
        e = lin_run<T, T, true, true, LIN_PLAIN, false>(x, rows, in, out, D, lo, ldo, W, nullptr, ldo, at, s);
        if (e != hipSuccess) return e;
        if (x.q.splits > 1) at += up256l((size_t)x.q.splits * (size_t)rows * in * 4);
    }
    e = gated ? lin_run<T, float, false, false, LIN_PLAIN, false>(w, in, out, rows, X, nullptr, ldi, D, lo, ldo, at, s)
              : lin_run<T, float, false, false, LIN_PLAIN, true>(w, in, out, rows, X, nullptr, ldi, D, nullptr, ldo, at, s);
    return e != hipSuccess ? e : run_join_bwd(x, w, s);
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
