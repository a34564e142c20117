// Newton-Schulz orthogonalisation of weight-shaped matrices and Muon's update
// with it.
//
// With X0 = U / (|U|_F + eps), m <= n its short and long side (a tall matrix
// is handled as its transpose), each of `steps` iterations is
//   A = X X^T,  X <- (a I + b A + c A^2) X.
// Every factor P_k = a I + b A_k + c A_k^2 is a polynomial in A_0, so they
// commute and the iteration runs on the short side alone:
//   A_0 = s^2 U U^T (s = 1 / (|U|_F + eps), |U|_F^2 = trace U U^T)
//   Q <- P_k Q,  A_{k+1} = P_k A_k P_k,   result = s Q U.
// The long side is read once for U U^T and once for Q U, in place of twice a
// step, and all products between are m x m and symmetric (only tiles on or
// above the diagonal are computed).
//
// Squaring the singular values costs half the digits of the small ones, and
// five steps raise them by up to a^5 = 485: with an fp32 U U^T the result of a
// square matrix is 30 times further from the exact one than fp32 products of
// X are.  U U^T and the m x m products therefore run on the fp64 matrix cores
// (products of fp32 values are exact in fp64); the result is then closer to
// the exact one than fp32 products of X.  Only the last product, s Q U, is
// fp32, as products of three bf16 parts.
//
// An eigenvalue of A_0 that should be 0 comes out as about +-2^-53 and grows by
// a^2 a step.  While it stays below 2^-24 (8 steps of a = 3.4445) it is no more
// than fp32's rounding.  With more steps it would come to matter, and a
// negative one would run away, since a + b t + c t^2 draws only positive ones
// back.  Such calls (ns_many) take A_0 + 2^-48 trace(A_0) I in place of A_0,
// which is what singular values of 2^-24 |X0|, fp32's rounding of X0, would
// add: no eigenvalue is negative then, and each ends where the polynomial's
// range ends.  Q holds factors of up to 2^24 beside those of 1 then, so s Q U
// is an fp64 product there too.  (128 x 4096 of rank 8, 20 steps: singular
// values up to 1.134, where X's own steps give them; without this, NaN.)
//
// Launches take a list of matrices; partial sums are added in a fixed order
// and there are no atomics: results are reproducible bit for bit.
//
// What bounds it: the chain of launches.  256 x 256 takes 111 us in 17 of them
// (a launch of this kind takes about 5 us with almost no work), the eight
// matrices of the 128^3 benchmark network 196 to 205 us: momentum 15, U U^T 32
// (fp64 matrix cores), its join 10, 14 rounds of 8, s Q U 32.  Shorter sides up to
// 64 iterate in one block instead (108 x 32: 21 us, 70 by rounds), and large
// matrices whose long side is not much longer take split products of X
// (k_ns_split.hip).
#include "cf_internal.h"

#include <algorithm>
#include <climits>
#include <cmath>

namespace cf {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int NS_T = 256;       // threads per block, 4 waves
constexpr int NS_TILE = 64;     // edge of an output tile of U U^T and of Q U
constexpr int NS_K = 32;        // reduction depth of a staged panel
constexpr int NS_SP = NS_TILE + 16;   // LDS row stride of a [k][64] panel: its 4 k rows x 16 columns of a
                                      // matrix-core operand fall on 64 different banks
constexpr int NS_SK = NS_K + 1;       // LDS row stride of a [64][k] panel

int up(int v, int m) { return (v + m - 1) / m * m; }
size_t up256b(size_t b) { return (b + 255) & ~(size_t)255; }

// First blocks of a launch's matrices; past the last one, past any block.
struct Starts {
    int at[CF_MAX_OPT_TENSORS];
    void set(int i, int first) { at[i] = first; }
    void clear()
    {
        for (int& v : at) v = INT_MAX;
    }
};
// The matrix whose range of blocks holds block b: every entry is read at once,
// a search would wait for one load after another.
__device__ __forceinline__ int find(const Starts& s, int b)
{
    int i = 0;
#pragma unroll
    for (int k = 1; k < CF_MAX_OPT_TENSORS; ++k) i += b >= s.at[k] ? 1 : 0;
    return i;
}

__device__ __forceinline__ float elem(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float elem(const uint16_t* p, int64_t i) { return bf2f(p[i]); }

// Tile pair index p >= 0 of the upper triangle, row by row: (ti, tj), ti <= tj < nt.
__device__ __forceinline__ void tile_pair(int p, int nt, int& ti, int& tj)
{
    ti = 0;
    while (p >= nt - ti) {
        p -= nt - ti;
        ++ti;
    }
    tj = ti + p;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Sum over the block in a fixed order, returned in every thread.
__device__ __forceinline__ double block_sum(double v, double* sh)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((sh[0] + sh[1]) + sh[2]) + sh[3];
}

// --------------------------------------------------------------------- U U^T
// One 64-row panel of NS_K values of the reduction.  TALL: U is [long][short]
// and the panel is stored [k][64]; otherwise U is [short][long], stored
// [64][k].  Rows and reduction indices outside the matrix read as zero.
constexpr int NS_PV = NS_TILE * NS_K / NS_T;     // values per thread

template <bool TALL, typename T>
__device__ __forceinline__ void panel_load(float (&v)[NS_PV], const T* U, int m, int n, int i0, int k0, int k1)
{
    const int t = (int)threadIdx.x;
#pragma unroll
    for (int r = 0; r < NS_PV; ++r) {
        const int i = i0 + (TALL ? t % NS_TILE : t / NS_K + r * (NS_T / NS_K));
        const int k = k0 + (TALL ? t / NS_TILE + r * (NS_T / NS_TILE) : t % NS_K);
        v[r] = i < m && k < k1 ? elem(U, TALL ? (int64_t)k * m + i : (int64_t)i * n + k) : 0.f;
    }
}
template <bool TALL> __device__ __forceinline__ void panel_store(const float (&v)[NS_PV], float* sh)
{
    const int t = (int)threadIdx.x;
#pragma unroll
    for (int r = 0; r < NS_PV; ++r) {
        if (TALL) sh[(t / NS_TILE + r * (NS_T / NS_TILE)) * NS_SP + t % NS_TILE] = v[r];
        else sh[(t / NS_K + r * (NS_T / NS_K)) * NS_SK + t % NS_K] = v[r];
    }
}
constexpr int NS_PANEL = NS_K * NS_SP > NS_TILE * NS_SK ? NS_K * NS_SP : NS_TILE * NS_SK;

struct GramArgs {
    Starts start;
    const void* u[CF_MAX_OPT_TENSORS];
    int m[CF_MAX_OPT_TENSORS], n[CF_MAX_OPT_TENSORS];
    int kc[CF_MAX_OPT_TENSORS];               // reduction indices per split
    int splits[CF_MAX_OPT_TENSORS];
    uint32_t tall;                            // bit per matrix
    int64_t part[CF_MAX_OPT_TENSORS];         // doubles from the workspace's start
};

// Block = (split, tile pair): its part of U U^T in fp64, and for a tile on the
// diagonal its part of the trace.  part: [split][pair][64][64], then
// [split][diagonal tile].  Four waves, each a 32 x 32 quadrant.
template <bool TALL, typename T>
__device__ void gram_tile(const T* U, int m, int n, int kc, int splits, int b, double* part, float* sh, double* red)
{
    const int nt = (m + NS_TILE - 1) / NS_TILE, pairs = nt * (nt + 1) / 2;
    const int split = b / pairs, p = b % pairs;
    int ti, tj;
    tile_pair(p, nt, ti, tj);
    const int i0 = ti * NS_TILE, j0 = tj * NS_TILE;
    const int k0 = split * kc, k1 = min(k0 + kc, n);
    float* A = sh;
    float* B = ti == tj ? sh : sh + NS_PANEL;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
    const bool idle = ti == tj && wi > wj;       // the mirror of quadrant (0, 1)
    f64x4 acc[2][2] = {};
    float va[NS_PV], vb[NS_PV];
    panel_load<TALL>(va, U, m, n, i0, k0, k1);
    if (ti != tj) panel_load<TALL>(vb, U, m, n, j0, k0, k1);
    for (int k = k0; k < k1; k += NS_K) {
        __syncthreads();
        panel_store<TALL>(va, A);
        if (ti != tj) panel_store<TALL>(vb, B);
        __syncthreads();
        if (k + NS_K < k1) {
            panel_load<TALL>(va, U, m, n, i0, k + NS_K, k1);
            if (ti != tj) panel_load<TALL>(vb, U, m, n, j0, k + NS_K, k1);
        }
        if (idle) continue;
#pragma unroll
        for (int s = 0; s < NS_K / 4; ++s) {
            double a[2], c[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int kk = s * 4 + lane / 16, i = wi + q * 16 + lane % 16, j = wj + q * 16 + lane % 16;
                a[q] = (double)A[TALL ? kk * NS_SP + i : i * NS_SK + kk];
                c[q] = (double)B[TALL ? kk * NS_SP + j : j * NS_SK + kk];
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    acc[q][r] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[q], c[r], acc[q][r], 0, 0, 0);
        }
    }
    // element v of a lane's four: row 4 v + lane / 16, column lane % 16
    double* out = part + ((int64_t)split * pairs + p) * (NS_TILE * NS_TILE);
    double tr = 0.0;
    if (!idle)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int i = wi + q * 16 + 4 * v + lane / 16, j = wj + r * 16 + lane % 16;
                    out[i * NS_TILE + j] = acc[q][r][v];
                    if (ti == tj && i == j) tr += acc[q][r][v];
                }
    if (ti == tj) {
        tr = block_sum(tr, red);
        if (threadIdx.x == 0) part[(int64_t)splits * pairs * (NS_TILE * NS_TILE) + split * nt + ti] = tr;
    }
}

template <typename T> __global__ __launch_bounds__(NS_T) void ns_gram_kernel(GramArgs g, double* ws)
{
    __shared__ float sh[2 * NS_PANEL];
    __shared__ double red[4];
    const int i = find(g.start, (int)blockIdx.x), b = (int)blockIdx.x - g.start.at[i];
    const T* U = (const T*)g.u[i];
    if (g.tall >> i & 1) gram_tile<true>(U, g.m[i], g.n[i], g.kc[i], g.splits[i], b, ws + g.part[i], sh, red);
    else gram_tile<false>(U, g.m[i], g.n[i], g.kc[i], g.splits[i], b, ws + g.part[i], sh, red);
}

// ------------------------------------------------- A_0 from the partial sums
struct SquareArgs {
    Starts start;
    int m[CF_MAX_OPT_TENSORS];
    int splits[CF_MAX_OPT_TENSORS];
    int64_t part[CF_MAX_OPT_TENSORS];     // doubles from the workspace's start
    int64_t sq[CF_MAX_OPT_TENSORS];       // the five m x m buffers, each ld x ld
};
// Rows, and values of a row, of an m x m fp64 buffer.
__host__ __device__ inline int ns_ld(int m) { return (m + NS_TILE - 1) / NS_TILE * NS_TILE; }
__host__ __device__ inline int64_t ns_size(int m) { return (int64_t)ns_ld(m) * ns_ld(m); }
// Values from one row to the next of the bf16 planes that Q ends in (they take
// the place of a buffer).  With rows of a power of two their columns would
// share few memory channels: the product with U took 28 us in place of 17 for
// 6912 x 256.
__host__ __device__ inline int ns_plane_ld(int m) { return ns_ld(m) + 16; }
__host__ __device__ inline int64_t ns_plane(int m) { return (int64_t)ns_ld(m) * ns_plane_ld(m); }

// Block = one row of a tile pair: four groups of threads each sum every fourth
// split, then the groups are added in order; scales by s^2 and writes the
// element and its mirror.  Block 0 of a matrix also stores s.  The diagonal is
// raised by `lift` times the trace.
__global__ __launch_bounds__(NS_T) void ns_join_kernel(SquareArgs g, int first, float eps, double lift, double* ws,
                                                       double* scale)
{
    __shared__ double red[4], group[4][NS_TILE];
    const int block = first + (int)blockIdx.x, q = find(g.start, block), b = block - g.start.at[q];
    const int m = g.m[q], splits = g.splits[q], ld = ns_ld(m), nt = ld / NS_TILE, pairs = nt * (nt + 1) / 2;
    const double* part = ws + g.part[q];
    const int p = b / NS_TILE, i = b % NS_TILE, j = (int)threadIdx.x % NS_TILE, w = (int)threadIdx.x / NS_TILE;
    const double* in = part + (int64_t)p * (NS_TILE * NS_TILE) + i * NS_TILE + j;
    const int64_t step = (int64_t)pairs * (NS_TILE * NS_TILE);
    double v = 0.0;
    int k = w;
    for (; k + 28 < splits; k += 32) {
        double x[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) x[l] = in[(k + 4 * l) * step];
#pragma unroll
        for (int l = 0; l < 8; ++l) v += x[l];
    }
    for (; k < splits; k += 4) v += in[k * step];
    group[w][j] = v;
    double tr = 0.0;
    for (int e = (int)threadIdx.x; e < splits * nt; e += NS_T) tr += part[(int64_t)splits * pairs * (NS_TILE * NS_TILE) + e];
    tr = block_sum(tr, red);      // (its barriers cover `group` too)
    const double s = 1.0 / (sqrt(tr) + (double)eps);
    if (b == 0 && threadIdx.x == 0) scale[q] = s;
    int ti, tj;
    tile_pair(p, nt, ti, tj);
    if (w != 0 || (ti == tj && i > j)) return;
    v = (((group[0][j] + group[1][j]) + group[2][j]) + group[3][j]) * (s * s);
    double* A = ws + g.sq[q];
    const int64_t I = ti * NS_TILE + i, J = tj * NS_TILE + j;
    if (I == J && I < m) v += lift * tr * (s * s);
    A[I * ld + J] = v;
    A[J * ld + I] = v;
}

// ------------------------------------------------------ m x m symmetric rounds
// D = X Y for symmetric commuting X, Y (so D is symmetric and both operands
// are read along their rows), optionally as a I + b Y + c X Y (X = Y = A).
struct Product {
    int x, y, d;         // buffer indices
    int poly;
    int last;            // D as three bf16 planes for the product with U
};
struct RoundArgs {
    SquareArgs s;
    Product p[2];
    int np;              // 1 or 2 products of every matrix in this launch
    float a, b, c;
};

// v = hi + mid + lo, each the bf16 nearest to what is left, up to 2^-24 of v;
// planes of `size` elements.
__device__ __forceinline__ void put_planes(uint16_t* p, int64_t size, int64_t i, double v)
{
    const uint16_t hi = f2bf((float)v);
    const double r = v - (double)bf2f(hi);
    const uint16_t mid = f2bf((float)r);
    p[i] = hi;
    p[size + i] = mid;
    p[2 * size + i] = f2bf((float)(r - (double)bf2f(mid)));
}

// Small matrices take tiles of 16, many of them, large ones tiles of 32, which
// read less: a whole iteration of 400 x 400 takes 180 and 209 us, 448 x 448
// 197 and 209, 500 x 500 259 and 242.
constexpr int NS_EDGE_16 = 448;

// Block = one (16 TS)^2 tile of the upper triangle; its four waves take every
// fourth 16-deep piece of the reduction and are joined through LDS in order.
// A lane's 16-byte loads cover k = 4 (lane / 16) + 0..3 of a piece: the order
// of k within a piece is the same for both operands.
constexpr int ns_unroll(int ts) { return ts == 1 ? 4 : 2; }      // 64 registers of operands in flight

template <int TS>
__global__ __launch_bounds__(NS_T) void ns_round_kernel(RoundArgs g, double* ws)
{
    constexpr int E = 16 * TS;
    __shared__ double sh[4][E * (E + 1)];
    const int q = find(g.s.start, (int)blockIdx.x), b = (int)blockIdx.x - g.s.start.at[q];
    const int m = g.s.m[q], ld = ns_ld(m), nt = (m + E - 1) / E, pairs = nt * (nt + 1) / 2;
    const Product pr = g.p[b / pairs];
    int ti, tj;
    tile_pair(b % pairs, nt, ti, tj);
    const int64_t sz = ns_size(m);
    const double* X = ws + g.s.sq[q] + pr.x * sz;
    const double* Y = ws + g.s.sq[q] + pr.y * sz;
    double* D = ws + g.s.sq[q] + pr.d * sz;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t at = (int64_t)(lane % 16) * ld + 4 * (lane / 16);
    const double* x = X + (int64_t)ti * E * ld + at;
    const double* y = Y + (int64_t)tj * E * ld + at;
    f64x4 acc[TS][TS] = {};
#pragma unroll ns_unroll(TS)
    for (int k = wave * 16; k < m; k += 64) {
        f64x4 u[TS], v[TS];
#pragma unroll
        for (int r = 0; r < TS; ++r) {
            u[r] = *reinterpret_cast<const f64x4*>(x + (int64_t)r * 16 * ld + k);
            v[r] = *reinterpret_cast<const f64x4*>(y + (int64_t)r * 16 * ld + k);
        }
#pragma unroll
        for (int l = 0; l < 4; ++l)
#pragma unroll
            for (int r = 0; r < TS; ++r)
#pragma unroll
                for (int c = 0; c < TS; ++c)
                    acc[r][c] = __builtin_amdgcn_mfma_f64_16x16x4f64(u[r][l], v[c][l], acc[r][c], 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < TS; ++r)
#pragma unroll
        for (int c = 0; c < TS; ++c)
#pragma unroll
            for (int l = 0; l < 4; ++l)
                sh[wave][(r * 16 + 4 * l + lane / 16) * (E + 1) + c * 16 + lane % 16] = acc[r][c][l];
    __syncthreads();
    // the tile's rows, then its mirror's rows
    for (int side = 0; side < (ti == tj ? 1 : 2); ++side)
        for (int e = (int)threadIdx.x; e < E * E; e += NS_T) {
            const int i = e / E, j = e % E;
            // a diagonal tile takes its lower half from the upper one
            const bool flip = side == 1 || (ti == tj && i > j);
            const int o = flip ? j * (E + 1) + i : i * (E + 1) + j;
            const int I = (side ? tj : ti) * E + i, J = (side ? ti : tj) * E + j;
            double v = ((sh[0][o] + sh[1][o]) + sh[2][o]) + sh[3][o];
            if (pr.poly) {
                v = (double)g.c * v + (double)g.b * Y[(int64_t)I * ld + J];
                if (I == J && I < m) v += (double)g.a;
            }
            if (I >= ld || J >= ld) continue;
            if (pr.last) put_planes((uint16_t*)D, ns_plane(m), (int64_t)I * ns_plane_ld(m) + J, v);
            else D[(int64_t)I * ld + J] = v;
        }
}

// ------------------------------------------------------------------ s Q U
// What is done with the product's element o at flat index i of the matrix.
struct StoreArgs {                      // out = o
    void* out[CF_MAX_OPT_TENSORS];
};
struct ApplyArgs {                      // w <- w keep - rate o
    float* w[CF_MAX_OPT_TENSORS];
    float rate[CF_MAX_OPT_TENSORS];
    float keep;
};
struct FinalArgs {
    Starts start;
    const void* u[CF_MAX_OPT_TENSORS];
    int m[CF_MAX_OPT_TENSORS], n[CF_MAX_OPT_TENSORS];
    uint32_t tall;
    int64_t q[CF_MAX_OPT_TENSORS];      // the Q buffer, doubles from the workspace's start
};

// Done in three passes over a tile's elements: loads, results, stores.  The
// compiler may not move a load past a store, and a wait for a load between
// stores would wait for the stores too.
__device__ __forceinline__ float before(const StoreArgs&, int, int64_t) { return 0.f; }
__device__ __forceinline__ float before(const ApplyArgs& a, int q, int64_t i) { return a.w[q][i]; }
__device__ __forceinline__ float result(const StoreArgs&, int, float o, float) { return o; }
__device__ __forceinline__ float result(const ApplyArgs& a, int q, float o, float w) { return fmaf(-a.rate[q], o, w * a.keep); }
template <typename T> __device__ __forceinline__ void finish(const StoreArgs& a, int q, int64_t i, float v)
{
    Elem<T>::store((T*)a.out[q], i, v);
}
template <typename T> __device__ __forceinline__ void finish(const ApplyArgs& a, int q, int64_t i, float v) { a.w[q][i] = v; }
// Keeps a result's computation before the stores.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// Block = a 64 (short side) x 64 (long side) tile of s Q U on the bf16 matrix
// cores, with both operands as hi + mid + lo (Q's planes from the last round, U
// split as it is staged; 24 bits, an fp32 value whole) and the six products
// above 2^-24: fp32's accuracy and range at 2.7 times its matrix rate.  A stage
// is 64 deep, for there are few: its loads, in flight while the stage before it
// is multiplied, are what takes the time.  The lanes that hold neighbouring
// outputs run along the matrix's rows in memory: short-side indices are the
// matrix core's columns for a tall matrix and its rows for a wide one.
constexpr int NF_K = 64;
constexpr int NF_ROW = NF_K + 8;                 // LDS row stride: 16 rows of an operand fall on all banks
constexpr int NF_PLANE = NS_TILE * NF_ROW;

template <bool TALL, typename T, typename F>
__device__ void final_tile(const T* U, const uint16_t* Q, double s, int m, int n, int b, const F& f, int q, uint16_t* sh)
{
    const int ld = ns_plane_ld(m), across = (m + 63) / 64;
    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
    const int i0 = b % across * 64, j0 = b / across * 64;      // short, long
    const int64_t size = ns_plane(m);
    uint16_t* const su = sh;                                   // [3][64 long][64 k]
    uint16_t* const sq = sh + 3 * NF_PLANE;                    // [3][64 short][64 k]
    // a thread stages twice 8 values of k of one row of each
    const int row = TALL ? t / 4 : t % 64, k8 = TALL ? t % 4 * 8 : t / 64 * 8;
    const int j = min(j0 + row, n - 1);
    const uint16_t* qp = Q + (int64_t)(i0 + t / 4) * ld + t % 4 * 8;
    T u[2][8];
    bf16x8 p[2][3];
    auto load = [&](int k0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int k = k0 + x * 32 + k8;
            if (k0 + NF_K <= m) {
                if (TALL) {
                    __builtin_memcpy(u[x], U + (int64_t)j * m + k, sizeof(u[x]));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[x][e] = U[(int64_t)(k + e) * n + j];
                }
            } else {
                asm volatile("");      // not joined with the wide loads above
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = min(k + e, m - 1);
                    u[x][e] = U[TALL ? (int64_t)j * m + c : (int64_t)c * n + j];
                }
                asm volatile("");
            }
#pragma unroll
            for (int e = 0; e < 3; ++e) p[x][e] = *reinterpret_cast<const bf16x8*>(qp + e * size + k0 + x * 32);
        }
    };
    auto store = [&](int k0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            bf16x8 d[3];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = k0 + x * 32 + k8 + e < m ? (float)((double)elem(u[x], e) * s) : 0.f;
                d[0][e] = (__bf16)v;
                const float v1 = v - (float)d[0][e];
                d[1][e] = (__bf16)v1;
                d[2][e] = (__bf16)(v1 - (float)d[1][e]);
            }
            // (Q's columns are zeros up to a multiple of 16 above m, and hold anything after it)
            if (k0 + x * 32 + t % 4 * 8 >= m)
#pragma unroll
                for (int e = 0; e < 3; ++e) p[x][e] = bf16x8{};
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                *reinterpret_cast<bf16x8*>(su + e * NF_PLANE + row * NF_ROW + x * 32 + k8) = d[e];
                *reinterpret_cast<bf16x8*>(sq + e * NF_PLANE + t / 4 * NF_ROW + x * 32 + t % 4 * 8) = p[x][e];
            }
        }
    };
    const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;      // this wave's quadrant: short, long
    const bf16x8* a = reinterpret_cast<const bf16x8*>(sq + (wi + lane % 32) * NF_ROW + lane / 32 * 8);
    const bf16x8* c = reinterpret_cast<const bf16x8*>(su + (wj + lane % 32) * NF_ROW + lane / 32 * 8);
    f32x16 acc = {}, small = {};
    // the stages in a round that starts elsewhere for the next block: all blocks at one k would read rows that lie
    // 4 m bytes apart, from a part of the memory channels
    const int stages = (m + NF_K - 1) / NF_K;
    int k0 = (b / across + b) % stages * NF_K;
    load(k0);
    for (int i = 0; i < stages; ++i) {
        __syncthreads();
        store(k0);
        __syncthreads();
        k0 = k0 + NF_K < m ? k0 + NF_K : 0;
        if (i + 1 < stages) load(k0);
#pragma unroll
        for (int k = 0; k < NF_K / 16; ++k) {
            bf16x8 x[3], y[3];
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                x[e] = a[(e * NF_PLANE + k * 16) / 8];
                y[e] = c[(e * NF_PLANE + k * 16) / 8];
            }
#pragma unroll
            for (int z = 0; z < 6; ++z) {
                    // (e, o): 02 00 11 01 20 10: three of the second order in one chain, three larger in the other
                    const int o = z % 2 == 0 ? 2 : z == 1 ? 0 : 1, e = z == 0 || z == 1 || z == 3 ? 0 : z == 4 ? 2 : 1;
                    f32x16& sum = o == 2 ? small : acc;
                    // rows from the first operand, columns (lanes) from the second
                    sum = TALL ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[o - e], x[e], sum, 0, 0, 0)
                               : __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[e], y[o - e], sum, 0, 0, 0);
                }
        }
    }
    // register v of a lane: row 8 (v / 4) + 4 (lane / 32) + v % 4, column lane % 32
    auto place = [&](int v) {
        const int r = 8 * (v / 4) + 4 * (lane / 32) + v % 4, l = lane % 32;
        const int I = i0 + wi + (TALL ? l : r), J = j0 + wj + (TALL ? r : l);
        return I < m && J < n ? TALL ? (int64_t)J * m + I : (int64_t)I * n + J : (int64_t)-1;
    };
    float w[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) w[v] = before(f, q, max(place(v), (int64_t)0));
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        w[v] = result(f, q, acc[v] + small[v], w[v]);
        settle(w[v]);
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int64_t at = place(v);
        if (at >= 0) finish<T>(f, q, at, w[v]);
    }
}

template <typename T, typename F>
__global__ __launch_bounds__(NS_T) void ns_final_kernel(FinalArgs g, int first, F f, const double* ws, const double* scale)
{
    __shared__ __attribute__((aligned(16))) uint16_t sh[6 * NF_PLANE];
    const int block = first + (int)blockIdx.x, i = find(g.start, block), b = block - g.start.at[i];
    const T* U = (const T*)g.u[i];
    const uint16_t* Q = (const uint16_t*)(ws + g.q[i]);
    if (g.tall >> i & 1) final_tile<true>(U, Q, scale[i], g.m[i], g.n[i], b, f, i, sh);
    else final_tile<false>(U, Q, scale[i], g.m[i], g.n[i], b, f, i, sh);
}

// Block = the same tile in fp64, with Q as the rounds leave it; each wave a
// 32 x 32 quadrant.  U's panel is staged in LDS, Q's rows come from memory, 32
// bytes a lane: k = 4 (lane / 16) + 0..3 of a piece of 16, for both operands.
// 449 x 4300 takes 65 us here and 41 with three bf16 parts.
template <bool TALL, typename T, typename F>
__device__ void final64_tile(const T* U, const double* Q, double s, int m, int n, int b, const F& f, int q, float* su)
{
    const int ld = ns_ld(m), across = (m + NS_TILE - 1) / NS_TILE;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, h = lane / 16, c = lane % 16;
    const int i0 = b % across * NS_TILE, j0 = b / across * NS_TILE;      // short, long
    const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
    const double* qr = Q + (int64_t)(i0 + wi + c) * ld + 4 * h;
    f64x4 acc[2][2] = {};      // [short][long]
    float v[NS_PV];
    panel_load<!TALL>(v, U, n, m, j0, 0, m);      // rows of the long side, the short side to be summed over
    for (int k0 = 0; k0 < m; k0 += NS_K) {
        __syncthreads();
        panel_store<!TALL>(v, su);
        __syncthreads();
        if (k0 + NS_K < m) panel_load<!TALL>(v, U, n, m, j0, k0 + NS_K, m);
#pragma unroll
        for (int p = 0; p < NS_K; p += 16) {
            if (k0 + p >= m) break;      // (Q's columns are zeros up to a multiple of 16 above m, and hold anything after it)
            f64x4 x[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) x[r] = *reinterpret_cast<const f64x4*>(qr + (int64_t)r * 16 * ld + k0 + p);
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const int k = p + 4 * h + l;
                double y[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int j = wj + r * 16 + c;
                    y[r] = (double)su[TALL ? j * NS_SK + k : k * NS_SP + j];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = TALL ? __builtin_amdgcn_mfma_f64_16x16x4f64(y[j], x[i][l], acc[i][j], 0, 0, 0)
                                         : __builtin_amdgcn_mfma_f64_16x16x4f64(x[i][l], y[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    // element e of a lane's four: row 4 e + lane / 16, column lane % 16
    auto place = [&](int i, int j, int e) {
        const int I = i0 + wi + i * 16 + (TALL ? c : 4 * e + h), J = j0 + wj + j * 16 + (TALL ? 4 * e + h : c);
        return I < m && J < n ? TALL ? (int64_t)J * m + I : (int64_t)I * n + J : (int64_t)-1;
    };
    float w[2][2][4];
#pragma unroll
    for (int e = 0; e < 16; ++e)
        w[e / 8][e / 4 % 2][e % 4] = before(f, q, max(place(e / 8, e / 4 % 2, e % 4), (int64_t)0));
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float& o = w[e / 8][e / 4 % 2][e % 4];
        o = result(f, q, (float)(acc[e / 8][e / 4 % 2][e % 4] * s), o);
        settle(o);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int64_t at = place(e / 8, e / 4 % 2, e % 4);
        if (at >= 0) finish<T>(f, q, at, w[e / 8][e / 4 % 2][e % 4]);
    }
}

template <typename T, typename F>
__global__ __launch_bounds__(NS_T) void ns_final64_kernel(FinalArgs g, int first, F f, const double* ws,
                                                          const double* scale)
{
    __shared__ float sh[NS_PANEL];
    const int block = first + (int)blockIdx.x, i = find(g.start, block), b = block - g.start.at[i];
    const T* U = (const T*)g.u[i];
    if (g.tall >> i & 1) final64_tile<true>(U, ws + g.q[i], scale[i], g.m[i], g.n[i], b, f, i, sh);
    else final64_tile<false>(U, ws + g.q[i], scale[i], g.m[i], g.n[i], b, f, i, sh);
}

// ----------------------------------------------- one block for a small matrix
// The iteration of a matrix with m <= 64 in one block's LDS: three fp64 m x m
// buffers, results held in registers until every wave has read.  64 x 512 takes
// 42 us for 14 rounds' 65; the matrix cores are busy half of the time, the rest
// is barriers and the uneven share of 10 tiles among 4 SIMDs.  WHOLE: also
// U U^T and s Q U, from U in LDS; else A_0 comes from the joining launch and Q
// goes to its planes, or as it is where s Q U is an fp64 product.
constexpr int NB_T = 1024;
constexpr int NB_W = NB_T / 64;                  // waves
constexpr int NB_M = 64;
constexpr int NB_BUF = NB_M * (NB_M + 2);        // a row of LD = 16 t + 2 doubles: the 16 rows of an operand start an
                                                 // odd number of 16-byte steps apart
constexpr int NB_U = 10240;                      // floats of U
__host__ __device__ inline int nb_ldu(int mp) { return mp + (mp % 32 == 0 ? 16 : 0); }      // 4 rows of 16: 64 banks
bool ns_whole(int m, int n) { return m <= NB_M && (int64_t)nb_ldu(up(m, 16)) * up(n, 16) <= NB_U; }

struct BlockArgs {
    const void* u[CF_MAX_OPT_TENSORS];
    int m[CF_MAX_OPT_TENSORS], n[CF_MAX_OPT_TENSORS];
    uint32_t tall;
    int64_t a[CF_MAX_OPT_TENSORS], q[CF_MAX_OPT_TENSORS];      // A_0 and Q's planes, doubles from the workspace's start
    int steps, many;
    float ca, cb, cc, eps;
    double lift;
};

template <bool WHOLE, typename T, typename F>
__global__ __launch_bounds__(NB_T) void ns_block_kernel(BlockArgs g, F f, double* ws)
{
    __shared__ double A[NB_BUF], P[NB_BUF], Q[NB_BUF];
    __shared__ double part[WHOLE ? 8 * 256 : 1], trace[4];
    __shared__ float us[WHOLE ? NB_U : 1];
    const int q = (int)blockIdx.x, m = g.m[q], n = g.n[q];
    const int mp = (m + 15) / 16 * 16, LD = mp + 2, nt = mp / 16, pairs = nt * (nt + 1) / 2;
    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
    const int r = lane % 16, h = lane / 16;      // operands: row r, k = h; results: row 4 v + h, column r
    const bool tall = g.tall >> q & 1;
    double s = 0.0;

    // a 16 x 16 tile of X Y, both symmetric
    auto product = [&](const double* X, const double* Y, int p) {
        int ti, tj;
        tile_pair(p, nt, ti, tj);
        const double* x = X + (ti * 16 + r) * LD + h;
        const double* y = Y + (tj * 16 + r) * LD + h;
        f64x4 a0 = {}, a1 = {};      // two chains: a matrix instruction waits for its own sum
#pragma unroll 2
        for (int k = 0; k < mp; k += 16) {
            a0 = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k], y[k], a0, 0, 0, 0);
            a1 = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k + 4], y[k + 4], a1, 0, 0, 0);
            a0 = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k + 8], y[k + 8], a0, 0, 0, 0);
            a1 = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k + 12], y[k + 12], a1, 0, 0, 0);
        }
        return a0 + a1;
    };
    // its upper part and mirror
    auto put = [&](double* D, int p, const f64x4& x) {
        int ti, tj;
        tile_pair(p, nt, ti, tj);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = ti * 16 + 4 * v + h, j = tj * 16 + r;
            if (i > j) continue;
            D[i * LD + j] = x[v];
            D[j * LD + i] = x[v];
        }
    };

    if constexpr (WHOLE) {
        const T* U = (const T*)g.u[q];
        const int ldu = nb_ldu(mp), np = (n + 15) / 16 * 16;
        for (int e = t; e < np * ldu; e += NB_T) us[e] = 0.f;
        __syncthreads();
        for (int e = t; e < n * m; e += NB_T) {
            const int k = tall ? e / m : e % n, i = tall ? e % m : e / n;
            us[k * ldu + i] = elem(U, e);
        }
        __syncthreads();
        // few tiles: their reductions are cut into parts, one for each wave
        const int parts = max(1, 8 / pairs);
        for (int w = wave; w < parts * pairs; w += NB_W) {
            int ti, tj;
            tile_pair(w % pairs, nt, ti, tj);
            f64x4 acc = {};
            for (int k = w / pairs * 4 + h; k < np; k += 4 * parts)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)us[k * ldu + ti * 16 + r], (double)us[k * ldu + tj * 16 + r],
                                                           acc, 0, 0, 0);
            if (parts > 1) {
#pragma unroll
                for (int v = 0; v < 4; ++v) part[w * 256 + v * 64 + lane] = acc[v];
            } else {
                put(A, w, acc);
            }
        }
        __syncthreads();
        if (parts > 1) {
            if (wave < pairs) {
                f64x4 acc = {};
                for (int x = 0; x < parts; ++x)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[v] += part[(x * pairs + wave) * 256 + v * 64 + lane];
                put(A, wave, acc);
            }
            __syncthreads();
        }
        if (wave == 0) {
            const double tr = wave_sum(lane < m ? A[lane * LD + lane] : 0.0);
            if (lane == 0) trace[0] = tr;
        }
        __syncthreads();
        s = 1.0 / (sqrt(trace[0]) + (double)g.eps);
        const double up = g.lift * trace[0];
        for (int e = t; e < mp * mp; e += NB_T) {
            double& v = A[e / mp * LD + e % mp];
            v = (e / mp == e % mp && e % mp < m ? v + up : v) * (s * s);
        }
    } else {
        const double* in = ws + g.a[q];
        const int ld = ns_ld(m);
        for (int e = t; e < mp * mp; e += NB_T) A[e / mp * LD + e % mp] = in[(int64_t)(e / mp) * ld + e % mp];
    }
    __syncthreads();
    for (int k = 0; k < g.steps; ++k) {
        const bool last = k + 1 == g.steps;
        for (int p = wave; p < pairs; p += NB_W) {
            f64x4 x = product(A, A, p);
            int ti, tj;
            tile_pair(p, nt, ti, tj);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int i = ti * 16 + 4 * v + h, j = tj * 16 + r;
                x[v] = (double)g.cc * x[v] + (double)g.cb * A[i * LD + j] + (i == j && i < m ? (double)g.ca : 0.0);
            }
            put(P, p, x);
            if (k == 0) put(Q, p, x);      // Q = P_0
        }
        __syncthreads();
        // P A (but for the last step), P Q (but for the first): A and Q are replaced when all have read them
        const int first = last ? pairs : 0, count = k == 0 ? pairs : 2 * pairs;
        f64x4 x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = first + wave + NB_W * i;
            if (w < count) x[i] = product(P, w < pairs ? A : Q, w < pairs ? w : w - pairs);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = first + wave + NB_W * i;
            if (w < count) put(w < pairs ? A : Q, w < pairs ? w : w - pairs, x[i]);
        }
        __syncthreads();
        if (last) break;
        if (wave < pairs) x[0] = product(A, P, wave);
        __syncthreads();
        if (wave < pairs) put(A, wave, x[0]);
        __syncthreads();
    }
    if constexpr (WHOLE) {
        const int ldu = nb_ldu(mp), np = (n + 15) / 16 * 16;
        for (int w = wave; w < np / 16 * nt; w += NB_W) {
            const int i0 = w % nt * 16, j0 = w / nt * 16;      // short, long
            f64x4 acc = {};
            for (int k = 0; k < mp; k += 4) {
                const double a = Q[(i0 + r) * LD + k + h], b = (double)us[(j0 + r) * ldu + k + h] * s;
                acc = tall ? __builtin_amdgcn_mfma_f64_16x16x4f64(b, a, acc, 0, 0, 0)
                           : __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, acc, 0, 0, 0);
            }
            int64_t at[4];
            float x[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int i = i0 + (tall ? r : 4 * v + h), j = j0 + (tall ? 4 * v + h : r);
                at[v] = i < m && j < n ? tall ? (int64_t)j * m + i : (int64_t)i * n + j : -1;
                x[v] = before(f, q, max(at[v], (int64_t)0));
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                x[v] = result(f, q, (float)acc[v], x[v]);
                settle(x[v]);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (at[v] >= 0) finish<T>(f, q, at[v], x[v]);
        }
    } else if (g.many) {
        const int ld = ns_ld(m);
        double* out = ws + g.q[q];
        for (int e = t; e < mp * mp; e += NB_T) out[(int64_t)(e / mp) * ld + e % mp] = Q[e / mp * LD + e % mp];
    } else {
        const int ld = ns_plane_ld(m);
        uint16_t* out = (uint16_t*)(ws + g.q[q]);
        for (int e = t; e < mp * mp; e += NB_T)
            put_planes(out, ns_plane(m), (int64_t)(e / mp) * ld + e % mp, Q[e / mp * LD + e % mp]);
    }
}

// --------------------------------------------------------------- momentum
struct MomentumArgs {
    Starts start;
    int64_t n[CF_MAX_OPT_TENSORS];
    const float* g[CF_MAX_OPT_TENSORS];
    float* m[CF_MAX_OPT_TENSORS];
    float* u[CF_MAX_OPT_TENSORS];       // g + mu m where nesterov, else unused
};
constexpr int MU_V = 4;                             // float4 per thread
constexpr int MU_CHUNK = NS_T * MU_V * 4;

__global__ __launch_bounds__(NS_T) void muon_momentum_kernel(MomentumArgs a, float mu, int nesterov)
{
    const int q = find(a.start, (int)blockIdx.x);
    const int64_t n = a.n[q], base = (int64_t)((int)blockIdx.x - a.start.at[q]) * MU_CHUNK;
    const float* g = a.g[q];
    float* m = a.m[q];
    float* u = a.u[q];
#pragma unroll
    for (int r = 0; r < MU_V; ++r) {
        const int64_t i = base + ((int64_t)r * NS_T + threadIdx.x) * 4;
        if (i + 4 <= n) {
            const float4 gv = *reinterpret_cast<const float4*>(g + i);
            float4 mv = *reinterpret_cast<const float4*>(m + i);
            mv.x = fmaf(mu, mv.x, gv.x);
            mv.y = fmaf(mu, mv.y, gv.y);
            mv.z = fmaf(mu, mv.z, gv.z);
            mv.w = fmaf(mu, mv.w, gv.w);
            *reinterpret_cast<float4*>(m + i) = mv;
            if (nesterov)
                *reinterpret_cast<float4*>(u + i) = make_float4(fmaf(mu, mv.x, gv.x), fmaf(mu, mv.y, gv.y),
                                                                fmaf(mu, mv.z, gv.z), fmaf(mu, mv.w, gv.w));
        } else {
            for (int64_t j = i; j < n; ++j) {
                const float mv = fmaf(mu, m[j], g[j]);
                m[j] = mv;
                if (nesterov) u[j] = fmaf(mu, mv, g[j]);
            }
        }
    }
}

// -------------------------------------------------------------------- plan
struct NsPlan {
    int64_t part[CF_MAX_OPT_TENSORS], sq[CF_MAX_OPT_TENSORS];   // doubles
    int kc[CF_MAX_OPT_TENSORS], splits[CF_MAX_OPT_TENSORS];
    int64_t doubles;
};
constexpr int NS_BLOCKS = 1024;     // blocks wanted of the U U^T launch
constexpr int NS_KC_MIN = 128;      // least reduction depth of a block

NsPlan ns_plan(const NsShapes& l)
{
    NsPlan p{};
    // the same work per block over the list
    double work = 0.0;
    for (int i = 0; i < l.count; ++i) {
        const int64_t nt = (l.m[i] + NS_TILE - 1) / NS_TILE;
        work += (double)(nt * (nt + 1) / 2) * l.n[i];
    }
    int64_t kc = (int64_t)(work / NS_BLOCKS) + 1;
    kc = std::max<int64_t>(NS_KC_MIN, (kc + NS_K - 1) / NS_K * NS_K);
    int64_t at = CF_MAX_OPT_TENSORS;        // the scales come first
    for (int i = 0; i < l.count; ++i) {
        const int64_t nt = ns_ld(l.m[i]) / NS_TILE, pairs = nt * (nt + 1) / 2;
        p.kc[i] = (int)std::min<int64_t>(kc, up(l.n[i], NS_K));
        p.splits[i] = (l.n[i] + p.kc[i] - 1) / p.kc[i];
        p.part[i] = at;
        at += p.splits[i] * (pairs * NS_TILE * NS_TILE + nt);
        at = (at + 31) / 32 * 32;
        p.sq[i] = at;
        at += 5 * ns_size(l.m[i]);
    }
    p.doubles = at;
    return p;
}

// Whether eigenvalues of A_0's rounding, 2^-53, could grow past 2^-24, a^2 a
// step; what the diagonal is raised by then.
bool ns_many(const NsCoef& c) { return std::fabs(c.a) > 1.f && 2.0 * c.steps * std::log2(std::fabs((double)c.a)) > 29.0; }
constexpr double NS_LIFT = 0x1p-48;

// Calls launch(first block, blocks) over a launch's blocks: more than once
// where they have 2^32 threads or more, which one launch may not (a matrix of
// 1 x 2^30 has 2^24 tiles).
template <typename L> hipError_t in_launches(int blocks, const L& launch)
{
    constexpr int most = (1 << 24) - 1;
    static_assert((int64_t)most * NS_T < (int64_t)1 << 32, "threads of a launch");
    for (int at = 0; at < blocks; at += most) {
        launch(at, dim3((unsigned)std::min(most, blocks - at)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Everything of a list from U on.
template <typename T, typename F>
hipError_t ns_f64(const NsShapes& l, const void* const* u, const NsCoef& c, const F& f, double* ws, hipStream_t s)
{
    const NsPlan p = ns_plan(l);
    const bool many = ns_many(c);
    const double lift = many ? NS_LIFT : 0.0;
    bool whole = true;
    int maxm = 0;
    BlockArgs k{};
    k.tall = l.tall;
    k.steps = c.steps;
    k.ca = c.a;
    k.cb = c.b;
    k.cc = c.c;
    k.eps = c.eps;
    k.many = many;
    k.lift = lift;
    for (int i = 0; i < l.count; ++i) {
        whole = whole && ns_whole(l.m[i], l.n[i]);
        maxm = std::max(maxm, l.m[i]);
        k.u[i] = u[i];
        k.m[i] = l.m[i];
        k.n[i] = l.n[i];
        k.a[i] = p.sq[i];
        k.q[i] = p.sq[i] + ns_size(l.m[i]);
    }
    if (whole) {
        hipLaunchKernelGGL((ns_block_kernel<true, T, F>), dim3((unsigned)l.count), dim3(NB_T), 0, s, k, f, ws);
        return hipGetLastError();
    }

    GramArgs g{};
    SquareArgs sq{};
    FinalArgs a{};
    g.start.clear();
    sq.start.clear();
    a.start.clear();
    int grams = 0, joins = 0, finals = 0;
    for (int i = 0; i < l.count; ++i) {
        const int nt = ns_ld(l.m[i]) / NS_TILE, pairs = nt * (nt + 1) / 2;
        g.u[i] = a.u[i] = u[i];
        g.m[i] = sq.m[i] = a.m[i] = l.m[i];
        g.n[i] = a.n[i] = l.n[i];
        g.kc[i] = p.kc[i];
        g.splits[i] = sq.splits[i] = p.splits[i];
        g.part[i] = sq.part[i] = p.part[i];
        sq.sq[i] = p.sq[i];
        g.start.set(i, grams);
        sq.start.set(i, joins);
        a.start.set(i, finals);
        grams += p.splits[i] * pairs;
        joins += pairs * NS_TILE;
        finals += nt * ((l.n[i] + 63) / 64);
    }
    g.tall = a.tall = l.tall;
    hipLaunchKernelGGL(ns_gram_kernel<T>, dim3((unsigned)grams), dim3(NS_T), 0, s, g, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = in_launches(joins, [&](int first, dim3 grid) {
        hipLaunchKernelGGL(ns_join_kernel, grid, dim3(NS_T), 0, s, sq, first, c.eps, lift, ws, ws);
    });
    if (e != hipSuccess) return e;

    int A = 0, T_ = 1, P = 2, Q = 3, R = 4;      // buffers: A_k, P A, P_k, Q and a free one
    if (maxm <= NB_M) {
        hipLaunchKernelGGL((ns_block_kernel<false, T, F>), dim3((unsigned)l.count), dim3(NB_T), 0, s, k, f, ws);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        Q = 1;
    } else {
        RoundArgs r{};
        r.s = sq;
        r.a = c.a;
        r.b = c.b;
        r.c = c.c;
        const int edge = maxm <= NS_EDGE_16 ? 16 : 32;
        auto round = [&](std::initializer_list<Product> ps) -> hipError_t {
            r.np = 0;
            for (const Product& x : ps) r.p[r.np++] = x;
            int blocks = 0;
            for (int i = 0; i < l.count; ++i) {
                const int nt = (l.m[i] + edge - 1) / edge;
                r.s.start.set(i, blocks);
                blocks += r.np * (nt * (nt + 1) / 2);
            }
            if (edge == 16) hipLaunchKernelGGL(ns_round_kernel<1>, dim3((unsigned)blocks), dim3(NS_T), 0, s, r, ws);
            else hipLaunchKernelGGL(ns_round_kernel<2>, dim3((unsigned)blocks), dim3(NS_T), 0, s, r, ws);
            return hipGetLastError();
        };
        for (int i = 0; i < c.steps; ++i) {
            const bool last = i + 1 == c.steps;
            const int planes = last && !many;
            if (i == 0) {
                if ((e = round({{A, A, Q, 1, planes}})) != hipSuccess) return e;      // Q = P_0
                if (!last && (e = round({{Q, A, T_, 0, 0}})) != hipSuccess) return e;
                if (!last && (e = round({{T_, Q, A, 0, 0}})) != hipSuccess) return e;
                continue;
            }
            if ((e = round({{A, A, P, 1, 0}})) != hipSuccess) return e;
            if (last) e = round({{P, Q, R, 0, planes}});
            else e = round({{P, A, T_, 0, 0}, {P, Q, R, 0, 0}});
            if (e != hipSuccess) return e;
            std::swap(Q, R);
            if (!last && (e = round({{T_, P, A, 0, 0}})) != hipSuccess) return e;
        }
    }
    for (int i = 0; i < l.count; ++i) a.q[i] = p.sq[i] + Q * ns_size(l.m[i]);
    return in_launches(finals, [&](int first, dim3 grid) {
        if (many) hipLaunchKernelGGL((ns_final64_kernel<T, F>), grid, dim3(NS_T), 0, s, a, first, f, ws, ws);
        else hipLaunchKernelGGL((ns_final_kernel<T, F>), grid, dim3(NS_T), 0, s, a, first, f, ws, ws);
    });
}

// The matrices of a list that take the fp64 launches together, and those that
// take split products one after another.
struct NsParts {
    NsShapes f64;
    int f64_at[CF_MAX_OPT_TENSORS];      // their places in the list
    int split[CF_MAX_OPT_TENSORS], splits;
};
NsParts ns_parts(const NsShapes& l, bool allow_split)
{
    NsParts p{};
    // Matrices that share the rounds' launches: with two or more, those of moderate size join them rather than take
    // 17 launches each (400 x 400 beside 256 x 6912: 264 us apart, 202 together).
    int rounds = 0;
    for (int i = 0; i < l.count; ++i)
        rounds += ns_split_size(l.m[i], l.n[i]) ? l.m[i] <= NS_EDGE_16 : l.m[i] > NB_M;
    for (int i = 0; i < l.count; ++i) {
        if (allow_split && ns_split_size(l.m[i], l.n[i]) && !(rounds > 1 && l.m[i] <= NS_EDGE_16)) {
            p.split[p.splits++] = i;
            continue;
        }
        const int k = p.f64.count++;
        p.f64.m[k] = l.m[i];
        p.f64.n[k] = l.n[i];
        p.f64.tall |= (l.tall >> i & 1u) << k;
        p.f64_at[k] = i;
    }
    return p;
}

size_t ns_f64_ws_bytes(const NsShapes& l) { return l.count ? up256b((size_t)ns_plan(l).doubles * sizeof(double)) : 0; }

}  // namespace

namespace {
size_t ns_parts_ws_bytes(const NsShapes& l, const NsParts& p)
{
    size_t b = ns_f64_ws_bytes(p.f64);
    for (int i = 0; i < p.splits; ++i) b = std::max(b, ns_split_ws_bytes(l.m[p.split[i]], l.n[p.split[i]]));
    return b;
}
}  // namespace

// What any coefficients need at most, and what these need.
size_t ns_ws_bytes(const NsShapes& l)
{
    return std::max(ns_parts_ws_bytes(l, ns_parts(l, false)), ns_parts_ws_bytes(l, ns_parts(l, true)));
}
size_t ns_ws_bytes(const NsShapes& l, const NsCoef& c) { return ns_parts_ws_bytes(l, ns_parts(l, ns_split_coef(c))); }

template <typename T>
hipError_t launch_newton_schulz(const NsShapes& l, const NsCoef& c, const void* const* x, void* const* out, void* ws,
                                hipStream_t s)
{
    const NsParts p = ns_parts(l, ns_split_coef(c));
    hipError_t e;
    for (int i = 0; i < p.splits; ++i) {
        const int k = p.split[i];
        if ((e = launch_ns_split<T>(l.m[k], l.n[k], l.tall >> k & 1, c, (const T*)x[k], (T*)out[k], ws, s)) !=
            hipSuccess)
            return e;
    }
    if (!p.f64.count) return hipSuccess;
    const void* u[CF_MAX_OPT_TENSORS];
    StoreArgs f{};
    for (int i = 0; i < p.f64.count; ++i) {
        u[i] = x[p.f64_at[i]];
        f.out[i] = out[p.f64_at[i]];
    }
    return ns_f64<T>(p.f64, u, c, f, (double*)ws, s);
}

size_t muon_ws_bytes(const NsShapes& l, const NsCoef& c, bool nesterov)
{
    size_t b = ns_ws_bytes(l, c);
    if (nesterov)
        for (int i = 0; i < l.count; ++i) b += up256b((size_t)l.m[i] * l.n[i] * sizeof(float));
    return b;
}

hipError_t launch_muon(const NsShapes& l, const NsCoef& c, const MuonArgs& h, float* const* w, const float* const* g,
                       float* const* m, void* ws, hipStream_t s)
{
    MomentumArgs a{};
    const float* u[CF_MAX_OPT_TENSORS];
    char* at = (char*)ws + ns_ws_bytes(l, c);
    a.start.clear();
    int blocks = 0;
    for (int i = 0; i < l.count; ++i) {
        a.start.set(i, blocks);
        a.n[i] = (int64_t)l.m[i] * l.n[i];
        a.g[i] = g[i];
        a.m[i] = m[i];
        u[i] = m[i];
        if (h.nesterov) {
            a.u[i] = (float*)at;
            u[i] = a.u[i];
            at += up256b((size_t)a.n[i] * sizeof(float));
        }
        blocks += (int)((a.n[i] + MU_CHUNK - 1) / MU_CHUNK);
    }
    hipLaunchKernelGGL(muon_momentum_kernel, dim3((unsigned)blocks), dim3(NS_T), 0, s, a, h.momentum,
                       (int)h.nesterov);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const NsParts p = ns_parts(l, ns_split_coef(c));
    for (int i = 0; i < p.splits; ++i) {
        const int k = p.split[i];
        if ((e = launch_ns_split_apply(l.m[k], l.n[k], l.tall >> k & 1, c, u[k], w[k], h.keep, h.rate[k], ws, s)) !=
            hipSuccess)
            return e;
    }
    if (!p.f64.count) return hipSuccess;
    const void* v[CF_MAX_OPT_TENSORS];
    ApplyArgs f{};
    f.keep = h.keep;
    for (int i = 0; i < p.f64.count; ++i) {
        v[i] = u[p.f64_at[i]];
        f.w[i] = w[p.f64_at[i]];
        f.rate[i] = h.rate[p.f64_at[i]];
    }
    return ns_f64<float>(p.f64, v, c, f, (double*)ws, s);
}

template hipError_t launch_newton_schulz<float>(const NsShapes&, const NsCoef&, const void* const*, void* const*,
                                                void*, hipStream_t);
template hipError_t launch_newton_schulz<uint16_t>(const NsShapes&, const NsCoef&, const void* const*, void* const*,
                                                   void*, hipStream_t);

}  // namespace cf
