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
// fp32.
//
// Launches take a list of matrices; partial sums are added in a fixed order
// and there are no atomics: results are reproducible bit for bit.
#include "cf_internal.h"

#include <algorithm>

namespace cf {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int NS_T = 256;       // threads per block, 4 waves
constexpr int NS_TILE = 64;     // edge of an output tile of U U^T and of Q U
constexpr int NS_K = 32;        // reduction depth of a staged panel
constexpr int NS_SP = NS_TILE + 16;   // LDS row stride of a [k][64] panel: its 4 k rows x 16 columns of a
                                      // matrix-core operand fall on 64 different banks
constexpr int NS_SK = NS_K + 1;       // LDS row stride of a [64][k] panel

int up(int v, int m) { return (v + m - 1) / m * m; }
size_t up256b(size_t b) { return (b + 255) & ~(size_t)255; }

// The matrix whose range of blocks holds block b.
__device__ __forceinline__ int find(const int* start, int count, int b)
{
    int i = 0;
    while (i + 1 < count && b >= start[i + 1]) ++i;
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
    int count;
    int start[CF_MAX_OPT_TENSORS + 1];        // first block of each matrix
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
    const int i = find(g.start, g.count, (int)blockIdx.x), b = (int)blockIdx.x - g.start[i];
    const T* U = (const T*)g.u[i];
    if (g.tall >> i & 1) gram_tile<true>(U, g.m[i], g.n[i], g.kc[i], g.splits[i], b, ws + g.part[i], sh, red);
    else gram_tile<false>(U, g.m[i], g.n[i], g.kc[i], g.splits[i], b, ws + g.part[i], sh, red);
}

// ------------------------------------------------- A_0 from the partial sums
struct SquareArgs {
    int count;
    int start[CF_MAX_OPT_TENSORS + 1];
    int m[CF_MAX_OPT_TENSORS];
    int splits[CF_MAX_OPT_TENSORS];
    int64_t part[CF_MAX_OPT_TENSORS];     // doubles from the workspace's start
    int64_t sq[CF_MAX_OPT_TENSORS];       // the five m x m buffers, each ld x ld
};
__host__ __device__ inline int ns_ld(int m) { return (m + NS_TILE - 1) / NS_TILE * NS_TILE; }

// Block = 16 rows of a tile pair: sums the splits in order, scales by s^2 and
// writes the element and its mirror; block 0 of a matrix also stores s.
constexpr int NS_JR = 16;
__global__ __launch_bounds__(NS_T) void ns_join_kernel(SquareArgs g, float eps, double* ws, double* scale)
{
    __shared__ double red[4];
    const int q = find(g.start, g.count, (int)blockIdx.x), b = (int)blockIdx.x - g.start[q];
    const int m = g.m[q], splits = g.splits[q], ld = ns_ld(m), nt = ld / NS_TILE, pairs = nt * (nt + 1) / 2;
    const double* part = ws + g.part[q];
    double tr = 0.0;
    for (int i = (int)threadIdx.x; i < splits * nt; i += NS_T)
        tr += part[(int64_t)splits * pairs * (NS_TILE * NS_TILE) + i];
    const double s = 1.0 / (sqrt(block_sum(tr, red)) + (double)eps);
    if (b == 0 && threadIdx.x == 0) scale[q] = s;
    const int p = b / (NS_TILE / NS_JR), r0 = b % (NS_TILE / NS_JR) * NS_JR;
    int ti, tj;
    tile_pair(p, nt, ti, tj);
    double* A = ws + g.sq[q];
    for (int e = (int)threadIdx.x; e < NS_JR * NS_TILE; e += NS_T) {
        const int i = r0 + e / NS_TILE, j = e % NS_TILE;
        if (ti == tj && i > j) continue;
        double v = 0.0;
        for (int k = 0; k < splits; ++k) v += part[((int64_t)k * pairs + p) * (NS_TILE * NS_TILE) + i * NS_TILE + j];
        v *= s * s;
        const int64_t I = ti * NS_TILE + i, J = tj * NS_TILE + j;
        A[I * ld + J] = v;
        A[J * ld + I] = v;
    }
}

// ------------------------------------------------------ m x m symmetric rounds
// D = X Y for symmetric commuting X, Y (so D is symmetric and both operands
// are read along their rows), optionally as a I + b Y + c X Y (X = Y = A).
struct Product {
    int x, y, d;         // buffer indices
    int poly;
};
struct RoundArgs {
    SquareArgs s;
    Product p[2];
    int np;              // 1 or 2 products of every matrix in this launch
    float a, b, c;
};

// Block = one (16 TS)^2 tile of the upper triangle; its four waves take every
// fourth 16-deep piece of the reduction and are joined through LDS in order.
// A lane's 16-byte loads cover k = 4 (lane / 16) + 0..3 of a piece: the order
// of k within a piece is the same for both operands.
template <int TS>
__global__ __launch_bounds__(NS_T) void ns_round_kernel(RoundArgs g, double* ws)
{
    constexpr int E = 16 * TS;
    __shared__ double sh[4][E * (E + 1)];
    const int q = find(g.s.start, g.s.count, (int)blockIdx.x), b = (int)blockIdx.x - g.s.start[q];
    const int m = g.s.m[q], ld = ns_ld(m), nt = (m + E - 1) / E, pairs = nt * (nt + 1) / 2;
    const Product pr = g.p[b / pairs];
    int ti, tj;
    tile_pair(b % pairs, nt, ti, tj);
    const int64_t sz = (int64_t)ld * ld;
    const double* X = ws + g.s.sq[q] + pr.x * sz;
    const double* Y = ws + g.s.sq[q] + pr.y * sz;
    double* D = ws + g.s.sq[q] + pr.d * sz;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t at = (int64_t)(lane % 16) * ld + 4 * (lane / 16);
    const double* x = X + (int64_t)ti * E * ld + at;
    const double* y = Y + (int64_t)tj * E * ld + at;
    f64x4 acc[TS][TS] = {};
#pragma unroll 2
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
            if (I < ld && J < ld) D[(int64_t)I * ld + J] = v;
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
    int count;
    int start[CF_MAX_OPT_TENSORS + 1];
    const void* u[CF_MAX_OPT_TENSORS];
    int m[CF_MAX_OPT_TENSORS], n[CF_MAX_OPT_TENSORS];
    uint32_t tall;
    int64_t q[CF_MAX_OPT_TENSORS];      // the Q buffer, doubles from the workspace's start
};

template <typename T> __device__ __forceinline__ void finish(const StoreArgs& a, int q, int64_t i, float o)
{
    Elem<T>::store((T*)a.out[q], i, o);
}
template <typename T> __device__ __forceinline__ void finish(const ApplyArgs& a, int q, int64_t i, float o)
{
    float* w = a.w[q] + i;
    *w = fmaf(-a.rate[q], o, *w * a.keep);
}

// Block = a 64 (short side) x 64 (long side) tile of s Q U on the fp32 matrix
// cores.  Both operands are staged [64][k] or [k][64] as U lies in memory; Q,
// symmetric, is staged as it is read.  The lanes that hold neighbouring
// outputs run along the matrix's rows in memory: short-side indices are the
// matrix core's columns for a tall matrix and its rows for a wide one.
template <bool TALL, typename T, typename F>
__device__ void final_tile(const T* U, const double* Q, double s, int m, int n, int b, const F& f, int q, float* sh)
{
    const int ld = ns_ld(m), nt = (m + NS_TILE - 1) / NS_TILE;
    const int i0 = b % nt * NS_TILE, c0 = b / nt * NS_TILE;     // short, long
    float* A = sh;                       // Q: [64 short][k]
    float* B = sh + NS_PANEL;            // U: [64 long][k] for a tall matrix, [k][64 long] for a wide one
    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
    const int ws = (wave >> 1) * 32, wl = (wave & 1) * 32;      // this wave's quadrant: short, long
    f32x4 acc[2][2] = {};
    float va[NS_PV], vb[NS_PV];
    auto load = [&](int k0) {
#pragma unroll
        for (int r = 0; r < NS_PV; ++r) {
            const int i = t / NS_K + r * (NS_T / NS_K), k = k0 + t % NS_K;
            // (beyond m the buffers hold anything)
            va[r] = i0 + i < m && k < m ? (float)(Q[(int64_t)(i0 + i) * ld + k] * s) : 0.f;
        }
        if (TALL) panel_load<false>(vb, U, n, m, c0, k0, m);
        else panel_load<true>(vb, U, n, m, c0, k0, m);
    };
    load(0);
    for (int k0 = 0; k0 < m; k0 += NS_K) {
        __syncthreads();
        panel_store<false>(va, A);
        panel_store<!TALL>(vb, B);
        __syncthreads();
        if (k0 + NS_K < m) load(k0 + NS_K);
#pragma unroll
        for (int st = 0; st < NS_K / 4; ++st) {
            float a[2], c[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int kk = st * 4 + lane / 16, i = ws + r * 16 + lane % 16, j = wl + r * 16 + lane % 16;
                a[r] = A[i * NS_SK + kk];
                c[r] = B[TALL ? j * NS_SK + kk : kk * NS_SP + j];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    // rows from the first operand, columns (lanes) from the second
                    acc[x][y] = TALL ? __builtin_amdgcn_mfma_f32_16x16x4f32(c[y], a[x], acc[x][y], 0, 0, 0)
                                     : __builtin_amdgcn_mfma_f32_16x16x4f32(a[x], c[y], acc[x][y], 0, 0, 0);
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int row = 4 * (lane / 16) + v, col = lane % 16;
                const int i = i0 + ws + x * 16 + (TALL ? col : row), j = c0 + wl + y * 16 + (TALL ? row : col);
                if (i < m && j < n) finish<T>(f, q, TALL ? (int64_t)j * m + i : (int64_t)i * n + j, acc[x][y][v]);
            }
}

template <typename T, typename F>
__global__ __launch_bounds__(NS_T) void ns_final_kernel(FinalArgs g, F f, const double* ws, const double* scale)
{
    __shared__ float sh[2 * NS_PANEL];
    const int i = find(g.start, g.count, (int)blockIdx.x), b = (int)blockIdx.x - g.start[i];
    const T* U = (const T*)g.u[i];
    if (g.tall >> i & 1) final_tile<true>(U, ws + g.q[i], scale[i], g.m[i], g.n[i], b, f, i, sh);
    else final_tile<false>(U, ws + g.q[i], scale[i], g.m[i], g.n[i], b, f, i, sh);
}

// --------------------------------------------------------------- momentum
struct MomentumArgs {
    int count;
    int start[CF_MAX_OPT_TENSORS + 1];
    int64_t n[CF_MAX_OPT_TENSORS];
    const float* g[CF_MAX_OPT_TENSORS];
    float* m[CF_MAX_OPT_TENSORS];
    float* u[CF_MAX_OPT_TENSORS];       // g + mu m where nesterov, else unused
};
constexpr int MU_V = 4;                             // float4 per thread
constexpr int MU_CHUNK = NS_T * MU_V * 4;

__global__ __launch_bounds__(NS_T) void muon_momentum_kernel(MomentumArgs a, float mu, int nesterov)
{
    const int q = find(a.start, a.count, (int)blockIdx.x);
    const int64_t n = a.n[q], base = (int64_t)((int)blockIdx.x - a.start[q]) * MU_CHUNK;
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
        const int64_t ld = ns_ld(l.m[i]), nt = ld / NS_TILE, pairs = nt * (nt + 1) / 2;
        p.kc[i] = (int)std::min<int64_t>(kc, up(l.n[i], NS_K));
        p.splits[i] = (l.n[i] + p.kc[i] - 1) / p.kc[i];
        p.part[i] = at;
        at += p.splits[i] * (pairs * NS_TILE * NS_TILE + nt);
        at = (at + 31) / 32 * 32;
        p.sq[i] = at;
        at += 5 * ld * ld;
    }
    p.doubles = at;
    return p;
}

// Runs U U^T to Q; *q receives the index of the buffer that holds Q.
template <typename T>
hipError_t ns_iterate(const NsShapes& l, const NsPlan& p, const void* const* u, const NsCoef& c, double* ws, int* q,
                      hipStream_t s)
{
    GramArgs g{};
    SquareArgs sq{};
    g.count = sq.count = l.count;
    int maxm = 0;
    for (int i = 0; i < l.count; ++i) {
        const int nt = ns_ld(l.m[i]) / NS_TILE, pairs = nt * (nt + 1) / 2;
        g.u[i] = u[i];
        g.m[i] = sq.m[i] = l.m[i];
        g.n[i] = l.n[i];
        g.kc[i] = p.kc[i];
        g.splits[i] = sq.splits[i] = p.splits[i];
        g.part[i] = sq.part[i] = p.part[i];
        sq.sq[i] = p.sq[i];
        g.start[i + 1] = g.start[i] + p.splits[i] * pairs;
        sq.start[i + 1] = sq.start[i] + pairs * (NS_TILE / NS_JR);
        maxm = std::max(maxm, l.m[i]);
    }
    g.tall = l.tall;
    hipLaunchKernelGGL(ns_gram_kernel<T>, dim3((unsigned)g.start[l.count]), dim3(NS_T), 0, s, g, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ns_join_kernel, dim3((unsigned)sq.start[l.count]), dim3(NS_T), 0, s, sq, c.eps, ws, ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    RoundArgs r{};
    r.s = sq;
    r.a = c.a;
    r.b = c.b;
    r.c = c.c;
    // small matrices: many small tiles; large ones: tiles that read less
    const int edge = maxm <= 256 ? 16 : 32;
    auto round = [&](std::initializer_list<Product> ps) -> hipError_t {
        r.np = 0;
        for (const Product& x : ps) r.p[r.np++] = x;
        r.s.start[0] = 0;
        for (int i = 0; i < l.count; ++i) {
            const int nt = (l.m[i] + edge - 1) / edge;
            r.s.start[i + 1] = r.s.start[i] + r.np * (nt * (nt + 1) / 2);
        }
        const dim3 grid((unsigned)r.s.start[l.count]);
        if (edge == 16) hipLaunchKernelGGL(ns_round_kernel<1>, grid, dim3(NS_T), 0, s, r, ws);
        else hipLaunchKernelGGL(ns_round_kernel<2>, grid, dim3(NS_T), 0, s, r, ws);
        return hipGetLastError();
    };
    int A = 0, T_ = 1, P = 2, Q = 3, R = 4;      // buffers: A_k, P A, P_k, Q and a free one
    for (int k = 0; k < c.steps; ++k) {
        const bool last = k + 1 == c.steps;
        if ((e = round({{A, A, P, 1}})) != hipSuccess) return e;
        if (k == 0) {
            std::swap(P, Q);                      // Q = P_0
            if (!last && (e = round({{Q, A, T_, 0}})) != hipSuccess) return e;
            if (!last && (e = round({{T_, Q, A, 0}})) != hipSuccess) return e;
            continue;
        }
        if (last) e = round({{P, Q, R, 0}});
        else e = round({{P, A, T_, 0}, {P, Q, R, 0}});
        if (e != hipSuccess) return e;
        std::swap(Q, R);
        if (!last && (e = round({{T_, P, A, 0}})) != hipSuccess) return e;
    }
    *q = Q;
    return hipSuccess;
}

template <typename T, typename F>
hipError_t ns_final(const NsShapes& l, const NsPlan& p, const void* const* u, int q, const F& f, const double* ws,
                    hipStream_t s)
{
    FinalArgs a{};
    a.count = l.count;
    a.tall = l.tall;
    for (int i = 0; i < l.count; ++i) {
        const int64_t ld = ns_ld(l.m[i]);
        a.u[i] = u[i];
        a.m[i] = l.m[i];
        a.n[i] = l.n[i];
        a.q[i] = p.sq[i] + q * ld * ld;
        a.start[i + 1] = a.start[i] + (int)(ld / NS_TILE) * ((l.n[i] + NS_TILE - 1) / NS_TILE);
    }
    hipLaunchKernelGGL((ns_final_kernel<T, F>), dim3((unsigned)a.start[l.count]), dim3(NS_T), 0, s, a, f, ws, ws);
    return hipGetLastError();
}

}  // namespace

namespace {

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
    for (int i = 0; i < l.count; ++i) {
        if (allow_split && ns_split_size(l.m[i])) {
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

// The sizes alone fix the workspace: the larger of what any coefficients need.
size_t ns_ws_bytes(const NsShapes& l)
{
    size_t b = ns_f64_ws_bytes(l);
    const NsParts p = ns_parts(l, true);
    b = std::max(b, ns_f64_ws_bytes(p.f64));
    for (int i = 0; i < p.splits; ++i) b = std::max(b, ns_split_ws_bytes(l.m[p.split[i]], l.n[p.split[i]]));
    return b;
}

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
    const NsPlan pl = ns_plan(p.f64);
    int q = 0;
    if ((e = ns_iterate<T>(p.f64, pl, u, c, (double*)ws, &q, s)) != hipSuccess) return e;
    return ns_final<T>(p.f64, pl, u, q, f, (const double*)ws, s);
}

size_t muon_ws_bytes(const NsShapes& l, bool nesterov)
{
    size_t b = ns_ws_bytes(l);
    if (nesterov)
        for (int i = 0; i < l.count; ++i) b += up256b((size_t)l.m[i] * l.n[i] * sizeof(float));
    return b;
}

hipError_t launch_muon(const NsShapes& l, const NsCoef& c, const MuonArgs& h, float* const* w, const float* const* g,
                       float* const* m, void* ws, hipStream_t s)
{
    MomentumArgs a{};
    const float* u[CF_MAX_OPT_TENSORS];
    char* at = (char*)ws + ns_ws_bytes(l);
    a.count = l.count;
    for (int i = 0; i < l.count; ++i) {
        a.n[i] = (int64_t)l.m[i] * l.n[i];
        a.g[i] = g[i];
        a.m[i] = m[i];
        u[i] = m[i];
        if (h.nesterov) {
            a.u[i] = (float*)at;
            u[i] = a.u[i];
            at += up256b((size_t)a.n[i] * sizeof(float));
        }
        a.start[i + 1] = a.start[i] + (int)((a.n[i] + MU_CHUNK - 1) / MU_CHUNK);
    }
    hipLaunchKernelGGL(muon_momentum_kernel, dim3((unsigned)a.start[l.count]), dim3(NS_T), 0, s, a, h.momentum,
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
    const NsPlan pl = ns_plan(p.f64);
    int q = 0;
    if ((e = ns_iterate<float>(p.f64, pl, v, c, (double*)ws, &q, s)) != hipSuccess) return e;
    return ns_final<float>(p.f64, pl, v, q, f, (const double*)ws, s);
}

template hipError_t launch_newton_schulz<float>(const NsShapes&, const NsCoef&, const void* const*, void* const*,
                                                void*, hipStream_t);
template hipError_t launch_newton_schulz<uint16_t>(const NsShapes&, const NsCoef&, const void* const*, void* const*,
                                                   void*, hipStream_t);

}  // namespace cf
