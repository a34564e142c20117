// Newton-Schulz orthogonalisation of one large matrix with products of fp32
// accuracy on the fp16 matrix cores.
//
// With X0 = U / (|U|_F + eps), m <= n its short and long side (a tall matrix
// is handled as its transpose), each step is
//   A = X X^T,  P = a I + b A + c A^2,  X <- P X,
// three products, the first two symmetric (only tiles on or above the diagonal
// are computed).
//
// A value v is kept as two fp16 values of one scale s (a power of two),
//   hi = fp16(s v), lo = fp16(s v - hi),
// whose sum is s v up to 2^-23 of it (or up to half of fp16's smallest step,
// 2^-25, whichever is more), and a product is hi hi + hi lo + lo hi with fp32
// sums: the missing lo lo is below 2^-22 of a term, with random sign.  Three
// fp16 products run at a third of 2.5 PFLOP/s, five times the fp32 matrix
// rate.  The scales come from the host: the iteration's polynomial bounds every
// singular value, and so every element, of every step's X, A and P
// (ns_bounds); coefficients without a small bound take the fp64 path.
//
// Layout: a row is cut into pieces of 32 values, each one 128-byte line, the
// 32 hi and then the 32 lo.  Both operands of a product are read along their
// rows, so X is kept as [m][n] for X X^T and as [n][m] for P X; the epilogues
// write both from LDS.  Columns past the end are written as zeros, rows past
// the end are readable and hold anything: they reach only results that are not
// written.
//
// Work split: a launch has one block per CU, and the (tile, piece of the
// reduction) units in tile order are cut into equal ranges, one for each block,
// since the number of tiles seldom fills the chip evenly (136 tiles of a
// symmetric 4096 x 4096 product for 256 CUs).  A block that holds all of a
// tile's reduction writes its result; others write fp32 sums that a joining
// launch adds in the order of the blocks.  No atomics and no waiting between
// blocks: results are reproducible bit for bit.
#include "cf_internal.h"

#include <algorithm>
#include <cmath>

namespace cf {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int SP_TILE = 256;      // edge of an output tile
constexpr int SP_T = 512;         // threads: 2 x 4 waves of 128 x 64
constexpr int SP_K = 32;          // reduction values of a piece
constexpr int SP_GRID = 256;      // blocks of a product, one per CU
constexpr int SP_SB = 36;         // LDS row stride of a 32 x 32 block, floats
constexpr int SP_PART = SP_TILE * SP_TILE;      // floats of a tile's partial sums

size_t up256b(size_t b) { return (b + 255) & ~(size_t)255; }
__host__ __device__ inline int pieces(int k) { return (k + SP_K - 1) / SP_K; }

// ---------------------------------------------------------------- epilogues
// What becomes of element (i, j) of the product C, i < m, j < n.
enum SpMode {
    SP_GRAM,     // D(i, j) = D(j, i) = f C
    SP_POLY,     // D(i, j) = D(j, i) = f C + g S(i, j) + diag [i = j], S split
    SP_BOTH,     // D(i, j) = f C and DT(j, i) = f C
    SP_OUT       // the caller's matrix, f C handed to its functor
};

struct SpProduct {
    const uint16_t* p;      // [rows of C] and
    const uint16_t* r;      // [columns of C] operands, pieces(k) lines a row
    int kb;                 // pieces of the reduction
    int mt, nt;             // tiles
    int sym;
    int last;               // the reduction of tile row i ends with pieces 8 i .. 8 i + 7: a I is in P, and
                            // the sum of the small terms is rounded at its own size
    int m, n;
    float f, g, diag;
    const uint16_t* s;
    uint16_t* d;
    uint16_t* dt;
    float* part;            // [2 SP_GRID] tiles of partial sums
    int grid;
};

__host__ __device__ inline int sp_tiles(const SpProduct& q) { return q.sym ? q.mt * (q.mt + 1) / 2 : q.mt * q.nt; }
// First unit of block b.
__host__ __device__ inline int64_t sp_first(const SpProduct& q, int b)
{
    return (int64_t)sp_tiles(q) * q.kb * b / q.grid;
}

__device__ __forceinline__ void sp_tile_at(const SpProduct& q, int t, int& ti, int& tj)
{
    if (!q.sym) {
        // bands of four tile rows, column by column: a chip's worth of
        // neighbouring tiles is a rectangle that shares its operands' rows
        const int band = t / (4 * q.nt), r = t - band * 4 * q.nt, h = min(4, q.mt - 4 * band);
        ti = 4 * band + r % h;
        tj = r / h;
        return;
    }
    ti = 0;
    while (t >= q.mt - ti) {
        t -= q.mt - ti;
        ++ti;
    }
    tj = ti + t;
}

// Orders a wave's LDS accesses: what its lanes wrote is read by other lanes.
__device__ __forceinline__ void sp_wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Writes the 32 x 32 block in LDS (rows of SP_SB floats; flip: its transpose)
// to rows r0.. and piece c0 / 32 of d.  Eight lanes write a row's line.
template <int MODE>
__device__ __forceinline__ void sp_put(const float* sh, bool flip, const SpProduct& q, uint16_t* d, int kd, int r0,
                                       int c0, int rows, int cols)
{
    const int lane = (int)threadIdx.x & 63, chunk = lane & 7, k8 = (chunk & 3) * 8;
    if (c0 >= kd * SP_K) return;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 8 + lane / 8;
        if (r0 + r >= rows) continue;
        const int64_t line = ((int64_t)(r0 + r) * kd + c0 / SP_K) * 64;
        f16x8 hi = {}, lo = {}, o;
        if (MODE == SP_POLY) {
            hi = *reinterpret_cast<const f16x8*>(q.s + line + k8);
            lo = *reinterpret_cast<const f16x8*>(q.s + line + 32 + k8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = q.f * (flip ? sh[(k8 + j) * SP_SB + r] : sh[r * SP_SB + k8 + j]);
            if (MODE == SP_POLY) {
                v = fmaf(q.g, (float)hi[j] + (float)lo[j], v);
                if (r0 + r == c0 + k8 + j) v += q.diag;
            }
            if (c0 + k8 + j >= cols) v = 0.f;
            const _Float16 h = (_Float16)v;
            o[j] = chunk < 4 ? h : (_Float16)(v - (float)h);
        }
        *reinterpret_cast<f16x8*>(d + line + chunk * 8) = o;
    }
}

// The caller's row-major matrix, [m][n] or (tall) [n][m].
struct SpStore {
    void* out;
};
struct SpApply {
    float* w;
    float keep, rate;
};
template <typename T> __device__ __forceinline__ void sp_finish(const SpStore& a, int64_t i, float o)
{
    Elem<T>::store((T*)a.out, i, o);
}
template <typename T> __device__ __forceinline__ void sp_finish(const SpApply& a, int64_t i, float o)
{
    a.w[i] = fmaf(-a.rate, o, a.w[i] * a.keep);
}
struct SpNone {};
template <typename T, typename F> struct SpFinal {
    F f;
    int tall;
};

// One 32 x 32 block of the product in a wave's registers, at row block bi and
// column block bj of C; sh: this wave's 32 x SP_SB floats.
template <int MODE, typename T, typename F>
__device__ __forceinline__ void sp_block(const f32x16& acc, float* sh, const SpProduct& q, const SpFinal<T, F>& fin,
                                         int bi, int bj)
{
    const int i0 = bi * 32, j0 = bj * 32, lane = (int)threadIdx.x & 63;
    if (i0 >= q.m || j0 >= q.n || (q.sym && bi > bj)) return;
    // register r of a lane: row 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
#pragma unroll
    for (int r = 0; r < 16; ++r) sh[(8 * (r / 4) + 4 * (lane / 32) + r % 4) * SP_SB + lane % 32] = acc[r];
    sp_wave_sync();
    if constexpr (MODE == SP_GRAM || MODE == SP_POLY) {
        sp_put<MODE>(sh, false, q, q.d, pieces(q.n), i0, j0, q.m, q.n);
        if (bi < bj) sp_put<MODE>(sh, true, q, q.d, pieces(q.n), j0, i0, q.m, q.n);
    } else if constexpr (MODE == SP_BOTH) {
        sp_put<MODE>(sh, false, q, q.d, pieces(q.n), i0, j0, q.m, q.n);
        sp_put<MODE>(sh, true, q, q.dt, pieces(q.m), j0, i0, q.n, q.m);
    } else {
        const int c = lane % 32, x0 = fin.tall ? j0 : i0, y0 = fin.tall ? i0 : j0;
        const int rows = fin.tall ? q.n : q.m, cols = fin.tall ? q.m : q.n;
#pragma unroll
        for (int it = 0; it < 16; ++it) {
            const int r = it * 2 + lane / 32;
            if (x0 + r < rows && y0 + c < cols)
                sp_finish<T>(fin.f, (int64_t)(x0 + r) * cols + y0 + c,
                             q.f * (fin.tall ? sh[c * SP_SB + r] : sh[r * SP_SB + c]));
        }
    }
    sp_wave_sync();
}

// ------------------------------------------------------------------ product
// A stage of one piece: 256 lines of p, then 256 of r.  The 16-byte chunk c of
// row r's line lies at slot c ^ (r / 2 & 7): sixteen rows read at one chunk
// fall on all banks.
constexpr int SP_STAGE = 2 * SP_TILE * 8;      // 16-byte chunks

__device__ __forceinline__ void sp_load(uint4* stage, const uint16_t* p, const uint16_t* r, int64_t ld, int piece)
{
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int q = wave * 4 + i % 4;      // eight rows of the panel
        const int row = q * 8 + lane / 8, chunk = (lane & 7) ^ ((row >> 1) & 7);
        const uint16_t* src = (i < 4 ? p : r) + row * ld + (int64_t)piece * 64 + chunk * 8;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                         (__attribute__((address_space(3))) void*)(stage + (i / 4) * (SP_TILE * 8) + q * 64),
                                         16, 0, 0);
    }
}

__device__ __forceinline__ void sp_multiply(const uint4* stage, f32x16 (&acc)[4][2])
{
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int wi = (wave >> 2) * 128, wj = (wave & 3) * 64;
    const int swz = (lane >> 1) & 7;
    const f16x8* A = reinterpret_cast<const f16x8*>(stage) + (wi + lane % 32) * 8;
    const f16x8* B = reinterpret_cast<const f16x8*>(stage) + (SP_TILE + wj + lane % 32) * 8;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int ch = (s * 2 + lane / 32) ^ swz, cl = (4 + s * 2 + lane / 32) ^ swz;
        f16x8 ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            bh[j] = B[j * 256 + ch];
            bl[j] = B[j * 256 + cl];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ah[i] = A[i * 256 + ch];
            al[i] = A[i * 256 + cl];
        }
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x == 2 ? al[i] : ah[i], x == 1 ? bl[j] : bh[j],
                                                                      acc[i][j], 0, 0, 0);
    }
}

// Barrier after which every wave's loads into LDS have landed.
__device__ __forceinline__ void sp_landed()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt 0
    __syncthreads();
}

template <int MODE, typename T, typename F>
__global__ __launch_bounds__(SP_T, 2) void sp_product_kernel(SpProduct q, SpFinal<T, F> fin)
{
    __shared__ uint4 s0[SP_STAGE];
    __shared__ uint4 s1[SP_STAGE];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int b = (int)xcd_remap(blockIdx.x, (uint32_t)q.grid);
    const int64_t u1 = sp_first(q, b + 1), ld = (int64_t)q.kb * 64;
    int64_t u = sp_first(q, b);
    for (int seg = 0; u < u1; seg = 1) {
        const int t = (int)(u / q.kb), k0 = (int)(u - (int64_t)t * q.kb);
        const int len = (int)min((int64_t)(q.kb - k0), u1 - u);
        int ti, tj;
        sp_tile_at(q, t, ti, tj);
        const uint16_t* p = q.p + (int64_t)ti * SP_TILE * ld;
        const uint16_t* r = q.r + (int64_t)tj * SP_TILE * ld;
        int piece = k0 + (q.last ? (ti + 1) * (SP_TILE / SP_K) : 0);
        piece %= q.kb;
        f32x16 acc[4][2] = {};
        auto next = [&] { piece = piece + 1 == q.kb ? 0 : piece + 1; };
        sp_load(s0, p, r, ld, piece);
        for (int i = 0; i < len; i += 2) {
            sp_landed();
            next();
            if (i + 1 < len) sp_load(s1, p, r, ld, piece);
            sp_multiply(s0, acc);
            if (i + 1 < len) {
                sp_landed();
                next();
                if (i + 2 < len) sp_load(s0, p, r, ld, piece);
                sp_multiply(s1, acc);
            }
        }
        const int wi = (wave >> 2) * 4, wj = (wave & 3) * 2;
        __syncthreads();
        if (len == q.kb) {
            float* sh = reinterpret_cast<float*>(s0) + wave * (32 * SP_SB);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    sp_block<MODE>(acc[i][j], sh, q, fin, ti * 8 + wi + i, tj * 8 + wj + j);
            __syncthreads();
        } else {
            // [block of 32 x 32][quarter of a lane's registers][lane]
            float4* out = reinterpret_cast<float4*>(q.part + ((int64_t)b * 2 + seg) * SP_PART);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        out[(((wi + i) * 8 + wj + j) * 4 + v) * 64 + lane] =
                            make_float4(acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                                        acc[i][j][4 * v + 3]);
        }
        u += len;
    }
}

// Adds the partial sums of the tiles that several blocks share.  A wave takes
// one 32 x 32 block.
template <int MODE, typename T, typename F>
__global__ __launch_bounds__(256) void sp_join_kernel(SpProduct q, SpFinal<T, F> fin)
{
    __shared__ float shared[4][32 * SP_SB];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int t = (int)blockIdx.x / 16, blk = (int)blockIdx.x % 16 * 4 + wave;
    const int64_t units = (int64_t)sp_tiles(q) * q.kb, ua = (int64_t)t * q.kb, ub = ua + q.kb - 1;
    // the block that holds unit u: the largest b with first(b) <= u
    auto holder = [&](int64_t u) {
        int b = (int)(u * q.grid / units);
        while (sp_first(q, b) > u) --b;
        while (sp_first(q, b + 1) <= u) ++b;
        return b;
    };
    const int ba = holder(ua), bb = holder(ub);
    if (ba == bb) return;
    f32x16 acc = {};
    for (int b = ba; b <= bb; ++b) {
        const int seg = sp_first(q, b) / q.kb == t ? 0 : 1;
        const float4* in = reinterpret_cast<const float4*>(q.part + ((int64_t)b * 2 + seg) * SP_PART) + blk * 256 + lane;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float4 w = in[v * 64];
            acc[4 * v] += w.x;
            acc[4 * v + 1] += w.y;
            acc[4 * v + 2] += w.z;
            acc[4 * v + 3] += w.w;
        }
    }
    int ti, tj;
    sp_tile_at(q, t, ti, tj);
    sp_block<MODE>(acc, shared[wave], q, fin, ti * 8 + blk / 8, tj * 8 + blk % 8);
}

template <int MODE, typename T = float, typename F = SpNone>
hipError_t sp_run(SpProduct q, const SpFinal<T, F>& fin, hipStream_t s)
{
    const int64_t units = (int64_t)sp_tiles(q) * q.kb;
    q.grid = (int)std::min<int64_t>(SP_GRID, (units + 1) / 2);
    hipLaunchKernelGGL((sp_product_kernel<MODE, T, F>), dim3((unsigned)q.grid), dim3(SP_T), 0, s, q, fin);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (units % q.grid == 0 && units / q.grid % q.kb == 0) return e;      // whole tiles everywhere
    hipLaunchKernelGGL((sp_join_kernel<MODE, T, F>), dim3((unsigned)sp_tiles(q) * 16), dim3(256), 0, s, q, fin);
    return hipGetLastError();
}

// ------------------------------------------------------------ norm and split
constexpr int SP_NORM = 512;      // blocks of the norm

__device__ __forceinline__ double sp_block_sum(double v, double* sh)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((sh[0] + sh[1]) + sh[2]) + sh[3];
}

template <typename T> __global__ __launch_bounds__(256) void sp_norm_kernel(const T* u, int64_t n, double* part)
{
    __shared__ double sh[4];
    constexpr int V = 16 / (int)sizeof(T);
    double a = 0.0;
    const int64_t vecs = n / V;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += SP_NORM * 256) {
        T v[V];
        __builtin_memcpy(v, u + i * V, 16);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double d = (double)Elem<T>::load(v, j);
            a = fma(d, d, a);
        }
    }
    if (blockIdx.x == 0 && (int64_t)threadIdx.x < n - vecs * V) {
        const double d = (double)Elem<T>::load(u, vecs * V + threadIdx.x);
        a = fma(d, d, a);
    }
    a = sp_block_sum(a, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// X0 = U / (|U|_F + eps) in both layouts; a wave takes 32 x 32 elements.
template <typename T>
__global__ __launch_bounds__(256) void sp_split_kernel(const T* u, int rows, int cols, const double* part, float eps,
                                                       float scale, SpProduct q, int tall)
{
    __shared__ double red[4];
    __shared__ float shared[4][32 * SP_SB];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    double a = 0.0;
    for (int i = (int)threadIdx.x; i < SP_NORM; i += 256) a += part[i];
    const double s = (double)scale / (sqrt(sp_block_sum(a, red)) + (double)eps);
    const int bc = pieces(cols);
    const int64_t blk = (int64_t)blockIdx.x * 4 + wave;
    const int64_t br = blk / bc;
    if (br >= pieces(rows)) return;
    const int r0 = (int)br * 32, c0 = (int)(blk - br * bc) * 32;
    float* sh = shared[wave];
#pragma unroll
    for (int it = 0; it < 16; ++it) {
        const int r = it * 2 + lane / 32, c = lane % 32;
        float v = 0.f;
        if (r0 + r < rows && c0 + c < cols) v = (float)((double)Elem<T>::load(u, (int64_t)(r0 + r) * cols + c0 + c) * s);
        sh[r * SP_SB + c] = v;
    }
    sp_wave_sync();
    sp_put<SP_BOTH>(sh, false, q, tall ? q.dt : q.d, bc, r0, c0, rows, cols);
    sp_put<SP_BOTH>(sh, true, q, tall ? q.d : q.dt, pieces(rows), c0, r0, cols, rows);
}

// -------------------------------------------------------------------- plan
// Bounds of the singular values of X_k and of the eigenvalues of P_k.
struct SpBounds {
    bool fits;
    double x[33], p[32];
};

SpBounds ns_bounds(const NsCoef& c)
{
    SpBounds r{};
    const double a = c.a, b = c.b, cc = c.c;
    r.x[0] = 1.0;
    r.fits = true;
    for (int k = 0; k < c.steps; ++k) {
        const double t1 = r.x[k] * r.x[k];      // lambda = sigma^2 in [0, t1]
        auto pol = [&](double t) { return a + b * t + cc * t * t; };
        double p = std::max(std::fabs(a), std::fabs(pol(t1)));
        if (cc != 0.0 && -b / (2 * cc) > 0.0 && -b / (2 * cc) < t1) p = std::max(p, std::fabs(pol(-b / (2 * cc))));
        double x = std::sqrt(t1) * std::fabs(pol(t1));
        // extremes of sigma (a + b t + c t^2): a + 3 b t + 5 c t^2 = 0
        const double disc = 9 * b * b - 20 * a * cc;
        if (cc != 0.0 && disc >= 0.0) {
            for (int sgn = -1; sgn <= 1; sgn += 2) {
                const double t = (-3 * b + sgn * std::sqrt(disc)) / (10 * cc);
                if (t > 0.0 && t < t1) x = std::max(x, std::sqrt(t) * std::fabs(pol(t)));
            }
        } else if (cc == 0.0 && b != 0.0) {
            const double t = -a / (3 * b);
            if (t > 0.0 && t < t1) x = std::max(x, std::sqrt(t) * std::fabs(pol(t)));
        }
        r.p[k] = p;
        r.x[k + 1] = 1.01 * x;      // (roundings)
        // a factor of 16 in X is one of 256 in A: still 2^-25 / 2^7 absolute
        if (!(r.x[k + 1] <= 16.0) || !(p <= 256.0)) r.fits = false;
        if (!r.fits) break;
    }
    return r;
}

// The power of two that brings a bound into (16384, 32768].
double sp_scale(double bound) { return std::ldexp(1.0, (int)std::floor(std::log2(32768.0 / std::max(bound, 1e-3)))); }

struct SpLayout {
    size_t norm, x, xt[2], a, p, part, bytes;
};
SpLayout sp_layout(int m, int n)
{
    SpLayout l{};
    auto rows = [](int v) { return ((size_t)v + SP_TILE - 1) / SP_TILE * SP_TILE; };
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t r = at;
        at += up256b(b);
        return r;
    };
    l.norm = take(SP_NORM * sizeof(double));
    l.x = take(rows(m) * pieces(n) * 128);
    l.xt[0] = take(rows(n) * pieces(m) * 128);
    l.xt[1] = take(rows(n) * pieces(m) * 128);
    l.a = take(rows(m) * pieces(m) * 128);
    l.p = take(rows(m) * pieces(m) * 128);
    l.part = take((size_t)2 * SP_GRID * SP_PART * sizeof(float));
    l.bytes = at;
    return l;
}

template <typename T, typename F>
hipError_t sp_newton_schulz(int m, int n, bool tall, const NsCoef& c, const T* u, const F& f, char* ws, hipStream_t s)
{
    const SpLayout l = sp_layout(m, n);
    const SpBounds bd = ns_bounds(c);
    double* norm = (double*)(ws + l.norm);
    uint16_t* X = (uint16_t*)(ws + l.x);
    uint16_t* XT[2] = {(uint16_t*)(ws + l.xt[0]), (uint16_t*)(ws + l.xt[1])};
    uint16_t* A = (uint16_t*)(ws + l.a);
    uint16_t* P = (uint16_t*)(ws + l.p);
    const int rows = tall ? n : m, cols = tall ? m : n;
    SpProduct q{};
    q.part = (float*)(ws + l.part);
    double sx = sp_scale(bd.x[0]);

    hipLaunchKernelGGL(sp_norm_kernel<T>, dim3(SP_NORM), dim3(256), 0, s, u, (int64_t)m * n, norm);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    q.f = 1.f;
    q.d = X;
    q.dt = XT[0];
    const int64_t blocks = ((int64_t)pieces(rows) * pieces(cols) + 3) / 4;
    hipLaunchKernelGGL(sp_split_kernel<T>, dim3((unsigned)blocks), dim3(256), 0, s, u, rows, cols, norm, c.eps,
                       (float)sx, q, (int)tall);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    const int mt = (m + SP_TILE - 1) / SP_TILE, nt = (n + SP_TILE - 1) / SP_TILE;
    const SpFinal<float, SpNone> none{};
    for (int k = 0; k < c.steps; ++k) {
        const double sa = sp_scale(1.01 * bd.x[k] * bd.x[k]), sp = sp_scale(1.01 * bd.p[k]);
        q.p = q.r = X;
        q.kb = pieces(n);
        q.mt = q.nt = mt;
        q.sym = 1;
        q.last = 0;
        q.m = q.n = m;
        q.f = (float)(sa / (sx * sx));
        q.d = A;
        if ((e = sp_run<SP_GRAM>(q, none, s)) != hipSuccess) return e;
        q.p = q.r = q.s = A;
        q.kb = pieces(m);
        q.f = (float)(sp * c.c / (sa * sa));
        q.g = (float)(sp * c.b / sa);
        q.diag = (float)(sp * c.a);
        q.d = P;
        if ((e = sp_run<SP_POLY>(q, none, s)) != hipSuccess) return e;
        q.p = P;
        q.r = XT[k & 1];
        q.nt = nt;
        q.sym = 0;
        q.last = 1;
        q.n = n;
        if (k + 1 < c.steps) {
            const double sn = sp_scale(bd.x[k + 1]);
            q.f = (float)(sn / (sp * sx));
            q.d = X;
            q.dt = XT[(k + 1) & 1];
            if ((e = sp_run<SP_BOTH>(q, none, s)) != hipSuccess) return e;
            sx = sn;
        } else {
            q.f = (float)(1.0 / (sp * sx));
            const SpFinal<T, F> fin{f, (int)tall};
            if ((e = sp_run<SP_OUT>(q, fin, s)) != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace

constexpr int SP_MIN = 512;

bool ns_split_size(int m, int n) { return m >= SP_MIN; }
bool ns_split_coef(const NsCoef& c) { return ns_bounds(c).fits; }
size_t ns_split_ws_bytes(int m, int n) { return sp_layout(m, n).bytes; }

template <typename T>
hipError_t launch_ns_split(int m, int n, bool tall, const NsCoef& c, const T* x, T* out, void* ws, hipStream_t s)
{
    return sp_newton_schulz<T>(m, n, tall, c, x, SpStore{out}, (char*)ws, s);
}
hipError_t launch_ns_split_apply(int m, int n, bool tall, const NsCoef& c, const float* x, float* w, float keep,
                                 float rate, void* ws, hipStream_t s)
{
    return sp_newton_schulz<float>(m, n, tall, c, x, SpApply{w, keep, rate}, (char*)ws, s);
}

template hipError_t launch_ns_split<float>(int, int, bool, const NsCoef&, const float*, float*, void*, hipStream_t);
template hipError_t launch_ns_split<uint16_t>(int, int, bool, const NsCoef&, const uint16_t*, uint16_t*, void*,
                                              hipStream_t);

}  // namespace cf
