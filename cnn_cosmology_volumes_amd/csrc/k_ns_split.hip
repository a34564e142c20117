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
// (ns_bounds); coefficients without a small bound take the fp64 path.  Where
// |U| is below eps, X_0 is small and so are the next steps' X, by more than
// the host can know: a power of two on top of each step's scale, found on the
// device (sp_lift), keeps their digits.
//
// Layout: a row is cut into pieces of 32 values, each one 128-byte line, the
// 32 hi and then the 32 lo.  Both operands of a product are read along their
// rows, so X is kept as [m][n] for X X^T and as [n][m] for P X; the epilogues
// write both from LDS.  Columns past the end are written as zeros, rows past
// the end are readable and hold anything: they reach only results that are not
// written.
//
// Work split: tiles of 64 x 64, a block each, where they are few (the block's
// waves share the reduction), else of 128 or 256 (sp_plan gives the rule).
// There a launch has one block per CU, and the (tile, piece of the reduction)
// units in tile order are cut into equal ranges, one for each block, since the
// number of tiles seldom fills the chip evenly (136 tiles of a symmetric
// 4096 x 4096 product for 256 CUs).  A block that holds all of a tile's
// reduction writes its result; others write fp32 sums that a joining launch
// adds in the order of the blocks.  No atomics and no waiting between blocks:
// results are reproducible bit for bit.
//
// What bounds it: 4096 x 4096 takes 3820 to 3890 us by card.  In a kernel trace,
// which adds up to 8% more, each P X takes 350 (1.18 PFLOP/s of fp16 products; a
// library fp16 product of that size reaches 1.26) with the matrix cores busy 77%
// of the cycles at 1.5 GHz: the chip's power.  2048 x 2048 takes 757 to 805 us;
// in a trace of 5 to 10% more, 56 to 59 for each P X (55% at 1.6 GHz) and 49 to
// 53 for each symmetric product, 13 to 15 of them the joining launch.
#include "cf_internal.h"

#include <algorithm>
#include <cmath>

namespace cf {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int SP_TILE = 256;      // largest edge of an output tile
constexpr int SP_K = 32;          // reduction values of a piece
constexpr int SP_GRID = 256;      // blocks of a product whose tiles are shared, one per CU
constexpr int SP_SB = 36;         // LDS row stride of a 32 x 32 block, floats
constexpr int SP_PART = SP_TILE * SP_TILE;      // floats of a tile's partial sums

size_t up256b(size_t b) { return (b + 255) & ~(size_t)255; }
__host__ __device__ inline int pieces(int k) { return (k + SP_K - 1) / SP_K; }
// Lines from one row to the next: an odd number, or the rows of a piece would
// share few memory channels.
__host__ __device__ inline int row_lines(int kb) { return kb | 1; }

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
    int tile, mt, nt;       // edge of a tile, tiles
    int sym;
    int last;               // a tile's reduction ends with its own rows' pieces: a I is in P, and the sum of
                            // the small terms is rounded at its own size
    int m, n;
    float f, g, diag;
    const float* lift;      // what f and g are multiplied by (but for SP_GRAM)
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
// SP_POLY adds S, and leaves the sums in LDS for the mirror; else the block is
// multiplied by f.
template <int MODE>
__device__ __forceinline__ void sp_put(float* sh, bool flip, float f, float g, const SpProduct& q, uint16_t* d, int kd,
                                       int r0, int c0, int rows, int cols)
{
    const int lane = (int)threadIdx.x & 63, chunk = lane & 7, k8 = (chunk & 3) * 8;
    if (c0 >= kd * SP_K) return;
    auto line = [&](int it) {
        return ((int64_t)min(r0 + it * 8 + lane / 8, rows - 1) * row_lines(kd) + c0 / SP_K) * 64;
    };
    f16x8 hi[4], lo[4], o[4];
    float sums[4][8];
    if (MODE == SP_POLY)
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            hi[it] = *reinterpret_cast<const f16x8*>(q.s + line(it) + k8);
            lo[it] = *reinterpret_cast<const f16x8*>(q.s + line(it) + 32 + k8);
        }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = it * 8 + lane / 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = f * (flip ? sh[(k8 + j) * SP_SB + r] : sh[r * SP_SB + k8 + j]);
            if (MODE == SP_POLY) {
                v = fmaf(g, (float)hi[it][j] + (float)lo[it][j], v);
                if (r0 + r == c0 + k8 + j) v += q.diag;
                sums[it][j] = v;
            }
            if (c0 + k8 + j >= cols) v = 0.f;
            const _Float16 h = (_Float16)v;
            o[it][j] = chunk < 4 ? h : (_Float16)(v - (float)h);
        }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it)
        if (r0 + it * 8 + lane / 8 < rows) *reinterpret_cast<f16x8*>(d + line(it) + chunk * 8) = o[it];
    if (MODE == SP_POLY && chunk < 4)
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int j = 0; j < 8; ++j) sh[(it * 8 + lane / 8) * SP_SB + k8 + j] = sums[it][j];
}

// The caller's row-major matrix, [m][n] or (tall) [n][m].
struct SpStore {
    void* out;
};
struct SpApply {
    float* w;
    float keep, rate;
};
// Done in three passes over a block's elements: loads, results, stores.  The
// compiler may not move a load past a store, and a wait for a load between
// stores would wait for the stores too.
__device__ __forceinline__ float sp_before(const SpStore&, int64_t) { return 0.f; }
__device__ __forceinline__ float sp_before(const SpApply& a, int64_t i) { return a.w[i]; }
__device__ __forceinline__ float sp_result(const SpStore&, float o, float) { return o; }
__device__ __forceinline__ float sp_result(const SpApply& a, float o, float w) { return fmaf(-a.rate, o, w * a.keep); }
template <typename T> __device__ __forceinline__ void sp_finish(const SpStore& a, int64_t i, float v)
{
    Elem<T>::store((T*)a.out, i, v);
}
template <typename T> __device__ __forceinline__ void sp_finish(const SpApply& a, int64_t i, float v) { a.w[i] = v; }
struct SpNone {};
template <typename T, typename F> struct SpFinal {
    F f;
    int tall;
};

// f and g of a product, with the lifts of its operands and its result.
template <int MODE> __device__ __forceinline__ float2 sp_factors(const SpProduct& q)
{
    if (MODE == SP_GRAM) return make_float2(q.f, 0.f);
    return make_float2(q.f * q.lift[0], MODE == SP_POLY ? q.g * q.lift[1] : 0.f);
}

// One 32 x 32 block of the product in a wave's registers, at row block bi and
// column block bj of C; sh: this wave's 32 x SP_SB floats; fg: sp_factors.
template <int MODE, typename T, typename F>
__device__ __forceinline__ void sp_block(const f32x16& acc, float* sh, const SpProduct& q, const SpFinal<T, F>& fin,
                                         float2 fg, int bi, int bj)
{
    const int i0 = bi * 32, j0 = bj * 32, lane = (int)threadIdx.x & 63;
    if (i0 >= q.m || j0 >= q.n || (q.sym && bi > bj)) return;
    // register r of a lane: row 8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
#pragma unroll
    for (int r = 0; r < 16; ++r) sh[(8 * (r / 4) + 4 * (lane / 32) + r % 4) * SP_SB + lane % 32] = acc[r];
    sp_wave_sync();
    if constexpr (MODE == SP_GRAM || MODE == SP_POLY) {
        sp_put<MODE>(sh, false, fg.x, fg.y, q, q.d, pieces(q.n), i0, j0, q.m, q.n);
        if (bi < bj) {
            // (S is symmetric: the mirror's sums are the same)
            if (MODE == SP_POLY) sp_wave_sync();
            sp_put<SP_GRAM>(sh, true, MODE == SP_POLY ? 1.f : fg.x, 0.f, q, q.d, pieces(q.n), j0, i0, q.m, q.n);
        }
    } else if constexpr (MODE == SP_BOTH) {
        sp_put<MODE>(sh, false, fg.x, 0.f, q, q.d, pieces(q.n), i0, j0, q.m, q.n);
        sp_put<MODE>(sh, true, fg.x, 0.f, q, q.dt, pieces(q.m), j0, i0, q.n, q.m);
    } else {
        const int c = lane % 32, x0 = fin.tall ? j0 : i0, y0 = fin.tall ? i0 : j0;
        const int rows = fin.tall ? q.n : q.m, cols = fin.tall ? q.m : q.n;
        float w[16];
#pragma unroll
        for (int it = 0; it < 16; ++it) {
            const int x = min(x0 + it * 2 + lane / 32, rows - 1), y = min(y0 + c, cols - 1);
            w[it] = sp_before(fin.f, (int64_t)x * cols + y);
        }
#pragma unroll
        for (int it = 0; it < 16; ++it) {
            const int r = it * 2 + lane / 32;
            w[it] = sp_result(fin.f, fg.x * (fin.tall ? sh[c * SP_SB + r] : sh[r * SP_SB + c]), w[it]);
            asm volatile("" : "+v"(w[it]));      // computed before the stores
        }
#pragma unroll
        for (int it = 0; it < 16; ++it) {
            const int r = it * 2 + lane / 32;
            if (x0 + r < rows && y0 + c < cols) sp_finish<T>(fin.f, (int64_t)(x0 + r) * cols + y0 + c, w[it]);
        }
    }
    sp_wave_sync();
}

// ------------------------------------------------------------------ product
// Two shapes of a block of 8 waves, with two stages in LDS (128 KB):
//   256: waves of 128 x 64, a stage holds a piece;
//   128: two groups of waves of 64 x 64, each with every other piece of the
//        tile: a stage holds a piece for each, and the two sums are added in
//        the end.  (One group with four stages takes the same time at 2048 x
//        2048, 763 us: what bounds these products is power, in which a byte
//        from L2 to LDS costs as much as the products made of it.  512 x 4096
//        takes 250 us that way, 255 this way, 2500 x 2500 1223 and 1200.)
template <int TILE> struct SpShape {
    static constexpr int WAVES = 8;
    static constexpr int GW = TILE / 32;            // waves of a group
    static constexpr int GROUPS = WAVES / GW;
    static constexpr int WC = GW / 2;               // waves side by side
    static constexpr int MI = TILE / 64;            // a wave's 32 x 32 blocks: rows,
    static constexpr int NJ = 2;                    // columns
    static constexpr int LINES = 2 * TILE * 8;      // 16-byte chunks of a piece
    static constexpr int CHUNKS = GROUPS * LINES;   // and of a stage
};

// Raw 32-bit words from p on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t sp_rsrc(const void* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0xffffffffu, 0x00020000);
}

// A piece in a stage: TILE lines of p, then TILE of r.  The 16-byte chunk c of row r's
// line lies at slot c ^ (r / 2 & 7): sixteen rows read at one chunk fall on all
// banks.
//
// Starts the loads of a stage; a wave's instruction takes eight rows' lines of
// its group's piece.
// src: this wave's first row of p and of r at that piece, off: the lane's
// offset in bytes from there, for an even and an odd group of eight rows.
template <int TILE>
__device__ __forceinline__ void sp_load(uint4* stage, const char* const (&src)[2], const uint32_t (&off)[2], int64_t ld)
{
    using S = SpShape<TILE>;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    uint4* to = stage + wave / S::GW * S::LINES + wave % S::GW * 4 * 64;
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                sp_rsrc(src[o]), (__attribute__((address_space(3))) void*)(to + o * (TILE * 8) + i * 64), 16, off[i & 1],
                i * 8 * (uint32_t)ld, 0, 0);
}
constexpr int SP_LOADS = 8;      // instructions of sp_load

// One half (16 values) of a piece for a wave's part of the tile.
template <int TILE> struct SpFrag {
    f16x8 ah[SpShape<TILE>::MI], al[SpShape<TILE>::MI], bh[SpShape<TILE>::NJ], bl[SpShape<TILE>::NJ];
};
template <int TILE> __device__ __forceinline__ void sp_read(SpFrag<TILE>& f, const uint4* stage, int half)
{
    using S = SpShape<TILE>;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, w = wave % S::GW;
    const int wi = w / S::WC * S::MI * 32, wj = w % S::WC * S::NJ * 32;
    stage += wave / S::GW * S::LINES;
    const int swz = (lane >> 1) & 7;
    const int ch = (half * 2 + lane / 32) ^ swz, cl = (4 + half * 2 + lane / 32) ^ swz;
    const f16x8* A = reinterpret_cast<const f16x8*>(stage) + (wi + lane % 32) * 8;
    const f16x8* B = reinterpret_cast<const f16x8*>(stage) + (TILE + wj + lane % 32) * 8;
#pragma unroll
    for (int j = 0; j < S::NJ; ++j) {
        f.bh[j] = B[j * 256 + ch];
        f.bl[j] = B[j * 256 + cl];
    }
#pragma unroll
    for (int i = 0; i < S::MI; ++i) {
        f.ah[i] = A[i * 256 + ch];
        f.al[i] = A[i * 256 + cl];
    }
}
template <int TILE>
__device__ __forceinline__ void sp_multiply(const SpFrag<TILE>& f, f32x16 (&acc)[SpShape<TILE>::MI][SpShape<TILE>::NJ])
{
    using S = SpShape<TILE>;
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int j = 0; j < S::NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x == 2 ? f.al[i] : f.ah[i], x == 1 ? f.bl[j] : f.bh[j],
                                                                  acc[i][j], 0, 0, 0);
}
// The LDS reads of the next half, and the loads of a piece, among the matrix
// instructions of this one.
template <int TILE, bool LOADS> __device__ __forceinline__ void sp_interleave()
{
    using S = SpShape<TILE>;
    constexpr int reads = 2 * (S::MI + S::NJ);
#pragma unroll
    for (int i = 0; i < reads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (LOADS && i < SP_LOADS) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 3 * S::MI * S::NJ - reads, 0);
}

// Barrier after which every wave's loads into LDS have landed but for the
// newest AHEAD pieces', and its LDS reads are done.
template <int AHEAD> __device__ __forceinline__ void sp_landed()
{
    asm volatile("" ::: "memory");
    constexpr int n = AHEAD * SP_LOADS;                                      // vmcnt: bits 0-3 and 14-15;
    __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);          // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int TILE, int MODE, typename T, typename F>
__global__ __launch_bounds__(64 * SpShape<TILE>::WAVES) void sp_product_kernel(SpProduct q, SpFinal<T, F> fin)
{
    using S = SpShape<TILE>;
    // (arrays of their own: loads into one do not hold up reads of another)
    __shared__ uint4 s0[S::CHUNKS];
    __shared__ uint4 s1[S::CHUNKS];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int group = wave / S::GW, w = wave % S::GW;
    const int b = (int)xcd_remap(blockIdx.x, (uint32_t)q.grid);
    const float2 fg = sp_factors<MODE>(q);
    const int64_t u1 = sp_first(q, b + 1), ld = (int64_t)row_lines(q.kb) * 128;      // bytes from row to row
    uint32_t off[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        off[i] = (uint32_t)(lane / 8 * ld) + ((uint32_t)(lane & 7) ^ (uint32_t)(i * 4 + lane / 16)) * 16;
    int64_t u = sp_first(q, b);
    for (int seg = 0; u < u1; seg = 1) {
        const int t = (int)(u / q.kb), k0 = (int)(u - (int64_t)t * q.kb);
        const int len = (int)min((int64_t)(q.kb - k0), u1 - u);
        int ti, tj;
        sp_tile_at(q, t, ti, tj);
        int piece = (k0 + group + (q.last ? (ti + 1) * (TILE / SP_K) : 0)) % q.kb;
        const char* src[2] = {(const char*)q.p + ((int64_t)ti * TILE + w * 32) * ld + (int64_t)piece * 128,
                              (const char*)q.r + ((int64_t)tj * TILE + w * 32) * ld + (int64_t)piece * 128};
        f32x16 acc[S::MI][S::NJ] = {};
        int left = (len - group + S::GROUPS - 1) / S::GROUPS;      // the group's pieces whose loads have not begun
        // (past the last piece it is loaded again and not used: the waits count on a load every time)
        auto load = [&](uint4* stage) {
            sp_load<TILE>(stage, src, off, ld);
            const bool wrap = piece + S::GROUPS >= q.kb, more = --left > 0;
            const int64_t step = more ? S::GROUPS * 128 - (wrap ? (int64_t)q.kb * 128 : 0) : 0;
            piece += S::GROUPS - (wrap ? q.kb : 0);
            src[0] += step;
            src[1] += step;
        };
        // The reads of a half are in flight while the half before it is multiplied, across the barrier too.
        SpFrag<TILE> f0, f1;
        load(s0);
        load(s1);
        sp_landed<1>();
        sp_read<TILE>(f0, s0, 0);
        auto pieces_of = [&](uint4* cur, uint4* nxt) {
            sp_read<TILE>(f1, cur, 1);
            sp_multiply<TILE>(f0, acc);
            sp_interleave<TILE, false>();
            sp_landed<0>();
            load(cur);
            sp_read<TILE>(f0, nxt, 0);      // (past the last piece: read and not used)
            sp_multiply<TILE>(f1, acc);
            sp_interleave<TILE, true>();
        };
        // the last one of an odd number is the first group's
        auto odd_piece = [&](uint4* cur) {
            if (S::GROUPS == 1 || group || !(len & 1)) return;
            sp_read<TILE>(f1, cur, 1);
            sp_multiply<TILE>(f0, acc);
            sp_multiply<TILE>(f1, acc);
        };
        const int stages = len / S::GROUPS;
        for (int i = 0; i < stages / 2; ++i) {
            pieces_of(s0, s1);
            pieces_of(s1, s0);
        }
        if (stages & 1) {
            pieces_of(s0, s1);
            odd_piece(s1);
        } else {
            odd_piece(s0);
        }
        constexpr int E = TILE / 32;
        const int wi = w / S::WC * S::MI, wj = w % S::WC * S::NJ;
        sp_landed<0>();
        // A wave ends with DONE rows of blocks, from row i0 of its own: with two groups, each hands the other the sums
        // of one of its two rows.
        constexpr int DONE = S::MI / S::GROUPS;
        const int i0 = S::GROUPS == 1 ? 0 : group;
        f32x16 total[DONE][S::NJ];
        if constexpr (S::GROUPS == 1) {
#pragma unroll
            for (int i = 0; i < DONE; ++i)
#pragma unroll
                for (int j = 0; j < S::NJ; ++j) total[i][j] = acc[i][j];
        } else {
            float4* swap = reinterpret_cast<float4*>(s0) + lane;
            auto slot = [&](int i, int j, int v) { return (((w * 2 + i) * S::NJ + j) * 4 + v) * 64; };
#pragma unroll
            for (int j = 0; j < S::NJ; ++j) {
                const f32x16 give = group ? acc[0][j] : acc[1][j];
                total[0][j] = group ? acc[1][j] : acc[0][j];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    swap[slot(1 - group, j, v)] = make_float4(give[4 * v], give[4 * v + 1], give[4 * v + 2],
                                                              give[4 * v + 3]);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < S::NJ; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float4 x = swap[slot(group, j, v)];
                    total[0][j][4 * v] += x.x;
                    total[0][j][4 * v + 1] += x.y;
                    total[0][j][4 * v + 2] += x.z;
                    total[0][j][4 * v + 3] += x.w;
                }
        }
        if (len == q.kb) {
            float* sh = reinterpret_cast<float*>(s1) + wave * (32 * SP_SB);
#pragma unroll
            for (int i = 0; i < DONE; ++i)
#pragma unroll
                for (int j = 0; j < S::NJ; ++j)
                    sp_block<MODE>(total[i][j], sh, q, fin, fg, ti * E + wi + i0 + i, tj * E + wj + j);
        } else {
            // [block of 32 x 32][quarter of a lane's registers][lane]
            float4* out = reinterpret_cast<float4*>(q.part + ((int64_t)b * 2 + seg) * (TILE * TILE));
#pragma unroll
            for (int i = 0; i < DONE; ++i)
#pragma unroll
                for (int j = 0; j < S::NJ; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        out[(((wi + i0 + i) * E + wj + j) * 4 + v) * 64 + lane] =
                            make_float4(total[i][j][4 * v], total[i][j][4 * v + 1], total[i][j][4 * v + 2],
                                        total[i][j][4 * v + 3]);
        }
        __syncthreads();      // before the next tile's loads into LDS
        u += len;
    }
}

// A block takes a 64 x 64 tile with its whole reduction: the four waves each
// take every fourth piece for all of the tile, from stages of their own, so
// that no wave waits for another until the end, when the four sums are added in
// order and each wave writes a quarter of the tile.
constexpr int SP_SMALL = 64;
constexpr int SP_LINES = 2 * SP_SMALL * 8;      // 16-byte chunks of a wave's stage

__device__ __forceinline__ void sp_small_load(uint4* stage, const char* const (&src)[2], const uint32_t (&off)[2],
                                              int64_t ld)
{
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int i = 0; i < SP_SMALL / 8; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                sp_rsrc(src[o]), (__attribute__((address_space(3))) void*)(stage + o * (SP_SMALL * 8) + i * 64), 16,
                off[i & 1], i * 8 * (uint32_t)ld, 0, 0);
}

struct SpPiece {
    f16x8 ah[2][2], al[2][2], bh[2][2], bl[2][2];      // [half][32 rows or columns]
};
__device__ __forceinline__ void sp_small_read(SpPiece& f, const uint4* stage)
{
    const int lane = (int)threadIdx.x & 63, swz = (lane >> 1) & 7;
    const f16x8* A = reinterpret_cast<const f16x8*>(stage) + (lane % 32) * 8;
    const f16x8* B = A + SP_SMALL * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int ch = (h * 2 + lane / 32) ^ swz, cl = (4 + h * 2 + lane / 32) ^ swz;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f.ah[h][i] = A[i * 256 + ch];
            f.al[h][i] = A[i * 256 + cl];
            f.bh[h][i] = B[i * 256 + ch];
            f.bl[h][i] = B[i * 256 + cl];
        }
    }
}
// One half's products, and 16 loads (mask 0x010) or LDS reads (0x100) among them.
template <int OTHERS>
__device__ __forceinline__ void sp_small_multiply(const SpPiece& f, int h, f32x16 (&acc)[2][2])
{
#pragma unroll
    for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x == 2 ? f.al[h][i] : f.ah[h][i],
                                                                  x == 1 ? f.bl[h][j] : f.bh[h][j], acc[i][j], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(OTHERS, 2, 0);
    }
#pragma unroll
    for (int i = 4; i < 12; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(OTHERS, 1, 0);
    }
}

template <int MODE, typename T, typename F>
__global__ __launch_bounds__(256) void sp_small_kernel(SpProduct q, SpFinal<T, F> fin)
{
    __shared__ uint4 sa[4 * SP_LINES];
    __shared__ uint4 sb[4 * SP_LINES];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int ti, tj;
    sp_tile_at(q, (int)xcd_remap(blockIdx.x, gridDim.x), ti, tj);
    const float2 fg = sp_factors<MODE>(q);
    const int64_t ld = (int64_t)row_lines(q.kb) * 128;
    uint32_t off[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        off[i] = (uint32_t)(lane / 8 * ld) + ((uint32_t)(lane & 7) ^ (uint32_t)(i * 4 + lane / 16)) * 16;
    f32x16 acc[2][2] = {};
    if (wave < q.kb) {
        uint4* const A = sa + wave * SP_LINES;
        uint4* const B = sb + wave * SP_LINES;
        const int count = (q.kb - wave + 3) / 4;
        const char* src[2] = {(const char*)q.p + (int64_t)ti * SP_SMALL * ld + wave * 128,
                              (const char*)q.r + (int64_t)tj * SP_SMALL * ld + wave * 128};
        int left = count;
        // (past the last piece it is loaded again and not used: the waits count on a load every time)
        auto load = [&](uint4* stage) {
            sp_small_load(stage, src, off, ld);
            const int step = --left > 0 ? 512 : 0;
            src[0] += step;
            src[1] += step;
        };
        // the older of the two pieces under way has landed
        auto landed = [] {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0x4f70);      // vmcnt 16
            asm volatile("" ::: "memory");
        };
        // this wave's LDS reads are done
        auto have_read = [] {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xc07f);      // lgkmcnt 0
            asm volatile("" ::: "memory");
        };
        SpPiece f0, f1;
        load(A);
        load(B);
        landed();
        sp_small_read(f0, A);
        auto piece_of = [&](const SpPiece& now, SpPiece& then, uint4* cur, uint4* nxt) {
            have_read();
            load(cur);
            sp_small_multiply<0x010>(now, 0, acc);
            landed();
            sp_small_read(then, nxt);
            sp_small_multiply<0x100>(now, 1, acc);
        };
        for (int i = 0; i < count / 2; ++i) {
            piece_of(f0, f1, A, B);
            piece_of(f1, f0, B, A);
        }
        if (count & 1) piece_of(f0, f1, A, B);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);      // vmcnt 0, lgkmcnt 0: nothing lands from here on
    asm volatile("" ::: "memory");
    __syncthreads();
    // [wave][quarter of the tile][quarter of a lane's registers][lane]
    float4* sum = reinterpret_cast<float4*>(sa);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                sum[((wave * 4 + i * 2 + j) * 4 + v) * 64 + lane] = make_float4(
                    acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]);
    __syncthreads();
    f32x16 total = {};
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float4 x = sum[((w * 4 + wave) * 4 + v) * 64 + lane];
            total[4 * v] += x.x;
            total[4 * v + 1] += x.y;
            total[4 * v + 2] += x.z;
            total[4 * v + 3] += x.w;
        }
    sp_block<MODE>(total, reinterpret_cast<float*>(sb) + wave * (32 * SP_SB), q, fin, fg, ti * 2 + wave / 2, tj * 2 + wave % 2);
}

// Adds the partial sums of the tiles that several blocks share.  A wave takes
// one 32 x 32 block.
template <int MODE, typename T, typename F>
__global__ __launch_bounds__(256) void sp_join_kernel(SpProduct q, SpFinal<T, F> fin)
{
    __shared__ float shared[4][32 * SP_SB];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int edge = q.tile / 32, per = edge * edge / 4;      // blocks of this launch per tile
    const int t = (int)blockIdx.x / per, blk = (int)blockIdx.x % per * 4 + wave;
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
    // (the tile's first block may have begun in an earlier tile: its sums of this one are in its second place)
    f32x16 acc = {};
    auto at = [&](int b) {
        const int seg = b == ba && sp_first(q, b) < ua ? 1 : 0;
        return reinterpret_cast<const float4*>(q.part + ((int64_t)b * 2 + seg) * q.tile * q.tile) + blk * 256 + lane;
    };
    auto add = [&](const float4 (&w)[4]) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            acc[4 * v] += w[v].x;
            acc[4 * v + 1] += w[v].y;
            acc[4 * v + 2] += w[v].z;
            acc[4 * v + 3] += w[v].w;
        }
    };
    int b = ba;
    for (; b + 3 <= bb; b += 4) {      // four blocks' loads in flight
        float4 w[4][4];
#pragma unroll
        for (int l = 0; l < 4; ++l)
#pragma unroll
            for (int v = 0; v < 4; ++v) w[l][v] = at(b + l)[v * 64];
#pragma unroll
        for (int l = 0; l < 4; ++l) add(w[l]);
    }
    for (; b <= bb; ++b) {
        float4 w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) w[v] = at(b)[v * 64];
        add(w);
    }
    int ti, tj;
    sp_tile_at(q, t, ti, tj);
    sp_block<MODE>(acc, shared[wave], q, fin, sp_factors<MODE>(q), ti * edge + blk / edge, tj * edge + blk % edge);
}

// Tiles and blocks of a product: those of least estimated time, in
// microseconds from timings of 512..4096 square and of long products.
//   64: 4.5 + 0.24 a piece for each round of a block per CU;
//   128 and 256, a block for each tile: 12 + 0.65 (0.76 in several rounds),
//   10 + 2.6 a piece and round;
//   128 and 256, the units cut into equal ranges for one block per CU (but no
//   more than 16 for a tile, whose partial sums the joining launch adds one
//   after another): 19 + 0.95 a piece of a block and 24 a tile of one that has
//   several, 28 + 2.9 a piece, the join among them.
// Times of P X (64, 128, 256): m = n = 1024 14, 26, 38 us; 2048: 77, 54, 75;
// 4096: 499, 390, 330.  X X^T with tiles of 128, whole and cut: 2048: 58, 45;
// 2500: 58, 74.
void sp_plan(SpProduct& q)
{
    double best = 0.0;
    SpProduct pick = q;
    auto offer = [&](int grid, double us) {
        if (best != 0.0 && us >= best) return;
        best = us;
        pick = q;
        pick.grid = grid;
    };
    for (int tile : {64, 128, 256}) {
        q.tile = tile;
        q.mt = (q.m + tile - 1) / tile;
        q.nt = (q.n + tile - 1) / tile;
        const int64_t t = sp_tiles(q), units = t * q.kb;
        const double whole = (double)((t + SP_GRID - 1) / SP_GRID) * q.kb;      // pieces of the busiest CU
        if (tile == SP_SMALL) {
            offer((int)t, (double)((t + SP_GRID - 1) / SP_GRID) * 4.5 + 0.24 * whole);
            continue;
        }
        offer((int)t, tile == 128 ? 12 + (t > SP_GRID ? 0.76 : 0.65) * whole : 10 + 2.6 * whole);
        const int grid = (int)std::min<int64_t>(std::min<int64_t>(SP_GRID, 16 * t), (units + 1) / 2);
        const double cut = (double)((units + grid - 1) / grid);
        const double restarts = t > grid ? 24.0 * (double)t / grid : 0.0;
        offer(grid, tile == 128 ? 19 + 0.95 * cut + restarts : 28 + 2.9 * cut);
    }
    q = pick;
}

template <int MODE, typename T = float, typename F = SpNone>
hipError_t sp_run(SpProduct q, const SpFinal<T, F>& fin, hipStream_t s)
{
    sp_plan(q);
    const int64_t tiles = sp_tiles(q), units = tiles * q.kb;
    if (q.tile == SP_SMALL) {
        hipLaunchKernelGGL((sp_small_kernel<MODE, T, F>), dim3((unsigned)q.grid), dim3(256), 0, s, q, fin);
        return hipGetLastError();
    }
    if (q.tile == 256)
        hipLaunchKernelGGL((sp_product_kernel<256, MODE, T, F>), dim3((unsigned)q.grid), dim3(512), 0, s, q, fin);
    else
        hipLaunchKernelGGL((sp_product_kernel<128, MODE, T, F>), dim3((unsigned)q.grid), dim3(512), 0, s, q, fin);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (units % q.grid == 0 && units / q.grid % q.kb == 0)) return e;      // whole tiles everywhere
    const int edge = q.tile / 32;
    hipLaunchKernelGGL((sp_join_kernel<MODE, T, F>), dim3((unsigned)(tiles * edge * edge / 4)), dim3(256), 0, s, q, fin);
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
    auto add = [&](const T* v) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double d = (double)Elem<T>::load(v, j);
            a = fma(d, d, a);
        }
    };
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (; i + 3 * SP_NORM * 256 < vecs; i += 4 * SP_NORM * 256) {      // four loads in flight
        T v[4][V];
#pragma unroll
        for (int l = 0; l < 4; ++l) __builtin_memcpy(v[l], u + (i + l * SP_NORM * 256) * V, 16);
#pragma unroll
        for (int l = 0; l < 4; ++l) add(v[l]);
    }
    for (; i < vecs; i += SP_NORM * 256) {
        T v[V];
        __builtin_memcpy(v, u + i * V, 16);
        add(v);
    }
    if (blockIdx.x == 0 && (int64_t)threadIdx.x < n - vecs * V) {
        const double d = (double)Elem<T>::load(u, vecs * V + threadIdx.x);
        a = fma(d, d, a);
    }
    a = sp_block_sum(a, sh);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The lift of X_k, log2: |X_k| is at most r = |U| / (|U| + eps) times the
// product of the bounds of P_0 .. P_{k-1}, and room[k] is X_k's bound over that
// product.  A is lifted twice as much, P not.  (Factors of f and g that
// underflow belong to terms that far below a I; up to 2^90, so that the last
// product's f, 2^-30, stays a normal number.)
constexpr int SP_STEPS = 32;
struct SpRoom {
    int steps;
    float room[SP_STEPS];
};
__device__ __forceinline__ int sp_lift(float room, double r)
{
    const double l = (double)room / r;
    return l >= 2.0 ? min(ilogb(l), 90) : 0;      // (0 also where r is no number)
}

// X0 = U / (|U|_F + eps) in both layouts; a wave takes 32 x 32 elements.  Block
// 0 also writes the lifts: of each step's f and g of P, and of f of P X.
template <typename T>
__global__ __launch_bounds__(256) void sp_split_kernel(const T* u, int rows, int cols, const double* part, float eps,
                                                       float scale, SpProduct q, int tall, SpRoom room, float* lift)
{
    __shared__ double red[4];
    __shared__ float shared[4][32 * SP_SB];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    double a = 0.0;
    for (int i = (int)threadIdx.x; i < SP_NORM; i += 256) a += part[i];
    const double norm = sqrt(sp_block_sum(a, red)), r = norm / (norm + (double)eps);
    const double s = ldexp((double)scale, sp_lift(room.room[0], r)) / (norm + (double)eps);
    if (blockIdx.x == 0 && (int)threadIdx.x < room.steps) {
        const int k = (int)threadIdx.x, now = sp_lift(room.room[k], r);
        const int next = k + 1 < room.steps ? sp_lift(room.room[k + 1], r) : 0;
        lift[3 * k] = (float)ldexp(1.0, -4 * now);
        lift[3 * k + 1] = (float)ldexp(1.0, -2 * now);
        lift[3 * k + 2] = (float)ldexp(1.0, next - now);
    }
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
    sp_put<SP_BOTH>(sh, false, 1.f, 0.f, q, tall ? q.dt : q.d, bc, r0, c0, rows, cols);
    sp_put<SP_BOTH>(sh, true, 1.f, 0.f, q, tall ? q.d : q.dt, pieces(rows), c0, r0, cols, rows);
}

// -------------------------------------------------------------------- plan
// Bounds of the singular values of X_k and of the eigenvalues of P_k.
struct SpBounds {
    bool fits;
    double x[SP_STEPS + 1], p[SP_STEPS];
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
    size_t norm, lift, x, xt[2], a, p, part, bytes;
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
    l.lift = take(3 * SP_STEPS * sizeof(float));
    l.x = take(rows(m) * row_lines(pieces(n)) * 128);
    l.xt[0] = take(rows(n) * row_lines(pieces(m)) * 128);
    l.xt[1] = take(rows(n) * row_lines(pieces(m)) * 128);
    l.a = take(rows(m) * row_lines(pieces(m)) * 128);
    l.p = take(rows(m) * row_lines(pieces(m)) * 128);
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
    float* lift = (float*)(ws + l.lift);
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
    q.d = X;
    q.dt = XT[0];
    SpRoom room{};
    room.steps = c.steps;
    double grown = 1.0;      // the bounds of the P before
    for (int k = 0; k < c.steps; ++k) {
        room.room[k] = (float)(bd.x[k] / grown);
        grown *= bd.p[k];
    }
    const int64_t blocks = ((int64_t)pieces(rows) * pieces(cols) + 3) / 4;
    hipLaunchKernelGGL(sp_split_kernel<T>, dim3((unsigned)blocks), dim3(256), 0, s, u, rows, cols, norm, c.eps,
                       (float)sx, q, (int)tall, room, lift);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    const SpFinal<float, SpNone> none{};
    for (int k = 0; k < c.steps; ++k) {
        const double sa = sp_scale(1.01 * bd.x[k] * bd.x[k]), sp = sp_scale(1.01 * bd.p[k]);
        q.p = q.r = X;
        q.kb = pieces(n);
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
        q.lift = lift + 3 * k;
        q.d = P;
        if ((e = sp_run<SP_POLY>(q, none, s)) != hipSuccess) return e;
        q.p = P;
        q.r = XT[k & 1];
        q.lift = lift + 3 * k + 2;
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

// Where these products beat the fp64 path, whose 14 rounds of m x m products
// cost as m^2 to m^3 while n costs it little (here, there, in microseconds):
// 320 x 320 125, 129 and x 640 134, 130; 360 x 1440 168, 170 and x 2880 224,
// 181; 512 x 4096 261, 273 and x 12288 421, 354; 768 x 18432 810, 846 and
// x 24576 1180, 968; 1024 x 16384 1071, 1425; 2048 x 65536 11714, 15895.
bool ns_split_size(int m, int n) { return 16 * (int64_t)n <= (int64_t)m * (m - 300); }
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
