// The join of a residual block: the norm after its branch, the branch's gate,
// the residual scale, and the norm before the next branch, all over the C
// channels of a voxel (a row):
//   H = post(F),  R = alpha X + gate H,  Y = pre(R)
//   RMS    norm(v) = v rstd gamma + beta, rstd = 1 / sqrt(sum v^2 / C + eps)
//   layer  norm(v) = (v - mean) rstd gamma + beta, rstd from the variance
// Backward, with fh and rh the normalised rows of F and R:
//   v = dY gpre,  d = dR + rstd_r (v - rh mean(v rh) [- mean(v)])
//   dX = alpha d,  u = gate gpost d,  dF = rstd_f (u - fh mean(u fh) [- mean(u)])
//   dgpre = sum dY rh, dbpre = sum dY, dgpost = sum gate d fh, dbpost = sum gate d,
//   dgate = sum d H
// (brackets: layer norm).  Every tensor is read once and written once; the rows'
// statistics are formed again in the backward, where the rows are in registers
// anyway, and not kept.
//
// A row is held by LPR lanes with E values each, 16 bytes at a time; a lane
// keeps its channels over all its rows, so that the vectors' products and the
// column sums stay in registers.  Rows that are not a multiple of 16 bytes long
// are read with unaligned 16-byte accesses, their last values one by one.
// A block takes a range of one sample's rows; the column sums of the blocks are
// added by a second launch, in a fixed order and in fp64: results are
// reproducible bit for bit.
//
// What bounds it: memory.  Forward, 8 x 64^3 x 64 bf16: 1.07 GB in 221 us (4.9 TB/s).
// Backward, 8 x 32^3 x 256 bf16: 805 MB in 175 us (4.6 TB/s) and 6 us for the join.
// There a lane has some 350 instructions a row, so that arithmetic alone is half of
// the time: the next row's loads are under way during it (239 us without), and sums
// between lanes are one instruction a step (shuffles go through LDS).
// 3 x 37 x 29 x 31 x 60 fp32: 33 us (4.3 TB/s) and 4.
#include "cf_internal.h"

namespace cf {
namespace {

constexpr int RN_T = 256;             // threads a block
constexpr int RN_FWD_BLOCKS = 2048;   // blocks of a forward launch, 8 a CU

// How the rows are dealt out: `samples` of `rows` rows, each cut into `parts`.
struct RnSplit {
    int64_t rows;
    int samples, parts, blocks;
};

struct RnArgs {
    int C;
    float inv_c, alpha, eps;
    const float *gpre, *bpre, *gpost, *bpost, *gate;
    int64_t gate_step;               // from one sample's gate to the next (0: one for all)
};

// v plus another lane's: 1, 2: lanes that differ in that bit; 4, 8: after the sums
// over the bits below, any lane of the other half will do, and mirrored rows of 8
// and 16 have one; 16, 32: rows and halves of the wave swapped.  One instruction
// each, where a shuffle goes through LDS.
template <int BIT> __device__ __forceinline__ float lane_sum(float v)
{
    if constexpr (BIT <= 8) {
        constexpr int ctrl = BIT == 1 ? 0xb1 : BIT == 2 ? 0x4e : BIT == 4 ? 0x141 : 0x140;
        return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xf, 0xf, true));
    } else {
        const unsigned u = __builtin_bit_cast(unsigned, v);
        const auto w = BIT == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                                 : __builtin_amdgcn_permlane32_swap(u, u, false, false);
        return __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
}

// Sum of v[0..N) over a row's lanes, in each of them.
template <int LPR, int N> __device__ __forceinline__ void row_sum(float (&v)[N], float* sh, int& turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (LPR > 1) v[i] = lane_sum<1>(v[i]);
        if (LPR > 2) v[i] = lane_sum<2>(v[i]);
        if (LPR > 4) v[i] = lane_sum<4>(v[i]);
        if (LPR > 8) v[i] = lane_sum<8>(v[i]);
        if (LPR > 16) v[i] = lane_sum<16>(v[i]);
        if (LPR > 32) v[i] = lane_sum<32>(v[i]);
    }
    if (LPR > 64) {
        // two buffers in turn: a wave writes one again only after a barrier that the readers of it have reached
        float* at = sh + turn * 16;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) at[i * 4 + (threadIdx.x >> 6)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (at[i * 4] + at[i * 4 + 1]) + (at[i * 4 + 2] + at[i * 4 + 3]);
    }
}

// A lane's E values of a row: E / V vectors of V, LPR vectors apart.  WHOLE: rows are
// whole vectors.
template <typename T, int LPR, int E, bool WHOLE> struct RnLane {
    static constexpr int V = 16 / (int)sizeof(T);
    static constexpr int VECS = E / V;
    static_assert(E % V == 0, "whole vectors");
    int lane, C;
    __device__ __forceinline__ int channel(int i) const { return ((i / V) * LPR + lane) * V + i % V; }
    // Whether value i lies in the row.
    __device__ __forceinline__ bool inside(int i) const { return channel(WHOLE ? i / V * V : i) < C; }
    struct Raw {
        uint4 v[VECS];
    };
    // Whole vectors without a branch, the last one of a row from V values before its
    // end on (lanes past the end read it too); unpack() moves the values to their
    // places.  Rows of less than V values, which lanes in pairs hold, one by one.
    // `row`: the values' distance from `from`, which all threads share.
    __device__ __forceinline__ void fetch(const T* from, uint32_t row, Raw& raw) const
    {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int c = channel(j * V);
            if (!WHOLE && LPR == 2 && C < V) {
                T t[V];
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = c + i < C ? from[row + (uint32_t)(c + i)] : (T)0;
                __builtin_memcpy(&raw.v[j], t, 16);
            } else {
                __builtin_memcpy(&raw.v[j], from + (row + (uint32_t)min(c, C - V)), 16);
            }
        }
    }
    __device__ __forceinline__ void unpack(const Raw& raw, float (&v)[E]) const
    {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int c = channel(j * V);
            uint32_t w[4] = {raw.v[j].x, raw.v[j].y, raw.v[j].z, raw.v[j].w};
            if (WHOLE || C >= V) {
                const int over = c - min(c, C - V);           // values before this vector's first
                if (!WHOLE) {
                    const int bytes = over * (int)sizeof(T);
                    if (bytes & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = 0;
                    if (bytes & 8) w[0] = w[2], w[1] = w[3], w[2] = w[3] = 0;
                    if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = w[i] >> 16 | (i < 3 ? w[i < 3 ? i + 1 : 3] << 16 : 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = over >= V ? 0 : w[i];
            }
            T t[V];
            __builtin_memcpy(t, w, 16);
#pragma unroll
            for (int i = 0; i < V; ++i) v[j * V + i] = widen(t[i]);
        }
    }
    __device__ __forceinline__ void store(T* from, uint32_t row, const float (&v)[E]) const
    {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int c = channel(j * V), n = C - c;
            T t[V];
#pragma unroll
            for (int i = 0; i < V; ++i) Elem<T>::store(t, i, v[j * V + i]);
            uint32_t w[4];
            __builtin_memcpy(w, t, 16);
            if (n >= V) __builtin_memcpy(from + (row + (uint32_t)c), w, 16);
            else if (!WHOLE && n > 0) {
                const int bytes = n * (int)sizeof(T);
                char* p = (char*)(from + (row + (uint32_t)c));
                if (bytes & 8) {
                    __builtin_memcpy(p, w, 8);
                    p += 8, w[0] = w[2], w[1] = w[3];
                }
                if (bytes & 4) {
                    __builtin_memcpy(p, w, 4);
                    p += 4, w[0] = w[1];
                }
                if (sizeof(T) == 2 && (bytes & 2)) __builtin_memcpy(p, w, 2);
            }
        }
    }
    // A vector of C floats (null: `other`), 0 past its end.
    __device__ __forceinline__ void vec(const float* p, float other, float (&v)[E]) const
    {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int c = channel(j * V);
            float t[V];
            if (!p) {
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = other;
            } else if (WHOLE) {
                __builtin_memcpy(t, p + (uint32_t)min(c, C - V), sizeof(t));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = p[(uint32_t)min(c + i, C - 1)];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) v[j * V + i] = inside(j * V + i) ? t[i] : 0.f;
        }
    }
};

// Normalises rows in place: v becomes (v - mean) rstd, and 0 past the row's end.
// The layer norm's mean is found in two steps, the second from the centred
// values: their sum and the sum of their squares come out of one reduction, and
// the mean's own rounding does not stay in v.
template <bool LAYER, int LPR, typename L, int E>
__device__ __forceinline__ float normalise(float (&v)[E], const L& ln, float inv_c, float eps, float* sh, int& turn)
{
    float s[2];
    if (LAYER) {
        float a[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) a[0] += v[i];
        row_sum<LPR>(a, sh, turn);
        const float m = a[0] * inv_c;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = ln.inside(i) ? v[i] - m : 0.f;
            s[0] += v[i];
            s[1] = fmaf(v[i], v[i], s[1]);
        }
        row_sum<LPR>(s, sh, turn);
        const float m2 = s[0] * inv_c;
        const float rstd = rsqrtf(fmaxf(fmaf(s[1], inv_c, -m2 * m2), 0.f) + eps);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = ln.inside(i) ? (v[i] - m2) * rstd : 0.f;
        return rstd;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) q[0] = fmaf(v[i], v[i], q[0]);
    row_sum<LPR>(q, sh, turn);
    const float rstd = rsqrtf(fmaf(q[0], inv_c, eps));
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= rstd;
    return rstd;
}

// The gradient that reaches the rows whose normalised values are `hat`, from that
// of the normalised values, d.
template <bool LAYER, int LPR, int E>
__device__ __forceinline__ void through_norm(float (&d)[E], const float (&hat)[E], float rstd, float inv_c, float* sh,
                                             int& turn)
{
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        s[0] = fmaf(d[i], hat[i], s[0]);
        s[1] += d[i];
    }
    if (LAYER) row_sum<LPR>(s, sh, turn);
    else {
        float q[1] = {s[0]};
        row_sum<LPR>(q, sh, turn);
        s[0] = q[0];
    }
    const float a = s[0] * inv_c, b = LAYER ? s[1] * inv_c : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = rstd * (fmaf(-hat[i], a, d[i]) - b);
}

template <typename T, bool LAYER, int LPR, int E, bool WHOLE>
__global__ __launch_bounds__(RN_T) void resnorm_fwd_kernel(RnArgs a, RnSplit q, const T* __restrict__ X,
                                                           const T* __restrict__ F, T* __restrict__ R,
                                                           T* __restrict__ Y)
{
    __shared__ float sh[32];
    int turn = 0;
    const RnLane<T, LPR, E, WHOLE> ln{(int)threadIdx.x % LPR, a.C};
    constexpr int ROWS = RN_T / LPR;
    const int mine = (int)threadIdx.x / LPR;      // this lane's row of the ROWS that a block works on
    using Raw = typename RnLane<T, LPR, E, WHOLE>::Raw;
    float gp[E], bp[E], ga[E], gb[E];
    ln.vec(a.gpre, 1.f, gp);
    ln.vec(a.bpre, 0.f, bp);
    int last = -1;
    const int64_t items = (int64_t)q.samples * q.parts;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int n = (int)(it / q.parts), p = (int)(it % q.parts);
        if (n != last) {
            float g[E];
            ln.vec(a.gate ? a.gate + n * a.gate_step : nullptr, 1.f, g);
            ln.vec(a.gpost, 1.f, ga);
            ln.vec(a.bpost, 0.f, gb);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                ga[i] *= g[i];
                if (a.bpost) gb[i] *= g[i];      // (no offset: 0, also where the gate is infinite)
            }
            last = n;
        }
        const int64_t r0 = q.rows * p / q.parts, r1 = q.rows * (p + 1) / q.parts;
        for (int64_t r = r0; r < r1; r += ROWS) {
            if (r + mine >= r1) break;
            const int64_t at = (n * q.rows + r) * a.C;
            const uint32_t row = (uint32_t)(mine * a.C);
            float f[E], v[E];
            Raw rf, rx;
            ln.fetch(F + at, row, rf);
            ln.fetch(X + at, row, rx);
            ln.unpack(rf, f);
            ln.unpack(rx, v);
            if (a.gpost) normalise<LAYER, LPR>(f, ln, a.inv_c, a.eps, sh, turn);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = fmaf(a.alpha, v[i], fmaf(f[i], ga[i], gb[i]));
            ln.store(R + at, row, v);
            if (Y) {
                // (of the unrounded values: one rounding in Y, not two)
                normalise<LAYER, LPR>(v, ln, a.inv_c, a.eps, sh, turn);
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = fmaf(v[i], gp[i], bp[i]);
                ln.store(Y + at, row, v);
            }
        }
    }
}

// Sums of a block's column sums, into out[C].
template <int LPR, int E, typename L>
__device__ __forceinline__ void column_sums(float (&v)[E], const L& ln, float* sh, float* out)
{
    if (LPR > 64) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (ln.channel(i) < ln.C) out[ln.channel(i)] = v[i];
        return;
    }
#pragma unroll
    for (int m = LPR; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += __shfl_xor(v[i], m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) < LPR)
#pragma unroll
        for (int i = 0; i < E; ++i) sh[(threadIdx.x >> 6) * (LPR * E) + ln.channel(i)] = v[i];
    __syncthreads();
    for (int c = (int)threadIdx.x; c < ln.C; c += RN_T)
        out[c] = (sh[c] + sh[LPR * E + c]) + (sh[2 * LPR * E + c] + sh[3 * LPR * E + c]);
}

// Waves a SIMD that the backward's registers leave room for.
template <typename T, int E, bool WHOLE> constexpr int rn_waves()
{
    return E == 8 ? (sizeof(T) == 2 && WHOLE ? 4 : 2) : (sizeof(T) == 2 && WHOLE ? 2 : 1);
}

// vecs: [4][blocks][C], the blocks' sums for dgpre, dbpre, dgpost, dbpost;
// gates: [samples * parts][C], dgate itself where a sample is one part.
template <typename T, bool LAYER, int LPR, int E, bool WHOLE>
__global__ __launch_bounds__(RN_T, (rn_waves<T, E, WHOLE>())) void resnorm_bwd_kernel(
    RnArgs a, RnSplit q, const T* __restrict__ F, const T* __restrict__ R, const T* __restrict__ dR,
    const T* __restrict__ dY, T* __restrict__ dX, T* __restrict__ dF, float* __restrict__ vecs, float* __restrict__ gates)
{
    __shared__ float sh[LPR > 64 ? 32 : 4 * LPR * E];
    // a thread's sums of gate d fh and gate d over all of its rows (items may have gates of their own)
    __shared__ float sg[2 * E * RN_T];
    int turn = 0;
    const RnLane<T, LPR, E, WHOLE> ln{(int)threadIdx.x % LPR, a.C};
    constexpr int ROWS = RN_T / LPR;
    const int mine = (int)threadIdx.x / LPR;      // this lane's row of the ROWS that a block works on
    using Raw = typename RnLane<T, LPR, E, WHOLE>::Raw;
    float gp[E];
    ln.vec(a.gpre, 1.f, gp);
    float t1[E] = {}, t0[E] = {};                       // sums of dY rh, dY over the block's rows
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) sg[i * RN_T + (int)threadIdx.x] = 0.f;
    const int64_t items = (int64_t)q.samples * q.parts;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int n = (int)(it / q.parts), p = (int)(it % q.parts);
        const float* gate_of = a.gate ? a.gate + n * a.gate_step : nullptr;
        float ga[E], s1[E] = {}, s0[E] = {};            // sums of d fh (of d F without a post norm) and d over the item's rows
        {
            float g[E];
            ln.vec(gate_of, 1.f, g);
            ln.vec(a.gpost, 1.f, ga);
#pragma unroll
            for (int i = 0; i < E; ++i) ga[i] *= g[i];
        }
        const int64_t r0 = q.rows * p / q.parts, r1 = q.rows * (p + 1) / q.parts;
        // the next row's values are under way while this one's are worked on
        Raw rf, rr, rd, ry;
        auto fetch = [&](int64_t r) {
            const int64_t at = (n * q.rows + r) * a.C;
            const uint32_t row = (uint32_t)(min((int64_t)mine, r1 - 1 - r) * a.C);
            ln.fetch(F + at, row, rf);
            if (dY) ln.fetch(R + at, row, rr), ln.fetch(dY + at, row, ry);
            if (dR) ln.fetch(dR + at, row, rd);
        };
        fetch(r0);
        for (int64_t r = r0; r < r1; r += ROWS) {
            const int64_t at = (n * q.rows + r) * a.C;
            const uint32_t row = (uint32_t)(mine * a.C);
            const Raw cf = rf, cr = rr, cd = rd, cy = ry;
            if (r + ROWS < r1) fetch(r + ROWS);
            if (r + mine >= r1) break;
            float d[E], f[E];
            if (dY) {
                float v[E], y[E];
                ln.unpack(cr, v);
                const float rstd = normalise<LAYER, LPR>(v, ln, a.inv_c, a.eps, sh, turn);
                ln.unpack(cy, y);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    t1[i] = fmaf(y[i], v[i], t1[i]);
                    t0[i] += y[i];
                    d[i] = y[i] * gp[i];
                }
                through_norm<LAYER, LPR>(d, v, rstd, a.inv_c, sh, turn);
                if (dR) {
                    ln.unpack(cd, y);
#pragma unroll
                    for (int i = 0; i < E; ++i) d[i] += y[i];
                }
            } else {
                ln.unpack(cd, d);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = a.alpha * d[i];
            ln.store(dX + at, row, f);
            ln.unpack(cf, f);
            float rstd = 1.f;
            if (a.gpost) rstd = normalise<LAYER, LPR>(f, ln, a.inv_c, a.eps, sh, turn);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (LAYER) d[i] = ln.inside(i) ? d[i] : 0.f;      // (what the norm took from all: its mean)
                s1[i] = fmaf(d[i], f[i], s1[i]);
                s0[i] += d[i];
                d[i] *= ga[i];
            }
            if (a.gpost) through_norm<LAYER, LPR>(d, f, rstd, a.inv_c, sh, turn);
            ln.store(dF + at, row, d);
        }
        float g[E];
        ln.vec(gate_of, 1.f, g);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float* at = sg + 2 * i * RN_T + (int)threadIdx.x;
            at[0] = fmaf(g[i], s1[i], at[0]);
            at[RN_T] = fmaf(g[i], s0[i], at[RN_T]);
        }
        if (a.gate) {
            float bo[E];
            ln.vec(a.gpost, 1.f, g);
            ln.vec(a.bpost, 0.f, bo);
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = a.bpost ? fmaf(g[i], s1[i], bo[i] * s0[i]) : g[i] * s1[i];
            column_sums<LPR, E>(g, ln, sh, gates + it * a.C);
        }
    }
    const int64_t block = (int64_t)gridDim.x * a.C;
    float* out = vecs + (int64_t)blockIdx.x * a.C;
    if (dY) {
        column_sums<LPR, E>(t1, ln, sh, out);
        column_sums<LPR, E>(t0, ln, sh, out + block);
    }
    if (a.gpost) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            t1[i] = sg[2 * i * RN_T + (int)threadIdx.x];
            t0[i] = sg[(2 * i + 1) * RN_T + (int)threadIdx.x];
        }
        column_sums<LPR, E>(t1, ln, sh, out + 2 * block);
        column_sums<LPR, E>(t0, ln, sh, out + 3 * block);
    }
}

// Adds partial sums: job j < 4 takes the blocks' sums of one kind, job 4 + n
// sample n's parts of dgate.  16 columns a block, 64 threads to a column: the few
// blocks that a narrow tensor has are bound by the latency of a thread's loads.
struct RnJoin {
    const float* vecs;
    const float* gates;
    float* out[4];
    float* dgate;
    int C, blocks, parts;
};
__global__ __launch_bounds__(1024) void resnorm_join_kernel(RnJoin q)
{
    __shared__ double sh[16][16];
    const int job = (int)blockIdx.y, c = (int)blockIdx.x * 16 + (int)threadIdx.x % 16, k = (int)threadIdx.x / 16;
    if (job < 4 && !q.out[job]) return;
    const int len = job < 4 ? q.blocks : q.parts;
    const float* src = job < 4 ? q.vecs + (int64_t)job * q.blocks * q.C : q.gates + (int64_t)(job - 4) * q.parts * q.C;
    double sum = 0.0;
    if (c < q.C)
#pragma unroll 8
        for (int i = k; i < len; i += 64) sum += (double)src[(int64_t)i * q.C + c];
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if ((threadIdx.x & 63) < 16) sh[threadIdx.x >> 6][threadIdx.x & 15] = sum;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += sh[(threadIdx.x >> 4) * 4 + i][threadIdx.x & 15];
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (threadIdx.x < 16 && c < q.C) (job < 4 ? q.out[job] : q.dgate + (int64_t)(job - 4) * q.C)[c] = (float)sum;
}

// Samples are told apart only where they have gates of their own.
RnSplit rn_split(const cf_dims& x, int gate_n, int blocks)
{
    RnSplit q;
    const int64_t vox = x.d * x.h * x.w;
    q.samples = gate_n > 1 ? gate_n : 1;
    q.rows = gate_n > 1 ? vox : x.n * vox;
    const int64_t want = blocks / q.samples > 1 ? blocks / q.samples : 1;
    const int64_t few = (q.rows + 3) / 4;          // at least four rows a part
    q.parts = (int)(want < few ? want : few);
    const int64_t items = (int64_t)q.samples * q.parts;
    q.blocks = (int)(items < blocks ? items : blocks);
    return q;
}

// Blocks of a backward launch: as many as the chip holds at once, since each
// leaves C sums of five kinds.
int rn_bwd_blocks(cf_dtype dt, const cf_dims& x)
{
    const bool wide = dt == CF_F32 || x.c % 8, long_lane = (x.c > 512 && x.c <= 1024) || x.c > 2048;
    return 256 * (long_lane ? (wide ? 1 : 2) : (wide ? 2 : 4));
}

size_t up256r(size_t b) { return (b + 255) & ~(size_t)255; }

template <typename T, bool LAYER, int LPR, int E, bool WHOLE> struct RnKernels {
    static void fwd(const RnArgs& a, const RnSplit& q, const void* X, const void* F, void* R, void* Y, hipStream_t s)
    {
        resnorm_fwd_kernel<T, LAYER, LPR, E, WHOLE><<<q.blocks, RN_T, 0, s>>>(a, q, (const T*)X, (const T*)F, (T*)R, (T*)Y);
    }
    static void bwd(const RnArgs& a, const RnSplit& q, const void* F, const void* R, const void* dR, const void* dY,
                    void* dX, void* dF, float* vecs, float* gates, hipStream_t s)
    {
        resnorm_bwd_kernel<T, LAYER, LPR, E, WHOLE><<<q.blocks, RN_T, 0, s>>>(a, q, (const T*)F, (const T*)R, (const T*)dR,
                                                                       (const T*)dY, (T*)dX, (T*)dF, vecs, gates);
    }
};

// Calls f with the kernels of a row of C channels: eight values a lane while a
// wave or less holds the row, sixteen where that saves the exchange between waves.
template <typename T, bool LAYER, bool WHOLE, typename Fn> void rn_pick(int C, Fn f)
{
    if (C <= 16) f(RnKernels<T, LAYER, 2, 8, WHOLE>());
    else if (C <= 32) f(RnKernels<T, LAYER, 4, 8, WHOLE>());
    else if (C <= 64) f(RnKernels<T, LAYER, 8, 8, WHOLE>());
    else if (C <= 128) f(RnKernels<T, LAYER, 16, 8, WHOLE>());
    else if (C <= 256) f(RnKernels<T, LAYER, 32, 8, WHOLE>());
    else if (C <= 512) f(RnKernels<T, LAYER, 64, 8, WHOLE>());
    else if (C <= 1024) f(RnKernels<T, LAYER, 64, 16, WHOLE>());
    else if (C <= 2048) f(RnKernels<T, LAYER, 256, 8, WHOLE>());
    else f(RnKernels<T, LAYER, 256, 16, WHOLE>());
}
template <typename T, typename Fn> void rn_pick(bool layer, int C, Fn f)
{
    const bool whole = C % (16 / (int)sizeof(T)) == 0;
    if (layer) whole ? rn_pick<T, true, true>(C, f) : rn_pick<T, true, false>(C, f);
    else whole ? rn_pick<T, false, true>(C, f) : rn_pick<T, false, false>(C, f);
}

RnArgs rn_args(const cf_dims& x, const ResnormArgs& p)
{
    RnArgs a;
    a.C = (int)x.c;
    a.inv_c = 1.f / (float)x.c;
    a.alpha = p.alpha;
    a.eps = p.eps;
    a.gpre = p.gpre;
    a.bpre = p.bpre;
    a.gpost = p.gpost;
    a.bpost = p.bpost;
    a.gate = p.gate;
    a.gate_step = p.gate_n > 1 ? x.c : 0;
    return a;
}

}  // namespace

size_t resnorm_ws_bytes(cf_dtype dt, const cf_dims& x, int gate_n)
{
    const RnSplit q = rn_split(x, gate_n, rn_bwd_blocks(dt, x));
    const size_t gates = gate_n ? (size_t)q.samples * q.parts * x.c * sizeof(float) : 0;
    return up256r((size_t)4 * q.blocks * x.c * sizeof(float)) + up256r(gates);
}

template <typename T>
hipError_t launch_resnorm_fwd(const cf_dims& x, const ResnormArgs& p, const void* X, const void* F, void* R, void* Y,
                              hipStream_t s)
{
    const RnSplit q = rn_split(x, p.gate_n, RN_FWD_BLOCKS);
    const RnArgs a = rn_args(x, p);
    auto go = [&](auto k) { k.fwd(a, q, X, F, R, Y, s); };
    rn_pick<T>(p.layer, a.C, go);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_resnorm_bwd(const cf_dims& x, const ResnormArgs& p, const void* F, const void* R, const void* dR,
                              const void* dY, void* dX, void* dF, const ResnormGrads& g, void* ws, hipStream_t s)
{
    const RnSplit q = rn_split(x, p.gate_n, rn_bwd_blocks(sizeof(T) == 4 ? CF_F32 : CF_BF16, x));
    const RnArgs a = rn_args(x, p);
    float* vecs = (float*)ws;
    float* parts = (float*)((char*)ws + up256r((size_t)4 * q.blocks * x.c * sizeof(float)));
    float* gates = q.parts == 1 ? g.gate : parts;
    auto go = [&](auto k) { k.bwd(a, q, F, R, dR, dY, dX, dF, vecs, gates, s); };
    rn_pick<T>(p.layer, a.C, go);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const RnJoin j = {vecs, parts, {dY ? g.gpre : nullptr, dY ? g.bpre : nullptr, g.gpost, g.bpost}, g.gate, a.C,
                      q.blocks, q.parts};
    const int jobs = 4 + (p.gate && q.parts > 1 ? q.samples : 0);
    resnorm_join_kernel<<<dim3((unsigned)((a.C + 15) / 16), (unsigned)jobs), 1024, 0, s>>>(j);
    return hipGetLastError();
}

template hipError_t launch_resnorm_fwd<float>(const cf_dims&, const ResnormArgs&, const void*, const void*, void*, void*,
                                              hipStream_t);
template hipError_t launch_resnorm_fwd<uint16_t>(const cf_dims&, const ResnormArgs&, const void*, const void*, void*,
                                                 void*, hipStream_t);
template hipError_t launch_resnorm_bwd<float>(const cf_dims&, const ResnormArgs&, const void*, const void*, const void*,
                                              const void*, void*, void*, const ResnormGrads&, void*, hipStream_t);
template hipError_t launch_resnorm_bwd<uint16_t>(const cf_dims&, const ResnormArgs&, const void*, const void*,
                                                 const void*, const void*, void*, void*, const ResnormGrads&, void*,
                                                 hipStream_t);

}  // namespace cf
