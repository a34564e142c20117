// Group normalisation with an activation on NDHWC activations, forward and
// backward.
//
// Per sample n and group g of cg = C / G neighbouring channels, over the M =
// D H W cg values of the group:
//   mean = sum x / M, var = sum (x - mean)^2 / M, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd, z = xhat gamma_c + beta_c, y = act(z)
// and, with dz = dy act'(z),
//   dgamma_c = sum_n,voxels dz xhat, dbeta_c = sum_n,voxels dz
//   dx = rstd (gamma_c dz - s1 - xhat s2), s1 = sum_group gamma dz / M,
//   s2 = sum_group gamma dz xhat / M.
//
// A sample is one flat array of D H W C values read 16 bytes at a time.  A
// "row" is lcm(V, C) values (V values per 16 bytes), so a thread that steps
// by whole rows meets the same V channels every time, whatever C is: its
// coefficients and its V partial sums stay in registers.  Blocks hold a whole
// number of rows (k rows of `cols` vectors) rounded up to whole waves, so few
// threads idle for any C.
// Vectors are loaded and stored without an alignment demand beyond the
// element's (odd C puts samples at odd offsets); the last S % row values of a
// sample go element by element.
//
// Sums: the forward adds x and x^2 in fp64 (products of fp32 values are exact
// there up to one rounding): the variance keeps about 52 - 2 log2(mean /
// spread) bits, and x - mean is taken with the fp64 mean, whose part below
// fp32 is folded into the offset.  The backward starts from the fp32 mean and
// adds fp32 products in fp64.  Blocks write partial sums that
// are added in a fixed order: no atomics, results are reproducible bit for
// bit.
//
// Groups small enough for one block's registers take a single launch that
// reads every input once (gn_*_small; the backward of samples that share no
// block adds one that joins dgamma and dbeta); larger ones take a reducing launch and
// an applying launch (with a short joining launch between them in the
// backward).
//
// What bounds it: large samples, memory: 8 x 128^3 x 32 bf16 forward takes 603
// us for 3.2 GB (x is read twice; 5.3 TB/s, a copy reaches 5.1), 8 x 64^3 x 64
// backward 287 us for 1.34 GB.  A few MB, the latencies of two or three
// dependent launches: 3 x 37 x 29 x 31 x 60 fp32 forward 20.4 us; 2 x 45 x 33 x
// 27 x 96 bf16 backward 32 us, whose two passes keep the VALU busy 43 to 47% of
// the cycles while waves wait for 57% of theirs (two waves a SIMD).
#include "cf_internal.h"

#include <algorithm>
#include <numeric>

namespace cf {
namespace {

constexpr int GN_T = 512;        // most threads of a streaming block
constexpr int GN_TS = 1024;      // most threads of a small-group block
constexpr int GN_ROWS_F = 8;     // vectors per thread held by the small forward
constexpr int GN_ROWS_B = 4;     // and by the small backward (of x and dy each)
constexpr size_t GN_LDS = 65536; // most LDS of a small-group block
constexpr int GN_FEW = 192;      // streaming blocks that leave CUs idle
constexpr int GN_SLICES = 256;   // blocks from which slices of more groups are taken
constexpr int GN_BLOCKS = 1024;  // streaming blocks per launch, about 4 per CU

// V values of T as one 16-byte access (V = 1: one element).
template <typename T, int V> struct Vec {
    T v[V];
};
template <typename T, int V> __device__ __forceinline__ Vec<T, V> vload(const T* p)
{
    Vec<T, V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
template <typename T, int V> __device__ __forceinline__ void vstore(T* p, const Vec<T, V>& r)
{
    __builtin_memcpy(p, &r, sizeof(r));
}
__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(uint16_t x) { return bf2f(x); }
__device__ __forceinline__ void narrow(float& d, float x) { d = x; }
__device__ __forceinline__ void narrow(uint16_t& d, float x) { d = f2bf(x); }

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// How a sample (or a slice of its channels) is cut into rows and blocks.
struct GnGeom {
    int64_t S;       // values per sample
    int64_t nrows;   // whole rows per sample
    int C, G, cg;
    int row;         // values per row
    int cols;        // vectors per row
    int cc;          // vectors of a row that one block takes
    int chunks;      // ceil(cols / cc)
    int k;           // rows a block has in flight; k * cc <= threads
    int nb;          // blocks per sample and chunk
};

// A block's sums.  Thread t < n = k * cc holds in v[j] a partial sum of row
// position t % cc * V + j; 2^lh neighbouring positions that go to the same sum
// are added first, leaving positions p of V >> lh planes a thread.  In LDS a
// plane's values lie thread by thread, so that neighbouring lanes use
// neighbouring banks.
struct RowSums {
    const double* sh;
    int lg, n, cc, parts;      // log2 of the planes, values of a plane, vectors, partial sums left of a position
    __device__ __forceinline__ double at(int p, int i) const
    {
        return sh[(p & ((1 << lg) - 1)) * n + i * cc + (p >> lg)];
    }
    // Position p's total.
    __device__ __forceinline__ double total(int p) const
    {
        double a = 0.0;
        for (int i = 0; i < parts; ++i) a += at(p, i);
        return a;
    }
};

template <int V> __device__ __forceinline__ void put_rows(const double (&v)[V], double* sh, int n, int lh,
                                                             int t = (int)threadIdx.x)
{
    if (t >= n) return;
    double w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = v[j];
#pragma unroll
    for (int l = 0; (1 << l) < V; ++l)
        if (lh > l)
#pragma unroll
            for (int j = 0; j + (1 << l) < V; j += 2 << l) w[j] += w[j + (1 << l)];
#pragma unroll
    for (int j = 0; j < V; ++j)
        if ((j & ((1 << lh) - 1)) == 0) sh[(j >> lh) * n + t] = w[j];
}

// Adds the k rows of each plane in levels, each with as many threads as it can
// use, until at most 8 partial sums of a position are left; returns how many.
__device__ __forceinline__ int fold_rows(double* sh, int planes, int k, int cc)
{
    const int t = (int)threadIdx.x, T = (int)blockDim.x, n = k * cc;
    int parts = k;
    do {
        const int next = max(1, min((parts + 3) / 4, T / (planes * cc))), m = next * cc;
        __syncthreads();
        for (int e = t; e < planes * m; e += T) {
            const int j = e / m, x = e - j * m;
            double* q = sh + j * n + x;
            double a = q[0];
            for (int i = m; x + i < parts * cc; i += m) a += q[i];
            q[0] = a;
        }
        parts = next;
    } while (parts > 8);
    __syncthreads();
    return parts;
}

// Total over the positions p0 <= p < p0 + W of a row whose channel (p mod C)
// lies in group g; one wave, returned in every lane.
__device__ __forceinline__ double group_total(const RowSums& r, int W, int p0, int g, int cg, int C, int row)
{
    const int lane = (int)(threadIdx.x & 63);
    int lc = 0;                                    // lanes: 2^lc channels x the partial sums
    while (lc < 6 && (1 << lc) < cg) ++lc;
    double a = 0.0;
    for (int c0 = g * cg - p0; c0 < row - p0 && c0 < W; c0 += C)
        for (int f = lane & ((1 << lc) - 1); f < cg; f += 1 << lc)
            if (c0 + f >= 0 && c0 + f < W)
                for (int i = lane >> lc; i < r.parts; i += 64 >> lc) a += r.at(c0 + f, i);
    return wave_sum(a);
}

// log2 of the positions of V neighbouring ones that always lie in one group.
__host__ __device__ __forceinline__ int same_group(int cg, int V)
{
    int l = 0;
    while ((2 << l) <= V && cg % (2 << l) == 0) ++l;
    return l;
}

// Mean and 1 / sqrt(var + eps) from fp64 sums of x and x^2 over M values; low:
// what the fp32 mean lacks.
__device__ __forceinline__ float2 moments(double s, double ss, double M, float eps, float& low)
{
    const double mu = s / M;
    double var = ss / M - mu * mu;
    if (var < 0.0) var = 0.0;
    low = (float)(mu - (double)(float)mu);
    return make_float2((float)mu, (float)(1.0 / sqrt(var + (double)eps)));
}

// The channel and group of neighbouring row positions, without a division
// for each.
struct Channel {
    int c, g, r;      // channel, its group, its place in the group
    __device__ __forceinline__ Channel(int position, int C, int cg) : c(position % C), g(c / cg), r(c - g * cg) {}
    __device__ __forceinline__ void next(int C, int cg)
    {
        ++c;
        if (++r == cg) {
            r = 0;
            ++g;
        }
        if (c == C) c = g = 0;
    }
};

// ------------------------------------------------------------- activation
template <int ACT> __device__ __forceinline__ float act_fwd(float z, float slope)
{
    if (ACT == CF_ACT_SILU) return z * __builtin_amdgcn_rcpf(1.f + __expf(-z));
    return z > 0.f ? z : slope * z;
}

// dz = dy act'(z).  The leaky ReLU's derivative jumps at z = 0, where fp32's
// rounding of z can take the wrong side: within that rounding (2^-21 of the
// product's size covers its three roundings) the sign is taken in fp64.
template <int ACT>
__device__ __forceinline__ float act_bwd(float dy, float x, float mu, float rs, float xhat, float ga, float be,
                                         float slope)
{
    const float t = xhat * ga;
    const float z = t + be;
    if (ACT == CF_ACT_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
        return dy * (s * (1.f + z * (1.f - s)));
    }
    bool pos = z > 0.f;
    if (fabsf(z) <= 0x1p-21f * fabsf(t))
        pos = ((double)x - (double)mu) * (double)rs * (double)ga + (double)be > 0.0;
    return pos ? dy : slope * dy;
}

// -------------------------------------------------------- streaming forward
// Partial sums of x and x^2: part[n][group][block][chunk] = (sum, squares).
template <typename T, int V>
__global__ __launch_bounds__(GN_T) void gn_stats_kernel(const T* __restrict__ X, GnGeom q, double2* __restrict__ part)
{
    extern __shared__ double sh[];
    const int t = (int)threadIdx.x, r = t / q.cc, col = (int)blockIdx.y * q.cc + t % q.cc;
    const T* x = X + (int64_t)blockIdx.z * q.S + (int64_t)col * V;
    double s[V] = {}, ss[V] = {};
    auto add1 = [&](int j, T w) {
        const double d = (double)wide(w);
        s[j] += d;
        ss[j] = fma(d, d, ss[j]);
    };
    if (r < q.k && col < q.cols) {
        const int64_t step = (int64_t)q.nb * q.k;
        int64_t i = (int64_t)blockIdx.x * q.k + r;
        for (; i + 3 * step < q.nrows; i += 4 * step) {
            Vec<T, V> u[4];
#pragma unroll
            for (int l = 0; l < 4; ++l) u[l] = vload<T, V>(x + (i + l * step) * q.row);
#pragma unroll
            for (int l = 0; l < 4; ++l)
#pragma unroll
                for (int j = 0; j < V; ++j) add1(j, u[l].v[j]);
        }
        for (; i < q.nrows; i += step) {
            const Vec<T, V> u = vload<T, V>(x + i * q.row);
#pragma unroll
            for (int j = 0; j < V; ++j) add1(j, u.v[j]);
        }
        if (blockIdx.x == 0 && r == 0) {      // the values after the last whole row
            const int64_t left = q.S - q.nrows * q.row - (int64_t)col * V;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) add1(j, x[q.nrows * q.row + j]);
        }
    }
    const int lh = same_group(q.cg, V), nv = V >> lh, n = q.k * q.cc;
    put_rows<V>(s, sh, n, lh);
    put_rows<V>(ss, sh + nv * n, n, lh);
    RowSums a{sh, 31 - __builtin_clz(nv), n, q.cc, fold_rows(sh, 2 * nv, q.k, q.cc)};
    RowSums b = a;
    b.sh += nv * n;
    const int npart = q.nb * q.chunks;
    double2* out = part + (int64_t)blockIdx.z * q.G * npart + (int64_t)blockIdx.x * q.chunks + blockIdx.y;
    for (int g = t >> 6; g < q.G; g += (int)blockDim.x >> 6) {
        const int W = q.cc * nv, p0 = (int)blockIdx.y * W;
        const double x = group_total(a, W, p0, g, q.cg >> lh, q.C >> lh, q.row >> lh);
        const double y = group_total(b, W, p0, g, q.cg >> lh, q.C >> lh, q.row >> lh);
        if ((t & 63) == 0) out[(int64_t)g * npart] = make_double2(x, y);
    }
}

// y = act((x - mean) (rstd gamma) + beta), with the mean's low part in beta.
// Every block first adds its sample's partial sums (npart of them per group, in
// the same order).
template <typename T, int V, int ACT>
__global__ __launch_bounds__(GN_T) void gn_apply_kernel(const T* __restrict__ X, GnGeom q, int npart,
                                                        const double2* __restrict__ part,
                                                        const float* __restrict__ gamma,
                                                        const float* __restrict__ beta, float eps, float slope,
                                                        T* __restrict__ Y, float* __restrict__ mean,
                                                        float* __restrict__ rstd)
{
    extern __shared__ float2 stat[];     // [G] mean, rstd; then [G] the mean's low parts
    float* lows = reinterpret_cast<float*>(stat + q.G);
    const int t = (int)threadIdx.x, n = (int)blockIdx.z;
    const int r = t / q.cc, col = (int)blockIdx.y * q.cc + t % q.cc;
    const bool on = r < q.k && col < q.cols;
    const int64_t at = (int64_t)n * q.S + (int64_t)col * V, step = (int64_t)q.nb * q.k;
    const T* x = X + at;
    T* y = Y + at;
    // the first rows are on their way while the sums are added
    Vec<T, V> u[4];
    auto load = [&](int64_t i) {
#pragma unroll
        for (int l = 0; l < 4; ++l) u[l] = vload<T, V>(x + min(i + l * step, q.nrows - 1) * q.row);
    };
    int64_t i = (int64_t)blockIdx.x * q.k + r;
    if (on && i < q.nrows) load(i);
    part += (int64_t)n * npart * q.G;
    for (int g = t >> 6; g < q.G; g += (int)blockDim.x >> 6) {
        double s = 0.0, ss = 0.0;
        const double2* in = part + (int64_t)g * npart;
        int b = t & 63;
        for (; b + 192 < npart; b += 256) {
            double2 v[4];
#pragma unroll
            for (int l = 0; l < 4; ++l) v[l] = in[b + 64 * l];
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                s += v[l].x;
                ss += v[l].y;
            }
        }
        for (; b < npart; b += 64) {
            const double2 v = in[b];
            s += v.x;
            ss += v.y;
        }
        s = wave_sum(s);
        ss = wave_sum(ss);
        if ((t & 63) == 0) {
            float low;
            const float2 m = moments(s, ss, (double)(q.S / q.C) * q.cg, eps, low);
            stat[g] = m;
            lows[g] = low;
            if (blockIdx.x == 0 && blockIdx.y == 0) {
                mean[(int64_t)n * q.G + g] = m.x;
                rstd[(int64_t)n * q.G + g] = m.y;
            }
        }
    }
    __syncthreads();
    if (!on) return;
    float mu[V], sc[V], be[V];
    Channel ch(col * V, q.C, q.cg);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 m = stat[ch.g];
        mu[j] = m.x;
        sc[j] = m.y * gamma[ch.c];
        be[j] = fmaf(-lows[ch.g], sc[j], beta[ch.c]);
        ch.next(q.C, q.cg);
    }
    auto out1 = [&](int j, T w) { return act_fwd<ACT>(fmaf(wide(w) - mu[j], sc[j], be[j]), slope); };
    auto out = [&](const Vec<T, V>& u, int64_t i) {
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) narrow(o.v[j], out1(j, u.v[j]));
        vstore<T, V>(y + i * q.row, o);
    };
    for (; i + 3 * step < q.nrows; i += 4 * step) {
        Vec<T, V> v[4];
#pragma unroll
        for (int l = 0; l < 4; ++l) v[l] = u[l];
        if (i + 4 * step < q.nrows) load(i + 4 * step);
#pragma unroll
        for (int l = 0; l < 4; ++l) out(v[l], i + l * step);
    }
#pragma unroll
    for (int l = 0; l < 3; ++l)
        if (i + l * step < q.nrows) out(u[l], i + l * step);
    if (blockIdx.x == 0 && r == 0) {
        const int64_t left = q.S - q.nrows * q.row - (int64_t)col * V;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) narrow(y[q.nrows * q.row + j], out1(j, x[q.nrows * q.row + j]));
    }
}

// ------------------------------------------------------- streaming backward
// Per-channel partial sums of dz and dz xhat: part[n][block][chunk][channel].
template <typename T, int V, int ACT>
__global__ __launch_bounds__(GN_T) void gn_bwd_sums_kernel(const T* __restrict__ X, const T* __restrict__ dY,
                                                           GnGeom q, const float* __restrict__ gamma,
                                                           const float* __restrict__ beta,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, float slope,
                                                           double2* __restrict__ part)
{
    extern __shared__ double sh[];
    const int t = (int)threadIdx.x, r = t / q.cc, col = (int)blockIdx.y * q.cc + t % q.cc;
    const int64_t at = (int64_t)blockIdx.z * q.S + (int64_t)col * V;
    const T* x = X + at;
    const T* dy = dY + at;
    double a[V] = {}, b[V] = {};
    if (r < q.k && col < q.cols) {
        float mu[V], rs[V], ga[V], be[V];
        Channel ch(col * V, q.C, q.cg);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t g = (int64_t)blockIdx.z * q.G + ch.g;
            mu[j] = mean[g];
            rs[j] = rstd[g];
            ga[j] = gamma[ch.c];
            be[j] = beta[ch.c];
            ch.next(q.C, q.cg);
        }
        auto add1 = [&](int j, T xw, T dw) {
            const float xv = wide(xw), xhat = (xv - mu[j]) * rs[j];
            const float dz = act_bwd<ACT>(wide(dw), xv, mu[j], rs[j], xhat, ga[j], be[j], slope);
            a[j] += (double)dz;
            b[j] += (double)(dz * xhat);
        };
        const int64_t step = (int64_t)q.nb * q.k;
        int64_t i = (int64_t)blockIdx.x * q.k + r;
        for (; i + step < q.nrows; i += 2 * step) {
            Vec<T, V> u[2], d[2];
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                u[l] = vload<T, V>(x + (i + l * step) * q.row);
                d[l] = vload<T, V>(dy + (i + l * step) * q.row);
            }
#pragma unroll
            for (int l = 0; l < 2; ++l)
#pragma unroll
                for (int j = 0; j < V; ++j) add1(j, u[l].v[j], d[l].v[j]);
        }
        if (i < q.nrows) {
            const Vec<T, V> u = vload<T, V>(x + i * q.row), d = vload<T, V>(dy + i * q.row);
#pragma unroll
            for (int j = 0; j < V; ++j) add1(j, u.v[j], d.v[j]);
        }
        if (blockIdx.x == 0 && r == 0) {
            const int64_t left = q.S - q.nrows * q.row - (int64_t)col * V;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) add1(j, x[q.nrows * q.row + j], dy[q.nrows * q.row + j]);
        }
    }
    const int n = q.k * q.cc, p0 = (int)blockIdx.y * q.cc * V, W = q.cc * V;
    put_rows<V>(a, sh, n, 0);
    put_rows<V>(b, sh + V * n, n, 0);
    RowSums ra{sh, 31 - __builtin_clz(V), n, q.cc, fold_rows(sh, 2 * V, q.k, q.cc)};
    RowSums rb = ra;
    rb.sh += V * n;
    double2* out = part + (((int64_t)blockIdx.z * q.nb + blockIdx.x) * q.chunks + blockIdx.y) * q.C;
    for (int c = t; c < q.C; c += (int)blockDim.x) {
        double x = 0.0, y = 0.0;
        for (int p = c - p0; p < W && p < q.row - p0; p += q.C)
            if (p >= 0) {
                x += ra.total(p);
                y += rb.total(p);
            }
        out[c] = make_double2(x, y);
    }
}

// One block per (group, sample): the blocks' partials to per-sample channel
// sums chan[n][c] = (sum dz, sum dz xhat) and the group's s12[n][g] = (s1, s2).
constexpr int GN_TJ = 256;
__global__ __launch_bounds__(GN_TJ) void gn_bwd_join_kernel(GnGeom q, int npart, const double2* __restrict__ part,
                                                            const float* __restrict__ gamma,
                                                            double2* __restrict__ chan, float2* __restrict__ s12)
{
    __shared__ double la[GN_TJ], lb[GN_TJ];
    const int t = (int)threadIdx.x, g = (int)blockIdx.x, n = (int)blockIdx.y;
    const int cw = min(q.cg, GN_TJ), ways = GN_TJ / cw;      // `ways` threads share a channel
    part += (int64_t)n * npart * q.C;
    double s1 = 0.0, s2 = 0.0;
    for (int c0 = 0; c0 < q.cg; c0 += cw) {
        const int i = t % cw, way = t / cw, c = g * q.cg + c0 + i;
        const bool on = way < ways && c0 + i < q.cg;
        double a = 0.0, b = 0.0;
        if (on) {
            int p = way;
            for (; p + 7 * ways < npart; p += 8 * ways) {      // eight loads in flight
                double2 v[8];
#pragma unroll
                for (int l = 0; l < 8; ++l) v[l] = part[(int64_t)(p + l * ways) * q.C + c];
#pragma unroll
                for (int l = 0; l < 8; ++l) {
                    a += v[l].x;
                    b += v[l].y;
                }
            }
            for (; p < npart; p += ways) {
                const double2 v = part[(int64_t)p * q.C + c];
                a += v.x;
                b += v.y;
            }
        }
        __syncthreads();
        la[t] = a;
        lb[t] = b;
        __syncthreads();
        if (on && way == 0) {
            for (int w = 1; w < ways; ++w) {
                a += la[w * cw + i];
                b += lb[w * cw + i];
            }
            chan[(int64_t)n * q.C + c] = make_double2(a, b);
            s1 += (double)gamma[c] * a;
            s2 += (double)gamma[c] * b;
        }
    }
    __syncthreads();
    la[t] = s1;
    lb[t] = s2;
    __syncthreads();
    if (t < 64) {
        double a = 0.0, b = 0.0;
        for (int i = t; i < GN_TJ; i += 64) {
            a += la[i];
            b += lb[i];
        }
        a = wave_sum(a);
        b = wave_sum(b);
        const double M = (double)(q.S / q.C) * q.cg;
        if (t == 0) s12[(int64_t)n * q.G + g] = make_float2((float)(a / M), (float)(b / M));
    }
}

// dx = rstd (gamma dz - s1 - xhat s2); the first block of sample 0 also adds
// the samples' channel sums into dgamma and dbeta.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(GN_T) void gn_bwd_apply_kernel(const T* __restrict__ X, const T* __restrict__ dY,
                                                            GnGeom q, int N, const float* __restrict__ gamma,
                                                            const float* __restrict__ beta,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, float slope,
                                                            const double2* __restrict__ chan,
                                                            const float2* __restrict__ s12, T* __restrict__ dX,
                                                            float* __restrict__ dgamma, float* __restrict__ dbeta)
{
    const int t = (int)threadIdx.x, r = t / q.cc, col = (int)blockIdx.y * q.cc + t % q.cc;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int c = t; c < q.C; c += (int)blockDim.x) {
            double a = 0.0, b = 0.0;
            for (int n = 0; n < N; ++n) {
                const double2 v = chan[(int64_t)n * q.C + c];
                a += v.x;
                b += v.y;
            }
            dbeta[c] = (float)a;
            dgamma[c] = (float)b;
        }
    if (r >= q.k || col >= q.cols) return;
    const int64_t at = (int64_t)blockIdx.z * q.S + (int64_t)col * V, step = (int64_t)q.nb * q.k;
    const T* x = X + at;
    const T* dy = dY + at;
    T* dx = dX + at;
    float mu[V], rs[V], ga[V], be[V], s1[V], s2[V];
    Channel ch(col * V, q.C, q.cg);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int64_t g = (int64_t)blockIdx.z * q.G + ch.g;
        mu[j] = mean[g];
        rs[j] = rstd[g];
        ga[j] = gamma[ch.c];
        be[j] = beta[ch.c];
        s1[j] = s12[g].x;
        s2[j] = s12[g].y;
        ch.next(q.C, q.cg);
    }
    auto out1 = [&](int j, T xw, T dw) {
        const float xv = wide(xw), xhat = (xv - mu[j]) * rs[j];
        const float dz = act_bwd<ACT>(wide(dw), xv, mu[j], rs[j], xhat, ga[j], be[j], slope);
        return rs[j] * (fmaf(ga[j], dz, -s1[j]) - xhat * s2[j]);
    };
    auto out = [&](const Vec<T, V>& u, const Vec<T, V>& d, int64_t i) {
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) narrow(o.v[j], out1(j, u.v[j], d.v[j]));
        vstore<T, V>(dx + i * q.row, o);
    };
    int64_t i = (int64_t)blockIdx.x * q.k + r;
    for (; i + step < q.nrows; i += 2 * step) {
        Vec<T, V> u[2], d[2];
#pragma unroll
        for (int l = 0; l < 2; ++l) {
            u[l] = vload<T, V>(x + (i + l * step) * q.row);
            d[l] = vload<T, V>(dy + (i + l * step) * q.row);
        }
#pragma unroll
        for (int l = 0; l < 2; ++l) out(u[l], d[l], i + l * step);
    }
    if (i < q.nrows) out(vload<T, V>(x + i * q.row), vload<T, V>(dy + i * q.row), i);
    if (blockIdx.x == 0 && r == 0) {
        const int64_t left = q.S - q.nrows * q.row - (int64_t)col * V;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j < left) narrow(dx[q.nrows * q.row + j], out1(j, x[q.nrows * q.row + j], dy[q.nrows * q.row + j]));
    }
}

// ------------------------------------------------------------ small groups
// A slice of `gs` whole groups (row = gs * cg values, one row per voxel) of
// one sample held in one block's registers: nrows <= k * rows per thread.
struct GnSlice {
    int64_t S;       // values per sample
    int nrows;       // voxels per sample
    int C, G, cg;
    int gs;          // groups of a slice
    int cols;        // vectors of a slice's row
    int k;           // rows in flight
    int p;           // samples of a block (the backward's); p * k * cols <= threads
};

template <typename T, int V, int ACT>
__global__ __launch_bounds__(V == 8 ? GN_T : GN_TS) void gn_small_kernel(const T* __restrict__ X, GnSlice q,
                                                         const float* __restrict__ gamma,
                                                         const float* __restrict__ beta, float eps, float slope,
                                                         T* __restrict__ Y, float* __restrict__ mean,
                                                         float* __restrict__ rstd)
{
    extern __shared__ double sh[];
    const int t = (int)threadIdx.x, r = t / q.cols, col = t % q.cols, n = (int)blockIdx.y;
    const int W = q.gs * q.cg, c0 = (int)blockIdx.x * W, g0 = (int)blockIdx.x * q.gs;
    float2* stat = reinterpret_cast<float2*>(sh + q.k * W);      // [gs] mean, rstd; then [gs] sums of x, in whose
                                                                 // place the mean's low parts come
    const int64_t at = (int64_t)n * q.S + c0 + (int64_t)col * V;
    const double M = (double)q.nrows * q.cg;
    Vec<T, V> u[GN_ROWS_F];
    double s[V] = {}, ss[V] = {};
    const bool on = r < q.k;
#pragma unroll
    for (int l = 0; l < GN_ROWS_F; ++l) {
        const int i = r + l * q.k;
        if (on && i < q.nrows) u[l] = vload<T, V>(X + at + (int64_t)i * q.C);
    }
#pragma unroll
    for (int l = 0; l < GN_ROWS_F; ++l)
        if (on && r + l * q.k < q.nrows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const double d = (double)wide(u[l].v[j]);
                s[j] += d;
                ss[j] = fma(d, d, ss[j]);
            }
    const int lh = same_group(q.cg, V), nv = V >> lh, threads = q.k * q.cols;
    RowSums a{sh, 31 - __builtin_clz(nv), threads, q.cols, 0}, b = a;
    auto groups = [&](const RowSums& r, auto done) {
        for (int g = t >> 6; g < q.gs; g += (int)blockDim.x >> 6) {
            const double v = group_total(r, W >> lh, 0, g, q.cg >> lh, W >> lh, W >> lh);
            if ((t & 63) == 0) done(g, v);
        }
    };
    put_rows<V>(s, sh, threads, lh);
    if (lh > 0) {      // both sums fit
        put_rows<V>(ss, sh + nv * threads, threads, lh);
        a.parts = b.parts = fold_rows(sh, 2 * nv, q.k, q.cols);
        b.sh += nv * threads;
        groups(a, [&](int g, double v) { sh[q.k * W + q.gs + g] = v; });
    } else {
        a.parts = fold_rows(sh, nv, q.k, q.cols);
        groups(a, [&](int g, double v) { sh[q.k * W + q.gs + g] = v; });
        __syncthreads();
        put_rows<V>(ss, sh, threads, lh);
        b.parts = fold_rows(sh, nv, q.k, q.cols);
    }
    groups(b, [&](int g, double v) {
        float low;
        const float2 m = moments(sh[q.k * W + q.gs + g], v, M, eps, low);
        stat[g] = m;
        sh[q.k * W + q.gs + g] = (double)low;
        mean[(int64_t)n * q.G + g0 + g] = m.x;
        rstd[(int64_t)n * q.G + g0 + g] = m.y;
    });
    __syncthreads();
    if (!on) return;
    float mu[V], sc[V], be[V];
    Channel ch(col * V, W, q.cg);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 m = stat[ch.g];
        mu[j] = m.x;
        sc[j] = m.y * gamma[c0 + col * V + j];
        be[j] = fmaf(-(float)sh[q.k * W + q.gs + ch.g], sc[j], beta[c0 + col * V + j]);
        ch.next(W, q.cg);
    }
#pragma unroll
    for (int l = 0; l < GN_ROWS_F; ++l) {
        const int i = r + l * q.k;
        if (i >= q.nrows) continue;
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j)
            narrow(o.v[j], act_fwd<ACT>(fmaf(wide(u[l].v[j]) - mu[j], sc[j], be[j]), slope));
        vstore<T, V>(Y + at + (int64_t)i * q.C, o);
    }
}

// The backward of a slice.  Where a block holds all samples beside each other
// it writes dgamma and dbeta; else it takes one sample and writes its channel
// sums, which gn_bwd_small_join_kernel adds.  (2 x 8^3 x 256 fp32: one launch
// 9.0 us, two 9.9; the samples one after another in one block 12.9, and 3 to 8
// us for each further one.  8 x 8^3 x 256 bf16: two launches 15.4, streaming
// 23.3.)
template <typename T, int V, int ACT>
__global__ __launch_bounds__(GN_T) void gn_bwd_small_kernel(const T* __restrict__ X, const T* __restrict__ dY,
                                                             GnSlice q, const float* __restrict__ gamma,
                                                             const float* __restrict__ beta,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, float slope,
                                                             T* __restrict__ dX, float* __restrict__ dgamma,
                                                             float* __restrict__ dbeta, double2* __restrict__ part)
{
    extern __shared__ double sh[];
    const int t = (int)threadIdx.x, T_ = (int)blockDim.x, per = q.k * q.cols, p = t / per, tp = t - p * per;
    const int r = tp / q.cols, col = tp % q.cols, n0 = (int)blockIdx.y * q.p, n = n0 + p;
    const int W = q.gs * q.cg, c0 = (int)blockIdx.x * W, g0 = (int)blockIdx.x * q.gs;
    double* cha = sh + q.p * q.k * W;        // [p][W] channel sums of dz, then of dz xhat
    double* chb = cha + q.p * W;
    float2* s12 = reinterpret_cast<float2*>(chb + q.p * W);
    float2* stat = s12 + q.p * q.gs;         // [p][gs] mean, rstd
    const double M = (double)q.nrows * q.cg;
    const bool on = p < q.p;
    const int64_t at = (int64_t)n * q.S + c0 + (int64_t)col * V;
    Vec<T, V> u[GN_ROWS_B], d[GN_ROWS_B];
    float ga[V] = {}, be[V] = {};
    if (on) {
#pragma unroll
        for (int l = 0; l < GN_ROWS_B; ++l) {
            const int i = min(r + l * q.k, q.nrows - 1);
            u[l] = vload<T, V>(X + at + (int64_t)i * q.C);
            d[l] = vload<T, V>(dY + at + (int64_t)i * q.C);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            ga[j] = gamma[c0 + col * V + j];
            be[j] = beta[c0 + col * V + j];
        }
    }
    for (int e = t; e < q.p * q.gs; e += T_) {
        const int64_t i = (int64_t)(n0 + e / q.gs) * q.G + g0 + e % q.gs;
        stat[e] = make_float2(mean[i], rstd[i]);
    }
    __syncthreads();
    const Channel first(col * V, W, q.cg);
    float mu[V] = {}, rs[V] = {};
    if (on) {
        Channel ch = first;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mu[j] = stat[p * q.gs + ch.g].x;
            rs[j] = stat[p * q.gs + ch.g].y;
            ch.next(W, q.cg);
        }
    }
    double a[V] = {}, b[V] = {};
#pragma unroll
    for (int l = 0; l < GN_ROWS_B; ++l)
        if (on && r + l * q.k < q.nrows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xv = wide(u[l].v[j]), xhat = (xv - mu[j]) * rs[j];
                const float dz = act_bwd<ACT>(wide(d[l].v[j]), xv, mu[j], rs[j], xhat, ga[j], be[j], slope);
                a[j] += (double)dz;
                b[j] += (double)(dz * xhat);
            }
    // channel sums of each sample
    auto sums = [&](const double (&v)[V], double* to) {
        put_rows<V>(v, sh + p * V * per, per, 0, on ? tp : per);
        const int parts = fold_rows(sh, q.p * V, q.k, q.cols);
        for (int e = t; e < q.p * W; e += T_) {
            const int i = e / W;
            to[e] = RowSums{sh + i * V * per, 31 - __builtin_clz(V), per, q.cols, parts}.total(e - i * W);
        }
        __syncthreads();
    };
    sums(a, cha);
    sums(b, chb);
    for (int g = t >> 6; g < q.p * q.gs; g += T_ >> 6) {
        double s1 = 0.0, s2 = 0.0;
        const int c = g % q.gs * q.cg;
        for (int i = t & 63; i < q.cg; i += 64) {
            const double gm = (double)gamma[c0 + c + i];
            s1 += gm * cha[g * q.cg + i];
            s2 += gm * chb[g * q.cg + i];
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if ((t & 63) == 0) s12[g] = make_float2((float)(s1 / M), (float)(s2 / M));
    }
    __syncthreads();
    for (int c = t; c < W; c += T_) {
        double ta = 0.0, tb = 0.0;
        for (int i = 0; i < q.p; ++i) {
            ta += cha[i * W + c];
            tb += chb[i * W + c];
        }
        if (part) {
            part[(int64_t)n0 * q.C + c0 + c] = make_double2(ta, tb);
        } else {
            dbeta[c0 + c] = (float)ta;
            dgamma[c0 + c] = (float)tb;
        }
    }
    if (!on) return;
    float s1[V], s2[V];
    Channel ch = first;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float2 v = s12[p * q.gs + ch.g];
        s1[j] = v.x;
        s2[j] = v.y;
        ch.next(W, q.cg);
    }
#pragma unroll
    for (int l = 0; l < GN_ROWS_B; ++l) {
        const int i = r + l * q.k;
        if (i >= q.nrows) continue;
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xv = wide(u[l].v[j]), xhat = (xv - mu[j]) * rs[j];
            const float dz = act_bwd<ACT>(wide(d[l].v[j]), xv, mu[j], rs[j], xhat, ga[j], be[j], slope);
            narrow(o.v[j], rs[j] * (fmaf(ga[j], dz, -s1[j]) - xhat * s2[j]));
        }
        vstore<T, V>(dX + at + (int64_t)i * q.C, o);
    }
}

// dgamma and dbeta: 32 channels a block, eight threads to a channel's samples.
__global__ __launch_bounds__(256) void gn_bwd_small_join_kernel(int C, int N, const double2* __restrict__ part,
                                                                float* __restrict__ dgamma, float* __restrict__ dbeta)
{
    __shared__ double2 sh[8][32];
    const int i = (int)threadIdx.x % 32, way = (int)threadIdx.x / 32, c = (int)blockIdx.x * 32 + i;
    double2 a = make_double2(0.0, 0.0);
    if (c < C)
        for (int n = way; n < N; n += 8) {
            const double2 v = part[(int64_t)n * C + c];
            a.x += v.x;
            a.y += v.y;
        }
    sh[way][i] = a;
    __syncthreads();
    if (way || c >= C) return;
    for (int w = 1; w < 8; ++w) {
        a.x += sh[w][i].x;
        a.y += sh[w][i].y;
    }
    dbeta[c] = (float)a.x;
    dgamma[c] = (float)a.y;
}

// -------------------------------------------------------------------- plans
int up64(int v) { return (v + 63) / 64 * 64; }
size_t up256b(size_t b) { return (b + 255) & ~(size_t)255; }

template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

template <typename T> GnGeom gn_geom(const cf_dims& x, int G)
{
    constexpr int V = vec_of<T>();
    GnGeom q{};
    q.C = (int)x.c;
    q.G = G;
    q.cg = q.C / G;
    q.S = x.d * x.h * x.w * x.c;
    q.row = (int)std::lcm((int64_t)V, x.c);
    q.cols = q.row / V;
    q.chunks = (q.cols + GN_T - 1) / GN_T;
    q.cc = (q.cols + q.chunks - 1) / q.chunks;
    q.k = GN_T / q.cc;
    q.nrows = q.S / q.row;
    // eight rows for each thread (a block's coefficients and sums cost as much), four where that leaves CUs idle
    int64_t want = (q.nrows + 8 * q.k - 1) / (8 * q.k);
    if (want * x.n * q.chunks < GN_FEW) want = (q.nrows + 4 * q.k - 1) / (4 * q.k);
    int64_t most = GN_BLOCKS / (x.n * q.chunks);
    if (most < 1) most = 1;
    q.nb = (int)(want < 1 ? 1 : want < most ? want : most);
    return q;
}

// The slice plan of a shape, or cols = 0 where a group does not fit one block.
// `held` vectors per thread, `arrays` doubles per channel beside the sums in
// LDS (2 in the backward), `p` samples of a block.
template <int V> GnSlice gn_slice(const cf_dims& x, int G, int esize, int threads, int held, int arrays, int p)
{
    threads /= p;
    GnSlice q{};
    const int64_t vox = x.d * x.h * x.w;
    q.C = (int)x.c;
    q.G = G;
    q.cg = q.C / G;
    q.S = vox * x.c;
    if (vox > (int64_t)threads * held || q.C % V) return q;
    q.nrows = (int)vox;
    q.p = p;
    // whole vectors, and 64 bytes of a voxel where the registers allow it and many blocks are left: what a block
    // computes takes longer than what it reads while every CU has one block at most (backward of 12 x 8^3 x 256 bf16:
    // 384 blocks of 16 bytes 26.4 us, 192 of 32 bytes 13.7)
    for (int gs = 1; gs <= G; ++gs) {
        const int W = gs * q.cg;
        if (G % gs || W % V) continue;
        const int cols = W / V;
        if (cols > threads) break;
        const int k = (int)std::min<int64_t>(vox, threads / cols);
        if ((vox + k - 1) / k > held) break;
        if (p * ((size_t)(k + arrays) * W + 2 * gs) * sizeof(double) > GN_LDS) break;
        q.gs = gs;
        q.cols = cols;
        q.k = k;
        if (W * esize >= 64 || G / gs * (x.n / p) <= GN_SLICES) break;
    }
    // more blocks of narrow slices take longer than streaming (24 x 12^3 x 128 bf16: 46.9 us, 41.0)
    if (q.cols && q.gs < G && q.gs * q.cg * esize < 64 && G / q.gs * (x.n / p) > GN_SLICES) q.cols = 0;
    return q;
}

template <typename T> GnSlice fwd_slice(const cf_dims& x, int G, int* V)
{
    constexpr int v = vec_of<T>();
    *V = v;
    GnSlice q = gn_slice<v>(x, G, (int)sizeof(T), v == 8 ? GN_T : GN_TS, GN_ROWS_F, 0, 1);
    if (q.cols) return q;
    *V = 1;
    return gn_slice<1>(x, G, (int)sizeof(T), GN_TS, GN_ROWS_F, 0, 1);
}
template <typename T> GnSlice bwd_slice(const cf_dims& x, int G, int* V)
{
    constexpr int v = vec_of<T>();
    // all samples in a block, if they fit, then one
    for (int p : {(int)x.n, 1}) {
        if (p > GN_T) continue;
        *V = v;
        GnSlice q = gn_slice<v>(x, G, (int)sizeof(T), GN_T, GN_ROWS_B, 2, p);
        if (q.cols) return q;
        *V = 1;
        q = gn_slice<1>(x, G, (int)sizeof(T), GN_T, GN_ROWS_B, 2, p);
        if (q.cols) return q;
    }
    return GnSlice{};
}

template <typename T, int V, int ACT>
hipError_t run_small_fwd(const GnSlice& q, int64_t N, const T* X, const float* gamma, const float* beta, float eps,
                         float slope, T* Y, float* mean, float* rstd, hipStream_t s)
{
    const size_t lds = ((size_t)q.k * q.gs * q.cg + 2 * q.gs) * sizeof(double);
    hipLaunchKernelGGL((gn_small_kernel<T, V, ACT>), dim3((unsigned)(q.G / q.gs), (unsigned)N),
                       dim3((unsigned)up64(q.k * q.cols)), lds, s, X, q, gamma, beta, eps, slope, Y, mean, rstd);
    return hipGetLastError();
}

template <typename T, int V, int ACT>
hipError_t run_small_bwd(const GnSlice& q, int64_t N, const T* X, const T* dY, const float* gamma, const float* beta,
                         const float* mean, const float* rstd, float slope, T* dX, float* dgamma, float* dbeta,
                         double2* part, hipStream_t s)
{
    const size_t lds = q.p * ((size_t)(q.k + 2) * q.gs * q.cg + 2 * q.gs) * sizeof(double);
    const bool join = N > q.p;
    hipLaunchKernelGGL((gn_bwd_small_kernel<T, V, ACT>), dim3((unsigned)(q.G / q.gs), (unsigned)(N / q.p)),
                       dim3((unsigned)up64(q.p * q.k * q.cols)), lds, s, X, dY, q, gamma, beta, mean, rstd, slope, dX,
                       dgamma, dbeta, join ? part : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !join) return e;
    hipLaunchKernelGGL(gn_bwd_small_join_kernel, dim3((unsigned)((q.C + 31) / 32)), dim3(256), 0, s, q.C, (int)N,
                       (const double2*)part, dgamma, dbeta);
    return hipGetLastError();
}

template <typename T, int ACT>
hipError_t run_fwd(const T* X, const float* gamma, const float* beta, float eps, float slope, T* Y, float* mean,
                   float* rstd, const cf_dims& x, int G, void* ws, hipStream_t s)
{
    constexpr int V = vec_of<T>();
    int v;
    const GnSlice sl = fwd_slice<T>(x, G, &v);
    if (sl.cols)
        return v == 1 ? run_small_fwd<T, 1, ACT>(sl, x.n, X, gamma, beta, eps, slope, Y, mean, rstd, s)
                      : run_small_fwd<T, V, ACT>(sl, x.n, X, gamma, beta, eps, slope, Y, mean, rstd, s);
    const GnGeom q = gn_geom<T>(x, G);
    const dim3 grid((unsigned)q.nb, (unsigned)q.chunks, (unsigned)x.n), block((unsigned)up64(q.k * q.cc));
    double2* part = (double2*)ws;
    hipLaunchKernelGGL((gn_stats_kernel<T, V>), grid, block,
                       (size_t)q.k * q.cc * (2 * V >> same_group(q.cg, V)) * sizeof(double), s, X, q, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gn_apply_kernel<T, V, ACT>), grid, block, (size_t)G * (sizeof(float2) + sizeof(float)), s, X, q,
                       q.nb * q.chunks, (const double2*)part, gamma, beta, eps, slope, Y, mean, rstd);
    return hipGetLastError();
}

template <typename T, int ACT>
hipError_t run_bwd(const T* X, const T* dY, const float* gamma, const float* beta, const float* mean,
                   const float* rstd, float slope, T* dX, float* dgamma, float* dbeta, const cf_dims& x, int G,
                   void* ws, hipStream_t s)
{
    constexpr int V = vec_of<T>();
    int v;
    const GnSlice sl = bwd_slice<T>(x, G, &v);
    if (sl.cols)
        return v == 1 ? run_small_bwd<T, 1, ACT>(sl, x.n, X, dY, gamma, beta, mean, rstd, slope, dX, dgamma, dbeta,
                                                 (double2*)ws, s)
                      : run_small_bwd<T, V, ACT>(sl, x.n, X, dY, gamma, beta, mean, rstd, slope, dX, dgamma, dbeta,
                                                 (double2*)ws, s);
    const GnGeom q = gn_geom<T>(x, G);
    const int npart = q.nb * q.chunks;
    char* p = (char*)ws;
    double2* part = (double2*)p;
    p += up256b((size_t)x.n * npart * q.C * sizeof(double2));
    double2* chan = (double2*)p;
    p += up256b((size_t)x.n * q.C * sizeof(double2));
    float2* s12 = (float2*)p;
    const dim3 grid((unsigned)q.nb, (unsigned)q.chunks, (unsigned)x.n), block((unsigned)up64(q.k * q.cc));
    hipLaunchKernelGGL((gn_bwd_sums_kernel<T, V, ACT>), grid, block, (size_t)q.k * q.cc * 2 * V * sizeof(double), s, X, dY,
                       q, gamma, beta, mean, rstd, slope, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gn_bwd_join_kernel, dim3((unsigned)G, (unsigned)x.n), dim3(GN_TJ), 0, s, q, npart,
                       (const double2*)part, gamma, chan, s12);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((gn_bwd_apply_kernel<T, V, ACT>), grid, block, 0, s, X, dY, q, (int)x.n, gamma, beta, mean,
                       rstd, slope, (const double2*)chan, (const float2*)s12, dX, dgamma, dbeta);
    return hipGetLastError();
}

template <typename T> size_t ws_bytes(const cf_dims& x, int G, bool bwd)
{
    int v;
    const GnSlice sl = bwd ? bwd_slice<T>(x, G, &v) : fwd_slice<T>(x, G, &v);
    if (sl.cols) return bwd && x.n > sl.p ? up256b((size_t)x.n * x.c * sizeof(double2)) : 0;
    const GnGeom q = gn_geom<T>(x, G);
    const size_t npart = (size_t)x.n * q.nb * q.chunks;
    if (!bwd) return up256b(npart * G * sizeof(double2));
    return up256b(npart * q.C * sizeof(double2)) + up256b((size_t)x.n * q.C * sizeof(double2)) +
           up256b((size_t)x.n * G * sizeof(float2));
}

}  // namespace

size_t gn_ws_bytes(cf_dtype dt, const cf_dims& x, int G, bool bwd)
{
    return dt == CF_F32 ? ws_bytes<float>(x, G, bwd) : ws_bytes<uint16_t>(x, G, bwd);
}

template <typename T>
hipError_t launch_gn_fwd(const T* X, const float* gamma, const float* beta, float eps, cf_act act, float slope, T* Y,
                         float* mean, float* rstd, const cf_dims& x, int G, void* ws, hipStream_t s)
{
    return act == CF_ACT_SILU
               ? run_fwd<T, CF_ACT_SILU>(X, gamma, beta, eps, slope, Y, mean, rstd, x, G, ws, s)
               : run_fwd<T, CF_ACT_LRELU>(X, gamma, beta, eps, slope, Y, mean, rstd, x, G, ws, s);
}

template <typename T>
hipError_t launch_gn_bwd(const T* X, const T* dY, const float* gamma, const float* beta, const float* mean,
                         const float* rstd, cf_act act, float slope, T* dX, float* dgamma, float* dbeta,
                         const cf_dims& x, int G, void* ws, hipStream_t s)
{
    return act == CF_ACT_SILU ? run_bwd<T, CF_ACT_SILU>(X, dY, gamma, beta, mean, rstd, slope, dX, dgamma, dbeta, x,
                                                        G, ws, s)
                              : run_bwd<T, CF_ACT_LRELU>(X, dY, gamma, beta, mean, rstd, slope, dX, dgamma, dbeta, x,
                                                         G, ws, s);
}

template hipError_t launch_gn_fwd<float>(const float*, const float*, const float*, float, cf_act, float, float*,
                                         float*, float*, const cf_dims&, int, void*, hipStream_t);
template hipError_t launch_gn_fwd<uint16_t>(const uint16_t*, const float*, const float*, float, cf_act, float,
                                            uint16_t*, float*, float*, const cf_dims&, int, void*, hipStream_t);
template hipError_t launch_gn_bwd<float>(const float*, const float*, const float*, const float*, const float*,
                                         const float*, cf_act, float, float*, float*, float*, const cf_dims&, int,
                                         void*, hipStream_t);
template hipError_t launch_gn_bwd<uint16_t>(const uint16_t*, const uint16_t*, const float*, const float*,
                                            const float*, const float*, cf_act, float, uint16_t*, float*, float*,
                                            const cf_dims&, int, void*, hipStream_t);

}  // namespace cf
