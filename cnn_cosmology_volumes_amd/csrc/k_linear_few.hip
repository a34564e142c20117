// Linear layers of a few rows (a dense head's small batches, serving): bound by the
// weights' bytes and by launches, so each direction is one launch in fp32
// arithmetic, and no partial sums leave a block.
//
// 1 x 2048 x 2048 bf16 takes 6.8 us (8.4 MB, 1.7 us of a copy; the call 8.8 to 9.4):
// its 64 blocks are a quarter of the chip's CUs, each with a whole reduction.  8 x 2048
// x 256 fp32 backward takes 5.1 (the call 12), where products, joins and all take 14
// and 26; 4 x 4096 x 4096 bf16 backward 31 us, its 100 MB at 3.3 TB/s.
#include "linear_common.h"

namespace cf {
namespace {

// v of the 16 lanes of a row, `by` further on.
template <int BY> __device__ __forceinline__ float rotated(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + BY, 0xf, 0xf, true));
}
// Sum over the wave's lanes that are equal modulo LP, in each of them.
template <int LP> __device__ __forceinline__ float lanes_sum(float v)
{
    if (LP <= 1) v += rotated<1>(v);
    if (LP <= 2) v += rotated<2>(v);
    if (LP <= 4) v += rotated<4>(v);
    v += rotated<8>(v);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Forward.  A block takes LP V columns with the whole reduction: LP lanes to a row
// of W, and each group of LP lanes takes V values of the reduction at a time, so
// that X is read 16 bytes at a time too and V loads of W are in flight a thread.
// ROWS rows of X a block (blockIdx.y: which).
template <int ROWS> constexpr int few_threads() { return ROWS >= 8 ? 512 : 1024; }
template <typename T, int ROWS, int LP>
__global__ __launch_bounds__(few_threads<ROWS>()) void lin_few_fwd_kernel(LinProduct<T> q)
{
    constexpr int V = 16 / (int)sizeof(T), THREADS = few_threads<ROWS>(), WAVES = THREADS / 64, COLS = LP * V;
    __shared__ float sh[WAVES][ROWS][COLS];
    const int lane = (int)threadIdx.x % LP, group = (int)threadIdx.x / LP;
    const int n = ((int)blockIdx.x * LP + lane) * V, r0 = (int)blockIdx.y * ROWS;
    const int K = (int)q.K;
    float acc[ROWS][V] = {};
    auto multiply = [&](const uint4 (&w)[V], const uint4 (&x)[ROWS]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            T t[V];
            __builtin_memcpy(t, &w[j], 16);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                T u[V];
                __builtin_memcpy(u, &x[r], 16);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[r][i] = fmaf(widen(u[j]), widen(t[i]), acc[r][i]);
            }
        }
    };
    // (rows past the last: the last one's sums again, which are not written)
    int k = group * V;
    if (((int)blockIdx.x + 1) * COLS <= q.N)      // loads without conditions go out one behind the other
        for (; k + V <= K; k += THREADS / LP * V) {
            uint4 w[V], x[ROWS];
#pragma unroll
            for (int j = 0; j < V; ++j) __builtin_memcpy(&w[j], q.B + (int64_t)(k + j) * q.N + n, 16);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) __builtin_memcpy(&x[r], q.A + (int64_t)min(r0 + r, (int)q.M - 1) * K + k, 16);
            multiply(w, x);
        }
    for (; k < K; k += THREADS / LP * V) {
        uint4 w[V], x[ROWS];
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = lin_chunk<T>(q.B + (int64_t)(k + j) * q.N + n, k + j < K ? q.N - n : 0, q.N >= V);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) x[r] = lin_chunk<T>(q.A + (int64_t)min(r0 + r, (int)q.M - 1) * K + k, K - k, K >= V);
        multiply(w, x);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = lanes_sum<LP>(acc[r][i]);
            if ((threadIdx.x & 63) < LP) sh[threadIdx.x >> 6][r][lane * V + i] = v;
        }
    __syncthreads();
    for (int t = (int)threadIdx.x; t < ROWS * COLS; t += THREADS) {
        const int r = r0 + t / COLS, c = (int)blockIdx.x * COLS + t % COLS;
        if (r >= (int)q.M || c >= q.N) continue;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) v += sh[i][t / COLS][t % COLS];
        const int64_t at = (int64_t)r * q.N + c;
        if (q.bias) v += q.bias[c];
        if (q.pre) Elem<T>::store(q.pre, at, v);
        v = lin_act<T>(q.act, v);
        if (q.R) v += widen(q.R[at]);
        Elem<T>::store((T*)q.C, at, v);
    }
}

// Backward.  A wave takes IN rows of W (and of dW), a block 8 waves; D = dY
// act'(pre) of 64 V columns at a time is formed once a block, in LDS.  From it and
// a row of W come that row's part of dX (the sums over the columns stay in
// registers to the end) and the row of dW.
constexpr int FEW_WAVES = 8;
// (what the registers hold; more rows a wave leave CUs idle: 4 x 4096 x 4096 bf16 31 us with two, 42 with four)
template <typename T, int ROWS> constexpr int few_in() { return ROWS * 16 / (int)sizeof(T) > 64 ? 1 : 2; }
template <typename T> struct FewBwd {
    const T *X, *W, *pre, *dY;
    T* dX;
    float *dW, *db;
    int rows, in, out;
    LinAct act;
    bool gated;
};
template <typename T, int ROWS>
__global__ __launch_bounds__(64 * FEW_WAVES) void lin_few_bwd_kernel(FewBwd<T> q)
{
    constexpr int V = 16 / (int)sizeof(T), CHUNK = 64 * V, IN = few_in<T, ROWS>();
    // value v of lane l at [v / 4][l][v % 4]: lanes read 16 bytes side by side
    __shared__ __attribute__((aligned(16))) float sd[ROWS][V / 4][64][4];
    __shared__ float sx[IN * FEW_WAVES][ROWS];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int first = (int)blockIdx.x * (IN * FEW_WAVES), i0 = first + wave * IN;
    for (int t = (int)threadIdx.x; t < IN * FEW_WAVES * ROWS; t += 64 * FEW_WAVES) {
        const int i = t % (IN * FEW_WAVES), r = t / (IN * FEW_WAVES);
        sx[i][r] = r < q.rows && first + i < q.in ? widen(q.X[(int64_t)r * q.in + first + i]) : 0.f;
    }
    float acc[IN][ROWS] = {};
    // The next columns' values are under way while these are worked on.  (Rows past the last, of W and of D:
    // the last one's, which reach nothing that is written but for D's, which are zeroed.)
    constexpr int MINE = (ROWS + FEW_WAVES - 1) / FEW_WAVES;      // rows of D that a wave forms
    uint4 w[IN], dv[MINE], zv[MINE];
    auto fetch = [&](int c0) {
        const int c = c0 + lane * V;
        const bool inside = c0 + CHUNK <= q.out;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const T* from = q.W + (int64_t)min(i0 + i, q.in - 1) * q.out + c;
            if (inside) __builtin_memcpy(&w[i], from, 16);
            else w[i] = lin_chunk<T>(from, q.out - c, q.out >= V);
        }
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
            const int64_t at = (int64_t)min(wave + m * FEW_WAVES, q.rows - 1) * q.out + c;
            if (inside) __builtin_memcpy(&dv[m], q.dY + at, 16);
            else dv[m] = lin_chunk<T>(q.dY + at, q.out - c, q.out >= V);
            if (!q.gated) continue;
            if (inside) __builtin_memcpy(&zv[m], q.pre + at, 16);
            else zv[m] = lin_chunk<T>(q.pre + at, q.out - c, q.out >= V);
        }
    };
    fetch(0);
    for (int c0 = 0; c0 < q.out; c0 += CHUNK) {
        const int c = c0 + lane * V, left = q.out - c;
        lds_barrier();      // (leaves the stores to dW and the next columns' loads in flight)
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
            const int r = wave + m * FEW_WAVES;
            if (r >= ROWS) break;
            T d[V], z[V];
            __builtin_memcpy(d, &dv[m], 16);
            __builtin_memcpy(z, &zv[m], 16);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = q.gated ? widen(d[j]) * lin_dact<T>(q.act, widen(z[j])) : widen(d[j]);
                sd[r][j / 4][lane][j % 4] = r < q.rows ? v : 0.f;
            }
        }
        lds_barrier();
        float wf[IN][V], dw[IN][V] = {}, sum[V] = {};
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            T t[V];
            __builtin_memcpy(t, &w[i], 16);
#pragma unroll
            for (int j = 0; j < V; ++j) wf[i][j] = widen(t[j]);
        }
        if (c0 + CHUNK < q.out) fetch(c0 + CHUNK);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float d[V];
#pragma unroll
            for (int j = 0; j < V; j += 4) __builtin_memcpy(d + j, sd[r][j / 4][lane], 16);
#pragma unroll
            for (int i = 0; i < IN; ++i) {
                const float x = sx[wave * IN + i][r];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    acc[i][r] = fmaf(wf[i][j], d[j], acc[i][r]);
                    dw[i][j] = fmaf(x, d[j], dw[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += d[j];
        }
#pragma unroll
        for (int i = 0; i < IN; ++i)
            if (i0 + i < q.in && left > 0) {
                float* to = q.dW + (int64_t)(i0 + i) * q.out + c;
                if (left >= V) __builtin_memcpy(to, dw[i], 4 * V);
                else
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (j < left) to[j] = dw[i][j];
            }
        // the blocks write the columns' sums in turn
        if (q.db && wave == 0 && c0 / CHUNK % (int)gridDim.x == (int)blockIdx.x)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) q.db[c + j] = sum[j];
    }
    if (!q.dX) return;
    // lane i ROWS + r keeps dX[r][i0 + i]
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < IN; ++i)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float v = lanes_sum<1>(acc[i][r]);
            if (lane == i * ROWS + r) mine = v;
        }
    const int i = i0 + lane / ROWS, r = lane % ROWS;
    if (lane < IN * ROWS && i < q.in && r < q.rows) Elem<T>::store(q.dX, (int64_t)r * q.in + i, mine);
}

template <typename T, int ROWS> void few_fwd(const LinProduct<T>& q, hipStream_t s)
{
    // Rows of W are read 64 bytes at a time where that leaves 32 blocks or more, else 16.
    constexpr int V = 16 / (int)sizeof(T);
    const int wide = (q.N + 4 * V - 1) / (4 * V), narrow = (q.N + V - 1) / V;
    const unsigned groups = (unsigned)((q.M + ROWS - 1) / ROWS);
    if (wide >= 32) lin_few_fwd_kernel<T, ROWS, 4><<<dim3((unsigned)wide, groups), few_threads<ROWS>(), 0, s>>>(q);
    else lin_few_fwd_kernel<T, ROWS, 1><<<dim3((unsigned)narrow, groups), few_threads<ROWS>(), 0, s>>>(q);
}

}  // namespace

template <typename T> hipError_t launch_lin_few_fwd(const LinProduct<T>& q, hipStream_t s)
{
    if (q.M <= 1) few_fwd<T, 1>(q, s);
    else if (q.M <= 2) few_fwd<T, 2>(q, s);
    else if (q.M <= 4) few_fwd<T, 4>(q, s);
    else few_fwd<T, 8>(q, s);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_lin_few_bwd(int rows, int in, int out, const T* X, const T* W, const T* pre, const T* dY, LinAct act,
                              bool gated, T* dX, float* dW, float* db, hipStream_t s)
{
    const FewBwd<T> q = {X, W, pre, dY, dX, dW, db, rows, in, out, act, gated};
    auto grid = [&](int each) { return (unsigned)((in + each * FEW_WAVES - 1) / (each * FEW_WAVES)); };
    if (rows <= 4) lin_few_bwd_kernel<T, 4><<<grid(few_in<T, 4>()), 64 * FEW_WAVES, 0, s>>>(q);
    else if (rows <= 8) lin_few_bwd_kernel<T, 8><<<grid(few_in<T, 8>()), 64 * FEW_WAVES, 0, s>>>(q);
    else lin_few_bwd_kernel<T, 16><<<grid(few_in<T, 16>()), 64 * FEW_WAVES, 0, s>>>(q);
    return hipGetLastError();
}

#define CF_LIN_FEW(T)                                                                                                \
    template hipError_t launch_lin_few_fwd<T>(const LinProduct<T>&, hipStream_t);                                    \
    template hipError_t launch_lin_few_bwd<T>(int, int, int, const T*, const T*, const T*, const T*, LinAct, bool, T*, \
                                              float*, float*, hipStream_t);
CF_LIN_FEW(float)
CF_LIN_FEW(uint16_t)

}  // namespace cf
