// Shared by the linear layers' products (k_linear.hip, k_linear_mm.hip).
#pragma once

#include "cf_internal.h"

#include <math.h>

namespace cf {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

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

// Orders a wave's LDS accesses: what its lanes wrote is read by other lanes.
__device__ __forceinline__ void lin_wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

// Eight neighbouring values of the result, of which n are inside.
template <typename T> __device__ __forceinline__ void load8(const T* p, int n, float (&v)[8])
{
    T t[8] = {};
    if (n >= 8) __builtin_memcpy(t, p, sizeof(t));
    else
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) t[i] = p[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = widen(t[i]);
}
template <typename T> __device__ __forceinline__ void store8(T* p, int n, const float (&v)[8])
{
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) Elem<T>::store(t, i, v[i]);
    if (n >= 8) __builtin_memcpy(p, t, sizeof(t));
    else
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = t[i];
}
// bias and r: the values' own bias and residual (LIN_FWD).
template <typename T, typename TO, int MODE>
__device__ __forceinline__ void lin_result(const LinProduct<T>& q, int64_t m, int n, float (&v)[8], const float (&bias)[8],
                                           const float (&r)[8])
{
    const int64_t at = m * q.N + n;
    if (MODE == LIN_FWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (q.pre) store8(q.pre + at, q.N - n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lin_act(q.act, v[i]) + r[i];
    }
    store8((TO*)q.C + at, q.N - n, v);
}

// A wave's 32 x (32 NJ) values in registers, register r of a lane at row
// 8 (r / 4) + 4 (lane / 32) + r % 4 and column lane % 32 of a block, go through LDS
// (32 rows of 32 NJ + 4 floats) so that each lane holds eight columns of a row and
// rows are read and written in whole lines.  m0, n0: the first row and column.
template <typename T, typename TO, int MODE, int NJ>
__device__ __forceinline__ void lin_rows(const f32x16 (&acc)[NJ], float* sh, const LinProduct<T>& q, int split, int64_t m0,
                                         int n0, const float (&bias)[8])
{
    constexpr int PITCH = 32 * NJ + 4, LPR = 4 * NJ, ROWS = 64 / LPR, STEPS = 32 / ROWS;
    const int lane = (int)threadIdx.x & 63, row = lane / LPR, n = n0 + lane % LPR * 8;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) sh[(8 * (r / 4) + 4 * (lane / 32) + r % 4) * PITCH + j * 32 + lane % 32] = acc[j][r];
    lin_wave_sync();
    if (n < q.N) {
        if (q.splits > 1) {
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int64_t m = m0 + i * ROWS + row;
                float v[8];
                __builtin_memcpy(v, sh + (i * ROWS + row) * PITCH + lane % LPR * 8, 32);
                if (m < q.M) store8(q.part + (split * q.M + m) * q.N + n, q.N - n, v);
            }
        } else {
            float res[STEPS][8] = {};
            if (MODE == LIN_FWD && q.R)
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int64_t m = m0 + i * ROWS + row;
                    if (m < q.M) load8(q.R + m * q.N + n, q.N - n, res[i]);
                }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int64_t m = m0 + i * ROWS + row;
                float v[8];
                __builtin_memcpy(v, sh + (i * ROWS + row) * PITCH + lane % LPR * 8, 32);
                if (m < q.M) lin_result<T, TO, MODE>(q, m, n, v, bias, res[i]);
            }
        }
    }
    lin_wave_sync();
}


// Tiles and splits of a product.
struct LinPlan {
    bool aligned;           // every row of every operand starts at a multiple of 16 bytes
    int tile;
    int64_t tiles_m;
    int tiles_n, kb, kb_split, splits;
    size_t part_bytes, db_bytes;
};

// The product of aligned operands (k_linear_mm.hip).
template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t launch_lin_mm(const LinPlan& p, const LinProduct<T>& q, hipStream_t s);

}  // namespace cf
