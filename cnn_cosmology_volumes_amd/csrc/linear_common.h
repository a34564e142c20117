// Shared by the linear layers' products (k_linear.hip, k_linear_mm.hip).
#pragma once

#include "cf_internal.h"

#include <math.h>

namespace cf {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct LinAct {
    int act;
    float slope;
};
// 1 / (1 + exp(-z)), and 1 minus that.  For fp32 results from the exponential of -|z|,
// which neither overflows nor loses digits to its argument's rounding (that of
// __expf is off by u |z|, 60 u at z = -80), so that both are within some 6 u = 6 2^-24.
// For bf16 results, of 8 bits (D: 16), __expf's digits are enough.
template <typename T> __device__ __forceinline__ void lin_sigmoid(float z, float& s, float& rest)
{
    if constexpr (sizeof(T) == 4) {
        const float e = expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.f + e);
        s = z < 0.f ? e * r : r;
        rest = z < 0.f ? r : e * r;
    } else {
        s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
        rest = 1.f - s;
    }
}
template <typename T> __device__ __forceinline__ float lin_act(const LinAct& a, float z)
{
    if (a.act == CF_ACT_SILU) {
        float s, rest;
        lin_sigmoid<T>(z, s, rest);
        return z * s;
    }
    return z > 0.f ? z : a.slope * z;
}
template <typename T> __device__ __forceinline__ float lin_dact(const LinAct& a, float z)
{
    if (a.act == CF_ACT_SILU) {
        float s, rest;
        lin_sigmoid<T>(z, s, rest);
        return s * fmaf(z, rest, 1.f);
    }
    return z > 0.f ? 1.f : a.slope;
}

// What becomes of the product.
enum LinMode {
    LIN_FWD,        // bias, pre, activation
    LIN_FWD_RES,    // and residual
    LIN_PLAIN       // rounded to TO
};

template <typename T> struct LinProduct {
    const T* A;
    const T* B;
    const T* A2;            // a second pass over K, of A2 and B2, where passes is 2
    const T* B2;
    int passes;
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

constexpr int LIN_PIECE = 64;       // bytes of a piece of the reduction

template <typename T> struct LinTile {
    static constexpr int V = 16 / (int)sizeof(T);      // values of 16 bytes
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

// The 16 bytes from p on, of which n values are inside; zeros for the others.  room:
// rows are 16 bytes or longer, so that a row's last values can be read as the 16 bytes
// that end with it, and moved to their places.
template <typename T> __device__ __forceinline__ uint4 lin_chunk(const T* p, int64_t n, bool room)
{
    constexpr int V = LinTile<T>::V;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n <= 0) return v;
    if (room) {
        const int over = n < V ? V - (int)n : 0, bytes = over * (int)sizeof(T);
        __builtin_memcpy(&v, p - over, 16);
        if (over) {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (bytes & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = 0;
            if (bytes & 8) w[0] = w[2], w[1] = w[3], w[2] = w[3] = 0;
            if (sizeof(T) == 2 && (bytes & 2)) {
                w[0] = w[0] >> 16 | w[1] << 16;
                w[1] = w[1] >> 16 | w[2] << 16;
                w[2] = w[2] >> 16 | w[3] << 16;
                w[3] = w[3] >> 16;
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        T t[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) t[i] = p[i];
        __builtin_memcpy(&v, t, 16);
        asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));      // (one register for two values from here on)
    }
    return v;
}

// Eight neighbouring values of the result, in words of 16 bytes: with an array of
// values that are stored whole or one by one, the compiler stores them in three pieces.
template <typename T> struct Lin8 {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(w, p, sizeof(w)); }
    // The first n < 8 only, zeros for the others.
    __device__ __forceinline__ void load(const T* p, int n)
    {
        if constexpr (sizeof(T) == 4) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
            set(v);
        } else {
            uint2 four = make_uint2(0, 0);
            uint32_t two = 0;
            uint16_t one = 0;
            if (n & 4) __builtin_memcpy(&four, p, 8);
            if (n & 2) __builtin_memcpy(&two, p + (n & 4), 4);
            if (n & 1) one = p[n & 6];
            const uint32_t x = n & 2 ? two : one, y = n & 2 ? one : 0;
            w[0] = n & 4 ? make_uint4(four.x, four.y, x, y) : make_uint4(x, y, 0, 0);
        }
    }
    __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, w, sizeof(w)); }
    __device__ __forceinline__ void store(T* p, int n) const
    {
        if constexpr (sizeof(T) == 4) {
            float v[8];
            get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        } else {
            const uint2 four = make_uint2(w[0].x, w[0].y);
            const uint32_t x = n & 4 ? w[0].z : w[0].x, y = n & 4 ? w[0].w : w[0].y;
            if (n & 4) __builtin_memcpy(p, &four, 8);
            if (n & 2) __builtin_memcpy(p + (n & 4), &x, 4);
            if (n & 1) p[n & 6] = (uint16_t)(n & 2 ? y : x);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (sizeof(T) == 4) v[4 * i + j] = __uint_as_float(u[j]);
                else v[2 * j] = __uint_as_float(u[j] << 16), v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            if (sizeof(T) == 4)
                w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                  __float_as_uint(v[4 * i + 3]));
            else
                w[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                  pack_bf16x2(v[6], v[7]));
        }
    }
};
// WHOLE: all eight; else n of them.
template <bool WHOLE, typename T> __device__ __forceinline__ void load8(const T* p, int n, float (&v)[8])
{
    Lin8<T> t;
    if (WHOLE || n >= 8) t.load(p);
    else t.load(p, n);
    t.get(v);
}
template <bool WHOLE, typename T> __device__ __forceinline__ void store8(T* p, int n, const float (&v)[8])
{
    Lin8<T> t;
    t.set(v);
    if (WHOLE || n >= 8) t.store(p);
    else t.store(p, n);
}
// at: where they are in the result, n: their column; bias: their own (LIN_FWD), res:
// their residual (LIN_FWD_RES).
template <bool WHOLE, typename T, typename TO, int MODE>
__device__ __forceinline__ void lin_result(const LinProduct<T>& q, int64_t at, int n, float (&v)[8], const float (&bias)[8],
                                           const Lin8<T>& res)
{
    if (MODE != LIN_PLAIN) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (q.pre) store8<WHOLE>(q.pre + at, q.N - n, v);
        if (q.act.act == CF_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = lin_act<T>(LinAct{CF_ACT_SILU, 0.f}, v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = lin_act<T>(LinAct{CF_ACT_LRELU, q.act.slope}, v[i]);
        }
    }
    if (MODE == LIN_FWD_RES) {
        float r[8];
        res.get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8<WHOLE>((TO*)q.C + at, q.N - n, v);
}

// Tiles and splits of a product.
struct LinPlan {
    int tm, tn;                         // edges of a tile
    int64_t tiles_m;
    int tiles_n;
    int kb, kb_split, splits;           // pieces of the reduction and of a split of it
    size_t part_bytes, db_bytes;        // sums of the splits, and of db's
};

// Rows that the kernels of k_linear_few.hip take.
constexpr int LIN_FEW = 16;
template <typename T> hipError_t launch_lin_few_fwd(const LinProduct<T>& q, hipStream_t s);
template <typename T>
hipError_t launch_lin_few_bwd(int rows, int in, int out, const T* X, const T* W, const T* pre, const T* dY, LinAct act,
                              bool gated, T* dX, float* dW, float* db, hipStream_t s);

// The product (k_linear_mm.hip): rows of its operands start at multiples of 16 bytes,
// with zeros up to the next one.
template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t launch_lin_mm(const LinPlan& p, const LinProduct<T>& q, hipStream_t s);

}  // namespace cf
