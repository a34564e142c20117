// The global norm of a list of gradients, and the gradients scaled to a largest
// norm:
//   norm = sqrt(sum over every tensor of g^2),
//   factor = max_norm / norm where norm > max_norm, else 1,  out = factor g.
//
// Two launches over chunks of 16 KB.  The first adds the squares in fp64 (the
// square of any fp32 value is finite and normal there, so neither large nor
// small gradients need a scale of their own) and leaves one sum a block.  In the
// second every block adds these sums in the same order, so that all get the same
// factor without a launch between, and scales its chunks, by products in fp64: a
// factor in fp32 would be one more rounding, and below 2^-126 it has few digits (values
// of 1e30 and a limit of 1e-12: 1e-42).  No atomics: results
// are reproducible bit for bit.  The second launch takes the chunks from the
// last to the first: what the first read last may still lie in the last-level
// cache.
//
// What bounds it: memory.  75.4 M fp32 values in 192 tensors take 181 us, which is
// their 302 MB read twice and written once at 5 TB/s; 5.0 M values in 11 tensors
// take 15.5 us in the two kernels and 17.6 with the call, which is then the host's.
#include "cf_internal.h"

#include <math.h>

namespace cf {
namespace {

constexpr int CLIP_T = 256;                 // threads a block
constexpr int CLIP_V = 4;                   // 16-byte vectors a thread and chunk
constexpr int CLIP_BYTES = CLIP_T * CLIP_V * 16;
constexpr int CLIP_LIST = 128;              // tensors a launch (its arguments stay below 4 KB)
constexpr int CLIP_BLOCKS = 2048;           // most blocks a launch, 8 a CU

template <typename T> struct ClipList {
    int count;
    int chunks;
    const T* g[CLIP_LIST];
    T* out[CLIP_LIST];
    int64_t n[CLIP_LIST];
    int start[CLIP_LIST + 1];               // first chunk of each tensor
};

// The tensor that holds chunk c.
template <typename T> __device__ __forceinline__ int clip_tensor(const ClipList<T>& l, int c)
{
    int lo = 0, hi = l.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (c >= l.start[mid]) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Sum over the block, in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* sh)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((sh[0] + sh[1]) + sh[2]) + sh[3];
}

// A thread's values of a chunk whose tensor has n left.
template <typename T> struct ClipVecs {
    static constexpr int V = 16 / (int)sizeof(T);
    T v[CLIP_V][V];
    __device__ __forceinline__ static int place(int k) { return (k * CLIP_T + (int)threadIdx.x) * V; }
    __device__ __forceinline__ void load(const T* g, int64_t n)
    {
        if (n >= CLIP_T * CLIP_V * V) {
#pragma unroll
            for (int k = 0; k < CLIP_V; ++k) __builtin_memcpy(v[k], g + place(k), 16);
            return;
        }
#pragma unroll
        for (int k = 0; k < CLIP_V; ++k) {
            const int i = place(k);
            if (i + V <= n) __builtin_memcpy(v[k], g + i, 16);
            else
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = i + e < n ? g[i + e] : (T)0;
        }
    }
};

template <typename T>
__global__ __launch_bounds__(CLIP_T) void clip_norm_kernel(ClipList<T> l, double* __restrict__ part)
{
    constexpr int V = 16 / (int)sizeof(T);
    __shared__ double sh[4];
    double sum[CLIP_V] = {};
    ClipVecs<T> x;
    auto fetch = [&](int c) {
        const int t = clip_tensor(l, c);
        const int64_t at = (int64_t)(c - l.start[t]) * (CLIP_T * CLIP_V * V);
        x.load(l.g[t] + at, l.n[t] - at);
    };
    fetch((int)blockIdx.x);
    for (int c = (int)blockIdx.x; c < l.chunks; c += (int)gridDim.x) {
        const ClipVecs<T> y = x;
        if (c + (int)gridDim.x < l.chunks) fetch(c + (int)gridDim.x);      // under way while these are added
#pragma unroll
        for (int k = 0; k < CLIP_V; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const double g = (double)widen(y.v[k][e]);
                sum[k] = fma(g, g, sum[k]);
            }
    }
    const double total = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), sh);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
}

// (fp32: the fp64 products' registers held to what leaves 8 waves a SIMD: 188 us for 191 with three more.  bf16's 94 leave 5.)
template <typename T>
__global__ __launch_bounds__(CLIP_T, (sizeof(T) == 4 ? 8 : 5)) void clip_scale_kernel(ClipList<T> l, const double* __restrict__ part, int parts,
                                                            float max_norm, float* __restrict__ stats)
{
    constexpr int V = 16 / (int)sizeof(T);
    __shared__ double sh[4];
    // the first chunk's values are under way while the sums are added
    ClipVecs<T> x;
    const T* g = nullptr;
    T* out = nullptr;
    int64_t n = 0;
    auto fetch = [&](int b) {
        const int c = l.chunks - 1 - b, t = clip_tensor(l, c);
        const int64_t at = (int64_t)(c - l.start[t]) * (CLIP_T * CLIP_V * V);
        g = l.g[t] + at;
        out = l.out[t] + at;
        n = l.n[t] - at;
        x.load(g, n);
    };
    fetch((int)blockIdx.x);
    double sum = 0.0;
#pragma unroll 4
    for (int i = (int)threadIdx.x; i < parts; i += CLIP_T) sum += part[i];
    const double norm = sqrt(block_sum(sum, sh));
    // (a norm that is not a number gives a factor that is none either)
    const double factor = norm <= (double)max_norm ? 1.0 : max_norm < INFINITY ? (double)max_norm / norm : 1.0;
    if (stats && blockIdx.x == 0 && threadIdx.x == 0) {
        stats[0] = (float)norm;
        stats[1] = (float)factor;
    }
    for (int b = (int)blockIdx.x;;) {
        if (factor != 1.0 || g != out)
#pragma unroll
            for (int k = 0; k < CLIP_V; ++k) {
                const int i = x.place(k);
#pragma unroll
                for (int e = 0; e < V; ++e) Elem<T>::store(x.v[k], e, (float)((double)widen(x.v[k][e]) * factor));
                if (i + V <= n) __builtin_memcpy(out + i, x.v[k], 16);
                else
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (i + e < n) out[i + e] = x.v[k][e];
            }
        b += (int)gridDim.x;
        if (b >= l.chunks) break;
        fetch(b);
    }
}

int64_t clip_chunks(int64_t n, int size) { return (n * size + CLIP_BYTES - 1) / CLIP_BYTES; }

int clip_grid(int64_t chunks) { return (int)(chunks < CLIP_BLOCKS ? chunks : CLIP_BLOCKS); }

}  // namespace

size_t clip_ws_bytes(cf_dtype dt, int count, const int64_t* n)
{
    const int size = dt == CF_F32 ? 4 : 2;
    size_t parts = 0;
    for (int i = 0; i < count; i += CLIP_LIST) {
        int64_t chunks = 0;
        for (int k = i; k < count && k < i + CLIP_LIST; ++k) chunks += clip_chunks(n[k], size);
        parts += (size_t)clip_grid(chunks);
    }
    return parts * sizeof(double);
}

template <typename T>
hipError_t launch_grad_clip(int count, const int64_t* n, const void* const* g, void* const* out, float max_norm,
                            float* stats, void* ws, hipStream_t s)
{
    double* part = (double*)ws;
    int parts = 0;
    const int last = (count - 1) / CLIP_LIST * CLIP_LIST;
    for (int pass = 0; pass < 2; ++pass)
        for (int at = 0; at < count; at += CLIP_LIST) {
            const int i = pass == 0 ? at : last - at;
            ClipList<T> l;
            l.count = count - i < CLIP_LIST ? count - i : CLIP_LIST;
            l.chunks = 0;
            for (int k = 0; k < l.count; ++k) {
                l.g[k] = (const T*)g[i + k];
                l.out[k] = (T*)out[i + k];
                l.n[k] = n[i + k];
                l.start[k] = l.chunks;
                l.chunks += (int)clip_chunks(n[i + k], (int)sizeof(T));
            }
            l.start[l.count] = l.chunks;
            const int grid = clip_grid(l.chunks);
            if (pass == 0) {
                clip_norm_kernel<T><<<grid, CLIP_T, 0, s>>>(l, part + parts);
                parts += grid;
            } else {
                clip_scale_kernel<T><<<grid, CLIP_T, 0, s>>>(l, part, parts, max_norm, i == 0 ? stats : nullptr);
            }
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

template hipError_t launch_grad_clip<float>(int, const int64_t*, const void* const*, void* const*, float, float*, void*,
                                            hipStream_t);
template hipError_t launch_grad_clip<uint16_t>(int, const int64_t*, const void* const*, void* const*, float, float*,
                                               void*, hipStream_t);

}  // namespace cf
