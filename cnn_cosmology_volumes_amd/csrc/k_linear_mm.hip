// The linear layers' products C = A B for operands whose rows all start at
// multiples of 16 bytes.
//
// A piece of the reduction is 128 bytes of it (64 bf16, 32 fp32 values).  Pieces of
// both operands go from memory straight to LDS, two stages in turn, as they lie:
// an operand along the reduction as lines of 128 bytes, one across it as rows of
// the tile's width; the matrix instructions' fragments of the latter come from
// transposing LDS reads.  16-byte chunks are swapped within lines so that the
// lanes of a read fall on all banks.  What lies past an operand's end (rows, or
// the reduction's rest) is read as zeros by way of an offset that the buffer
// descriptor refuses.
#include "linear_common.h"

namespace cf {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t MM_OUTSIDE = 0x80000000u;      // an offset past every descriptor's range

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_rsrc(const void* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)MM_OUTSIDE, 0x00020000);
}

template <int TILE> struct MmShape;
template <> struct MmShape<64> {
    static constexpr int WAVES = 4, WC = 2, MI = 1, NJ = 1, BLOCKS = 4;
};
template <> struct MmShape<128> {
    static constexpr int WAVES = 4, WC = 2, MI = 2, NJ = 2, BLOCKS = 2;
};
template <> struct MmShape<256> {
    static constexpr int WAVES = 8, WC = 4, MI = 4, NJ = 2, BLOCKS = 2;
};

// A piece of an operand: R rows of the tile.
template <typename T, bool ALONG, int R, int WAVES> struct MmOperand {
    static constexpr int V = 16 / (int)sizeof(T), BK = 128 / (int)sizeof(T);
    static constexpr int CHUNKS = R * 8, LOADS = R / 8 / WAVES;      // of a stage; instructions of a wave
    static constexpr int CH = R / V;                                 // chunks of a row across the reduction
    static_assert(R / 8 % WAVES == 0, "whole instructions");

    // The chunk of memory that LDS chunk `slot` holds, and its row (along) or k (across).
    __device__ static __forceinline__ int swz(int k) { return sizeof(T) == 2 ? 4 * (k & 3) : 8 * (k >> 2 & 1); }
    __device__ static __forceinline__ void place(int slot, int& line, int& chunk)
    {
        if (ALONG) {
            line = slot / 8;
            chunk = slot % 8 ^ (line >> 1 & 7);
        } else {
            line = slot / CH;
            chunk = (slot % CH ^ swz(line)) % CH;
        }
    }
    __device__ static __forceinline__ int slot(int i)
    {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        return (wave * LOADS + i) * 64 + ((int)threadIdx.x & 63);
    }
    // Byte offsets of a wave's loads from the tile's first value of a piece.
    __device__ static __forceinline__ void offsets(uint32_t (&off)[LOADS], int64_t ld, int64_t rows)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int line, chunk;
            place(slot(i), line, chunk);
            const bool inside = (ALONG ? line : chunk * V) < rows;
            off[i] = inside ? (uint32_t)(line * ld * (int64_t)sizeof(T)) + chunk * 16 : MM_OUTSIDE;
        }
    }
    // Starts the loads of a piece; left: what is left of the reduction from it on.
    __device__ static __forceinline__ void load(uint4* stage, const T* src, const uint32_t (&off)[LOADS], int64_t left)
    {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const __amdgpu_buffer_rsrc_t rsrc = mm_rsrc(src);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            uint32_t o = off[i];
            if (left < BK) {
                int line, chunk;
                place(slot(i), line, chunk);
                if ((ALONG ? chunk * V : line) >= left) o = MM_OUTSIDE;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)(stage + (wave * LOADS + i) * 64), 16, o, 0, 0, 0);
        }
    }
    // The fragment of rows r.. for step ks of the piece (see LinOperand::frag).
    __device__ static __forceinline__ bf16x8 frag(const uint4* stage, int r, int ks, uint16_t)
    {
        const int lane = (int)threadIdx.x & 63;
        if (ALONG) {
            const int chunk = (ks * 2 + lane / 32) ^ (lane >> 1 & 7);
            return *reinterpret_cast<const bf16x8*>(stage + (r + lane % 32) * 8 + chunk);
        }
        // Sixteen lanes read four values of four rows of k each; lane i gets
        // column i of these 4 x 16 values.
        const int i = lane & 15, k = ks * 16 + lane / 32 * 8 + (i >> 2);
        const int chunk = (((r + (lane & 16)) / 8 + (i >> 1 & 1)) ^ swz(i >> 2)) % CH;
        const uint16_t* at = reinterpret_cast<const uint16_t*>(stage) + (k * CH + chunk) * 8 + 4 * (i & 1);
        typedef __attribute__((address_space(3))) s16x4* lds4;
        union {
            s16x4 h[2];
            bf16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)at);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + 4 * CH * 8));
        return u.v;
    }
    __device__ static __forceinline__ f32x4 frag(const uint4* stage, int r, int ks, float)
    {
        const int lane = (int)threadIdx.x & 63;
        if (ALONG) {
            const int chunk = (ks * 2 + lane / 32) ^ (lane >> 1 & 7);
            return *reinterpret_cast<const f32x4*>(stage + (r + lane % 32) * 8 + chunk);
        }
        const int k = ks * 8 + lane / 32 * 4, n = r + lane % 32;
        const float* at = reinterpret_cast<const float*>(stage) + (k * CH + (n / 4 ^ swz(k)) % CH) * 4 + n % 4;
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = at[j * CH * 4];
        return v;
    }
};

// Barrier after which every wave's loads into LDS have landed but for the newest N,
// and its LDS reads are done.
template <int N> __device__ __forceinline__ void mm_landed()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);      // vmcnt: bits 0-3 and 14-15; lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <typename T, typename TO, bool AA, bool BA, int TILE, int MODE, bool DB>
__global__ __launch_bounds__(64 * MmShape<TILE>::WAVES, MmShape<TILE>::BLOCKS) void lin_mm_kernel(LinProduct<T> q)
{
    using S = MmShape<TILE>;
    using OA = MmOperand<T, AA, TILE, S::WAVES>;
    using OB = MmOperand<T, BA, TILE, S::WAVES>;
    using Frag = decltype(OA::frag(nullptr, 0, 0, T()));
    constexpr int STEPS = 4, MI = S::MI, NJ = S::NJ, LOADS = OA::LOADS + OB::LOADS;
    constexpr int OUT = S::WAVES / 2 * 32 * (32 * NJ + 4) / 4;      // chunks that half of the waves' results take
    constexpr int STAGE = OA::CHUNKS + OB::CHUNKS;
    // (arrays of their own: loads into one do not hold up reads of another)
    __shared__ uint4 s0[STAGE > OUT ? STAGE : OUT];
    __shared__ uint4 s1[STAGE > OUT ? STAGE : OUT];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wi = wave / S::WC * MI * 32, wj = wave % S::WC * NJ * 32;
    const int64_t units = q.tiles_m * q.tiles_n * q.splits;
    for (int64_t u = xcd_remap(blockIdx.x, gridDim.x); u < units; u += gridDim.x) {
        const int split = (int)(u % q.splits);
        const int64_t t = u / q.splits;
        // bands of four tile rows, column by column: a chip's worth of neighbouring
        // tiles is a rectangle that shares its operands' rows
        const int64_t band = t / (4 * q.tiles_n);
        const int r = (int)(t - band * 4 * q.tiles_n), h = (int)min((int64_t)4, q.tiles_m - 4 * band);
        const int64_t ti = 4 * band + r % h, i0 = ti * TILE;
        const int tj = r / h, j0 = tj * TILE;
        const int b0 = split * q.kb_split, b1 = min(b0 + q.kb_split, q.B2 ? 2 * q.kb : q.kb);
        uint32_t offa[OA::LOADS], offb[OB::LOADS];
        OA::offsets(offa, q.lda, q.M - i0);
        OB::offsets(offb, q.ldb, q.N - j0);
        auto load = [&](uint4* stage, int b) {
            const bool second = b >= q.kb;
            const int64_t k0 = (int64_t)(second ? b - q.kb : b) * OA::BK, left = q.K - k0;
            OA::load(stage, q.A + (AA ? i0 * q.lda + k0 : k0 * q.lda + i0), offa, left);
            OB::load(stage + OA::CHUNKS, (second ? q.B2 : q.B) + (BA ? j0 * q.ldb + k0 : k0 * q.ldb + j0), offb, left);
        };
        f32x16 acc[MI][NJ] = {};
        f32x16 col[NJ] = {};
        const bool sums = DB && ti == 0 && wi == 0;
        Frag fa[2][MI], fb[2][NJ];
        auto read = [&](int f, const uint4* stage, int ks) {
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[f][i] = OA::frag(stage, wi + i * 32, ks, T());
#pragma unroll
            for (int j = 0; j < NJ; ++j) fb[f][j] = OB::frag(stage + OA::CHUNKS, wj + j * 32, ks, T());
        };
        auto multiply = [&](int f) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) lin_mma(fa[f][i], fb[f][j], acc[i][j]);
            if (DB && sums)
#pragma unroll
                for (int j = 0; j < NJ; ++j) lin_mma(ones(fb[f][j]), fb[f][j], col[j]);
        };
        load(s0, b0);
        if (b0 + 1 < b1) {
            load(s1, b0 + 1);
            mm_landed<LOADS>();
        } else {
            mm_landed<0>();
        }
        read(0, s0, 0);
        // The reads of a step are in flight while the step before it is multiplied, across the barrier too.
        auto piece = [&](uint4* cur, uint4* nxt, int b) {
            read(1, cur, 1);
            multiply(0);
            read(0, cur, 2);
            multiply(1);
            read(1, cur, 3);
            multiply(0);
            if (b + 1 < b1) {
                mm_landed<0>();
                if (b + 2 < b1) load(cur, b + 2);
                read(0, nxt, 0);
            }
            multiply(1);
        };
        int b = b0;
        for (; b + 1 < b1; b += 2) {
            piece(s0, s1, b);
            piece(s1, s0, b + 1);
        }
        if (b < b1) piece(s0, s1, b);
        __syncthreads();
        if (DB && sums && lane < 32 && q.db)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = j0 + wj + j * 32 + lane;
                if (n >= q.N) continue;
                if (q.splits > 1) q.db_part[(int64_t)split * q.N + n] = col[j][0];
                else q.db[n] = col[j][0];
            }
        const int n = j0 + wj + lane % (4 * NJ) * 8;
        float bias[8] = {};
        if (MODE == LIN_FWD && q.bias && n < q.N) load8(q.bias + n, q.N - n, bias);
        float* sh = (float*)(wave < S::WAVES / 2 ? s0 : s1) + wave % (S::WAVES / 2) * 32 * (32 * NJ + 4);
#pragma unroll
        for (int i = 0; i < MI; ++i) lin_rows<T, TO, MODE, NJ>(acc[i], sh, q, split, i0 + wi + i * 32, j0 + wj, bias);
        __syncthreads();
    }
}

}  // namespace

template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t launch_lin_mm(const LinPlan& p, const LinProduct<T>& q, hipStream_t s)
{
    const int64_t units = p.tiles_m * p.tiles_n * p.splits, most = 1 << 20;
    const unsigned grid = (unsigned)(units < most ? units : most);
    if (p.tile == 256) lin_mm_kernel<T, TO, AA, BA, 256, MODE, DB><<<grid, 64 * MmShape<256>::WAVES, 0, s>>>(q);
    else if (p.tile == 128) lin_mm_kernel<T, TO, AA, BA, 128, MODE, DB><<<grid, 64 * MmShape<128>::WAVES, 0, s>>>(q);
    else lin_mm_kernel<T, TO, AA, BA, 64, MODE, DB><<<grid, 64 * MmShape<64>::WAVES, 0, s>>>(q);
    return hipGetLastError();
}

#define CF_LIN_MM(T)                                                                                                      \
    template hipError_t launch_lin_mm<T, T, true, false, LIN_FWD, false>(const LinPlan&, const LinProduct<T>&, hipStream_t);   \
    template hipError_t launch_lin_mm<T, T, true, true, LIN_PLAIN, false>(const LinPlan&, const LinProduct<T>&, hipStream_t);  \
    template hipError_t launch_lin_mm<T, float, false, false, LIN_PLAIN, false>(const LinPlan&, const LinProduct<T>&,          \
                                                                                hipStream_t);                                  \
    template hipError_t launch_lin_mm<T, float, false, false, LIN_PLAIN, true>(const LinPlan&, const LinProduct<T>&, hipStream_t);
CF_LIN_MM(float)
CF_LIN_MM(uint16_t)

}  // namespace cf
