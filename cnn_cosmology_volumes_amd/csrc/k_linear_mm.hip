// The linear layers' products C = A B.  Rows of the operands start at multiples of 16
// bytes, and hold zeros from their end to the next multiple.
//
// A piece of the reduction is 64 bytes of it (32 bf16, 16 fp32 values).  Pieces of
// both operands go from memory straight to LDS, three or four stages in turn, as they lie:
// an operand along the reduction as lines of 64 bytes, one across it as rows of
// the tile's width; the matrix instructions' fragments of the latter come from
// transposing LDS reads.  16-byte chunks are swapped within lines so that the
// lanes of a read fall on all banks.  What lies past an operand's end (rows, or
// the reduction's rest) is read as zeros by way of an offset that the buffer
// descriptor refuses.
//
// What bounds it: 32768 x 2048 x 2048 bf16 takes 262 us, about 200 of them in the
// pieces (a library product without the epilogue 217), the rest in the four rounds'
// results, which all CUs read (residuals) and write at about the same time.  262144
// x 128 x 512 bf16 with pre takes 139: its 604 MB at 4.3 TB/s.  4096 x 2048 x 2048
// fp32 takes 256: 134 TFLOP/s, the fp32 matrix cores' rate at this clock.
// What else was tried: results written from the registers' own layout, 32 bytes of a
// row at a time, take 2.2 times as long at 262144 x 128 x 512 (lines are written in
// parts); a wait for a residual or a bias between stores is a wait for the stores
// (185 us for 135 there); a stage of 128 bytes and two of them, 318 us for 295 at
// 32768 x 2048 x 2048; tiles of 256 x 128, two blocks a CU, overlap one's results with
// the other's pieces but load half as much again (307 for 264).
#include "linear_common.h"

#include <type_traits>

namespace cf {
namespace {

constexpr int MM_PIECE = LIN_PIECE;
constexpr uint32_t MM_OUTSIDE = 0x80000000u;      // an offset past every descriptor's range

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mm_rsrc(const void* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)MM_OUTSIDE, 0x00020000);
}

// A tile of TM x TN: WAVES waves, WC of them side by side, of 32 MI x 32 NJ; stages of
// pieces; waves a SIMD that registers are kept for.  A CU's 160 KB of LDS hold the
// stages of 5, 2, 2 and 1 blocks (32, 64, 72 and 128 KB each), which are the slots that
// lin_plan counts; 64 x 64 with residuals or db's sums takes 97 registers and runs 4.
template <int TM, int TN> struct MmShape;
template <> struct MmShape<64, 64> {
    static constexpr int WAVES = 4, WC = 2, MI = 1, NJ = 1, STAGES = 4, SIMD_WAVES = 4;
};
template <> struct MmShape<128, 128> {
    static constexpr int WAVES = 4, WC = 2, MI = 2, NJ = 2, STAGES = 4, SIMD_WAVES = 2;
};
template <> struct MmShape<256, 128> {
    static constexpr int WAVES = 4, WC = 2, MI = 4, NJ = 2, STAGES = 3, SIMD_WAVES = 2;
};
template <> struct MmShape<256, 256> {
    static constexpr int WAVES = 8, WC = 4, MI = 4, NJ = 2, STAGES = 4, SIMD_WAVES = 2;
};

// A piece of an operand: R rows of the tile.
template <typename T, bool ALONG, int R, int WAVES> struct MmOperand {
    static constexpr int V = 16 / (int)sizeof(T), BK = MM_PIECE / (int)sizeof(T);
    static constexpr int CHUNKS = R * 4, LOADS = R / 16 / WAVES;     // of a stage; instructions of a wave
    static constexpr int CH = R / V;                                 // chunks of a row across the reduction
    static constexpr int READS = ALONG ? 1 : sizeof(T) == 2 ? 2 : 4;  // LDS reads of a fragment
    static_assert(R / 16 % WAVES == 0, "whole instructions");

    // The chunk of memory that LDS chunk `slot` holds, and its row (along) or k (across).
    __device__ static __forceinline__ int swz(int k) { return sizeof(T) == 2 ? 4 * (k & 3) : 8 * (k >> 2 & 1); }
    __device__ static __forceinline__ void place(int slot, int& line, int& chunk)
    {
        if (ALONG) {
            line = slot / 4;
            chunk = slot % 4 ^ (line >> 2 & 3);
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
    // Byte offsets of a wave's loads from the tile's first value of a piece, and the place in
    // the piece's reduction that each starts at.
    __device__ static __forceinline__ void offsets(uint32_t (&off)[LOADS], int (&k)[LOADS], int64_t ld, int64_t rows)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int line, chunk;
            place(slot(i), line, chunk);
            const bool inside = (ALONG ? line : chunk * V) < rows;
            off[i] = inside ? (uint32_t)(line * ld * (int64_t)sizeof(T)) + chunk * 16 : MM_OUTSIDE;
            k[i] = ALONG ? chunk * V : line;
        }
    }
    // Starts the loads of a piece; left: what is left of the reduction from it on (none:
    // the loads touch no memory).
    __device__ static __forceinline__ void load(uint4* stage, const T* src, const uint32_t (&off)[LOADS],
                                                const int (&k)[LOADS], int left)
    {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const __amdgpu_buffer_rsrc_t rsrc = mm_rsrc(src);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)(stage + (wave * LOADS + i) * 64), 16,
                k[i] < left ? off[i] : MM_OUTSIDE, 0, 0, 0);
    }
    // The fragment of rows r.. for step ks of the piece of a product: bf16 row
    // r + lane % 32, k = 16 ks + 8 (lane / 32) + 0..7 of a 32 x 32 x 16 one; fp32 the same
    // row, k = 8 ks + 4 (lane / 32) + 0..3, one for each of four 32 x 32 x 2.
    __device__ static __forceinline__ bf16x8 frag(const uint4* stage, int r, int ks, uint16_t)
    {
        const int lane = (int)threadIdx.x & 63;
        if (ALONG) {
            const int chunk = (ks * 2 + lane / 32) ^ (lane >> 2 & 3);
            return *reinterpret_cast<const bf16x8*>(stage + (r + lane % 32) * 4 + chunk);
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
            const int chunk = (ks * 2 + lane / 32) ^ (lane >> 2 & 3);
            return *reinterpret_cast<const f32x4*>(stage + (r + lane % 32) * 4 + chunk);
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
    __builtin_amdgcn_sched_barrier(0);      // (matrix instructions before it stay before it)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);      // vmcnt: bits 0-3 and 14-15; lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The LDS reads of the next step, and the loads of a piece, among the matrix
// instructions of this one.
template <int MFMAS, int READS, int LOADS> __device__ __forceinline__ void mm_interleave()
{
    constexpr int MOST = MFMAS > READS ? MFMAS : READS;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        if (i < MFMAS) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (i < LOADS) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
}

template <typename T, typename TO, bool AA, bool BA, int TM, int TN, int MODE, bool DB>
__global__ __launch_bounds__((64 * MmShape<TM, TN>::WAVES), (MmShape<TM, TN>::SIMD_WAVES)) void lin_mm_kernel(LinProduct<T> q)
{
    using S = MmShape<TM, TN>;
    using OA = MmOperand<T, AA, TM, S::WAVES>;
    using OB = MmOperand<T, BA, TN, S::WAVES>;
    using Frag = decltype(OA::frag(nullptr, 0, 0, T()));
    constexpr int MI = S::MI, NJ = S::NJ, LOADS = OA::LOADS + OB::LOADS;
    constexpr int MFMAS = MI * NJ * (sizeof(T) == 2 ? 1 : 4);                                     // of a step
    constexpr int READS = MI * OA::READS + NJ * OB::READS;
    constexpr int STAGE = OA::CHUNKS + OB::CHUNKS;
    static_assert(S::WAVES / S::WC == 2 && 32 * TN / 4 <= STAGE, "a strip of results for each half of the waves");
    // (arrays of their own: loads into one do not hold up reads of another)
    __shared__ uint4 s0[STAGE];
    __shared__ uint4 s1[STAGE];
    __shared__ uint4 s2[STAGE];
    __shared__ uint4 s3[S::STAGES > 3 ? STAGE : 1];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wi = wave / S::WC * MI * 32, wj = wave % S::WC * NJ * 32;
    const int64_t units = q.tiles_m * q.tiles_n * q.splits;
    for (int64_t u = xcd_remap(blockIdx.x, gridDim.x); u < units; u += gridDim.x) {
        // all tiles of a split before the next one: an XCD's blocks share their part of the reduction's operands
        const int64_t tiles = q.tiles_m * q.tiles_n, t = u % tiles;
        const int split = (int)(u / tiles);
        // bands of four tile rows, column by column: a chip's worth of neighbouring
        // tiles is a rectangle that shares its operands' rows
        const int64_t band = t / (4 * q.tiles_n);
        const int r = (int)(t - band * 4 * q.tiles_n), h = (int)min((int64_t)4, q.tiles_m - 4 * band);
        const int64_t ti = 4 * band + r % h, i0 = ti * TM;
        const int tj = r / h, j0 = tj * TN;
        const int b0 = split * q.kb_split, b1 = min(b0 + q.kb_split, q.passes * q.kb);
        uint32_t offa[OA::LOADS], offb[OB::LOADS];
        int ka[OA::LOADS], kb[OB::LOADS];
        OA::offsets(offa, ka, q.lda, q.M - i0);
        OB::offsets(offb, kb, q.ldb, q.N - j0);
        auto load = [&](uint4* stage, int b) {
            const bool second = b >= q.kb;
            const int64_t k0 = (int64_t)(second ? b - q.kb : b) * OA::BK;
            const int left = b < b1 ? (int)min(q.K - k0, (int64_t)OA::BK) : 0;
            OA::load(stage, (second ? q.A2 : q.A) + (AA ? i0 * q.lda + k0 : k0 * q.lda + i0), offa, ka, left);
            OB::load(stage + OA::CHUNKS, (second ? q.B2 : q.B) + (BA ? j0 * q.ldb + k0 : k0 * q.ldb + j0), offb, kb, left);
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
                for (int j = 0; j < NJ; ++j) lin_mma(fb[f][j], fa[f][i], acc[i][j]);
            if (DB && sums)
#pragma unroll
                for (int j = 0; j < NJ; ++j) lin_mma(ones(fb[f][j]), fb[f][j], col[j]);
        };
        // All stages but one are under way while that one is worked on; past the last one, loads that
        // touch no memory keep the count that the waits go by.  The reads of a step are in
        // flight while the step before it is multiplied, across the barrier too.
        load(s0, b0);
        load(s1, b0 + 1);
        load(s2, b0 + 2);
        if constexpr (S::STAGES > 3) load(s3, b0 + 3);
        mm_landed<(S::STAGES - 1) * LOADS>();
        read(0, s0, 0);
        auto piece = [&](uint4* cur, uint4* nxt, int b) {
            read(1, cur, 1);
            multiply(0);
            mm_interleave<MFMAS, READS, 0>();
            mm_landed<(S::STAGES - 2) * LOADS>();
            load(cur, b + S::STAGES);
            read(0, nxt, 0);      // (past the last piece: read and not used)
            multiply(1);
            mm_interleave<MFMAS, READS, LOADS>();
        };
        int b = b0;
        for (; b + S::STAGES <= b1; b += S::STAGES) {
            piece(s0, s1, b);
            piece(s1, s2, b + 1);
            if constexpr (S::STAGES > 3) {
                piece(s2, s3, b + 2);
                piece(s3, s0, b + 3);
            } else {
                piece(s2, s0, b + 2);
            }
        }
        if (b < b1) piece(s0, s1, b);
        if (b + 1 < b1) piece(s1, s2, b + 1);
        if (S::STAGES > 3 && b + 2 < b1) piece(s2, s3, b + 2);
        mm_landed<0>();
        if (DB && sums && lane < 32 && q.db)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int n = j0 + wj + j * 32 + lane;
                if (n >= q.N) continue;
                if (q.splits > 1) q.db_part[(int64_t)split * q.N + n] = col[j][0];
                else q.db[n] = col[j][0];
            }
        // Results, 32 rows of the waves side by side at a time, through LDS, so that a wave reads
        // and writes whole rows of the tile: register r of a lane is row lane % 32, column 8 (r / 4)
        // + 4 (lane / 32) + r % 4 of a block (the product is formed as its transpose).  Chunks are
        // swapped within a row of the strip: sixteen rows at one chunk fall on all banks.
        //
        // Memory operations complete in order: a wait for a residual would be one for the
        // stores before it too, so a strip's residuals are read before the stores of the strip
        // before it, and tiles that lie inside the result take a path without conditions, in
        // which the compiler can count on them.
        constexpr int LPR = TN / 8, RPI = 64 / LPR, STEPS = 32 / RPI / S::WC;      // lanes of a row, rows of an access
        float4* const strip = reinterpret_cast<float4*>(wave / S::WC ? s1 : s0);
        const int side = wave % S::WC, row = lane % 32, n = j0 + lane % LPR * 8;
        float bias[8] = {};
        if (MODE != LIN_PLAIN && q.bias && n < q.N) load8<false>(q.bias + n, q.N - n, bias);
        const int r0 = side * RPI + lane / LPR;                                    // a lane's first row of a strip
        const int64_t m0 = i0 + wi + r0, at0 = m0 * q.N + n;
        const int64_t step = (int64_t)(RPI * S::WC) * q.N;
        auto put = [&](int i) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    strip[row * (TN / 4) + (((side * NJ + j) * 8 + 2 * g + lane / 32) ^ (row & 15))] =
                        make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
        };
        auto take = [&](int k, float (&v)[8]) {
            const int r = r0 + k * RPI * S::WC;
            *reinterpret_cast<float4*>(v) = strip[r * (TN / 4) + (lane % LPR * 2 ^ (r & 15))];
            *reinterpret_cast<float4*>(v + 4) = strip[r * (TN / 4) + ((lane % LPR * 2 + 1) ^ (r & 15))];
        };
        // fp32 results without an epilogue and a split's sums are the same but for their place
        constexpr bool SUMS = MODE == LIN_PLAIN && sizeof(TO) == 4;
        float* const sums_to = q.splits > 1 ? q.part + split * q.M * q.N : (float*)q.C;
        if ((SUMS || q.splits == 1) && i0 + TM <= q.M && j0 + TN <= q.N) {
            Lin8<T> res[2][STEPS];
            int64_t ahead = at0, at = at0;
            auto fetch = [&](int i) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k, ahead += step) res[i & 1][k].load(q.R + ahead);
            };
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                put(i);
                if (MODE == LIN_FWD_RES && i == 0) fetch(0);
                if (MODE == LIN_FWD_RES && i + 1 < MI) fetch(i + 1);
                lds_barrier();
#pragma unroll
                for (int k = 0; k < STEPS; ++k, at += step) {
                    float v[8];
                    take(k, v);
                    if (SUMS) store8<true>(sums_to + at, 8, v);
                    else lin_result<true, T, TO, MODE>(q, at, n, v, bias, res[i & 1][k]);
                }
                lds_barrier();      // (not one that waits for the stores)
            }
        } else {
            int64_t at = at0, m = m0;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                put(i);
                lds_barrier();
#pragma unroll 1
                for (int k = 0; k < STEPS; ++k, at += step, m += RPI * S::WC) {
                    float v[8];
                    take(k, v);
                    if (m >= q.M || n >= q.N) continue;
                    if (SUMS || q.splits > 1) {
                        store8<false>(sums_to + at, q.N - n, v);
                        continue;
                    }
                    Lin8<T> res;
                    if (MODE == LIN_FWD_RES) {
                        if (q.N - n >= 8) res.load(q.R + at);
                        else res.load(q.R + at, q.N - n);
                    }
                    lin_result<false, T, TO, MODE>(q, at, n, v, bias, res);
                }
                lds_barrier();
            }
        }
    }
}

}  // namespace

template <typename T, typename TO, bool AA, bool BA, int MODE, bool DB>
hipError_t launch_lin_mm(const LinPlan& p, const LinProduct<T>& q, hipStream_t s)
{
    const int64_t units = p.tiles_m * p.tiles_n * p.splits, most = 1 << 20;
    const unsigned grid = (unsigned)(units < most ? units : most);
    auto go = [&](auto tm, auto tn) {
        constexpr int TM = decltype(tm)::value, TN = decltype(tn)::value;
        lin_mm_kernel<T, TO, AA, BA, TM, TN, MODE, DB><<<grid, (64 * MmShape<TM, TN>::WAVES), 0, s>>>(q);
    };
    if constexpr (!DB) {
        if constexpr (sizeof(T) == 2) {
            if (p.tn == 256) {
                go(std::integral_constant<int, 256>(), std::integral_constant<int, 256>());
                return hipGetLastError();
            }
        }
        if (p.tm == 256) {
            go(std::integral_constant<int, 256>(), std::integral_constant<int, 128>());
            return hipGetLastError();
        }
    }
    if (p.tm == 128) go(std::integral_constant<int, 128>(), std::integral_constant<int, 128>());
    else go(std::integral_constant<int, 64>(), std::integral_constant<int, 64>());
    return hipGetLastError();
}

#define CF_LIN_MM(T)                                                                                                      \
    template hipError_t launch_lin_mm<T, T, true, false, LIN_FWD, false>(const LinPlan&, const LinProduct<T>&, hipStream_t);   \
    template hipError_t launch_lin_mm<T, T, true, false, LIN_FWD_RES, false>(const LinPlan&, const LinProduct<T>&,             \
                                                                            hipStream_t);                                      \
    template hipError_t launch_lin_mm<T, T, true, true, LIN_PLAIN, false>(const LinPlan&, const LinProduct<T>&, hipStream_t);  \
    template hipError_t launch_lin_mm<T, float, false, false, LIN_PLAIN, false>(const LinPlan&, const LinProduct<T>&,          \
                                                                                hipStream_t);                                  \
    template hipError_t launch_lin_mm<T, float, false, false, LIN_PLAIN, true>(const LinPlan&, const LinProduct<T>&, hipStream_t);
CF_LIN_MM(float)
CF_LIN_MM(uint16_t)

}  // namespace cf
