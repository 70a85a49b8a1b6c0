// Device side of the product of two matrices in the 8-bit form, for CDNA4
// (gfx950):  out[m][n] = T(sum_k a[m][k] b[n][k] + add[m][n]).
//
// Scales are powers of two, one for 128 values along k, so the scaled matrix
// instructions (32x32x64 and 16x16x128, one scale byte a lane and operand)
// take them as they are: the sum over k stays in the accumulators from the
// first block to the last, with no arithmetic beside the instructions.  The
// hardware aligns the products of eight neighbouring k to the largest of them and
// cuts each, towards zero, at 2^-13 of that one's power of two (a code below the
// normal ones counts with their smallest exponent there); the eights' sums are
// added in fp32.  This is the choice for 16-bit outputs, which it gives at twice
// the rate: on normal data it moves a result by 2^-16 of its size, far less than
// the codes' own rounding did and than the output's does (8192 x 6400 x 1600
// bf16: 1.6626e-3 of the norm against float64, 1.6625e-3 with sums in fp32).  Its bound, 7 *
// 2^-13 of the products' magnitudes, is not that small where they cancel, or
// where a group's largest factors are subnormal codes (measured: up to 3.4e-3 of
// the magnitudes).  fp32 outputs, and products whose time is not the
// instructions', widen the codes to bf16 (exact, the scale with them) and take
// the bf16 instructions, at half the rate.
//
// The order in which an instruction takes its k does not matter as long as
// both operands have the same, which leaves the layouts in LDS free.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/zero_dp.h"
#include "zero_dp_block8.h"
#include "zero_dp_fp8.h"

namespace {

using zdp::kB8;
using zdp::ProductArgs;
using zdp::ProductSide;
using zdp::scale_value;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32_1 __attribute__((aligned(1)));

// ----------------------------------------------------------------- outputs
template <int kType>
struct Out;
template <>
struct Out<ZERO_TYPE_F32> {
    typedef float T;
};
template <>
struct Out<ZERO_TYPE_F16> {
    typedef _Float16 T;
};
template <>
struct Out<ZERO_TYPE_BF16> {
    typedef __bf16 T;
};

// kN neighbouring elements of a row, of which the first `left` are there; the
// row is aligned to its elements only.
template <typename T, int kN>
struct Pack {
    typedef T V __attribute__((ext_vector_type(kN), aligned(sizeof(T))));
};

template <typename T, int kN, bool kAdd>
__device__ __forceinline__ void store_whole(T* to, const float (&v)[kN], const T* add) {
    typedef typename Pack<T, kN>::V V;
    V x, y = {};
    if (kAdd) y = *reinterpret_cast<const V*>(add);
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = static_cast<T>(kAdd ? v[i] + static_cast<float>(y[i]) : v[i]);
    *reinterpret_cast<V*>(to) = x;
}

template <typename T, int kN>
__device__ __forceinline__ void store_run(T* to, const float (&v)[kN], const T* add, int64_t left) {
    if (left >= kN) {
        if (add != nullptr)
            store_whole<T, kN, true>(to, v, add);
        else
            store_whole<T, kN, false>(to, v, add);
        return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (i < left) to[i] = static_cast<T>(v[i] + (add != nullptr ? static_cast<float>(add[i]) : 0.0f));
}

// ------------------------------------------------------------------- codes
// Codes of which the first `left` count, the others zero.
template <typename V>
__device__ __forceinline__ V keep(V x, int left) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(V) / 4); ++i) {
        const int b = left - 4 * i;
        x[i] = b >= 4 ? x[i] : b <= 0 ? 0 : x[i] & static_cast<int>((1u << (8 * b)) - 1u);
    }
    return x;
}

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) { return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// Eight codes (two words) as bf16 under a scale; exact between 2^-126 and 2^127.
__device__ __forceinline__ bf16x8 widen(int lo, int hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Codes under the scale byte 255 are NaN, whatever they are.
__device__ __forceinline__ int poisoned(int word, uint32_t byte) { return byte == 255u ? 0x7F7F7F7F : word; }

__device__ __forceinline__ const uint8_t* scale_row(const ProductSide& s, int64_t row) {
    return s.scales + (row >> s.shift) * s.scales_stride;
}

// From the scales of row r0 to those of row r0 + p.
__device__ __forceinline__ uint32_t scale_offset(const ProductSide& s, int64_t r0, int p) {
    return static_cast<uint32_t>(((r0 + p) >> s.shift) - (r0 >> s.shift)) * static_cast<uint32_t>(s.scales_stride);
}

// ------------------------------------------------------------------- tiles
// A workgroup computes kBM x kBN of out with kWM x kWN waves, each of them
// kFM x kFN squares of 32.  Blocks of 128 k of both operands go to one of kS
// places in LDS through direct loads (16 bytes a lane, no registers), and from
// there to registers, half a block at a time.  Everything is ahead of the
// matrix instructions:
//
//   first half of block b:   multiply it; read b's second half
//   barrier                  (b is in registers now, b + 1 is in LDS)
//   second half of block b:  load b + kS over b; read b + 1's first half; multiply
//
// so that a block has kS - 1 blocks' time to come out of memory, a read half a
// block's, and there is one barrier for 128 k.  Small tiles take more places:
// a block's time is shorter than memory's latency there.  Scales go the same
// way, four blocks in a word of a row.
//
// In LDS a row's 128 bytes are eight pieces of 16, piece q of row p at place
// q ^ (p / 2 % 8): the rows that a read takes at one piece lie in different
// banks.  b's rows are dealt to LDS so that the kFN squares of a lane hold
// neighbouring columns of out, which it stores at once.
//
// Bound by the matrix instructions at the clock that real data allow: 8192 x
// 8192 x 8192 bf16 in 256 x 256 tiles 402 us, 2740 TFLOP/s, on operands that the
// caches hold, 438 us on three pairs in turn (busy 73 % of the cycles; eight
// waves read 192 KB of LDS a block, four of 128 x 128 would read 128 KB at the
// same rate, but have no second wave to hide an epilogue behind); fp32 out 810 us,
// 1360.  Short k pays for each round's first loads and last stores: 8192 x 6400
// x 1600 bf16 96 us, 1740 TFLOP/s, of which 88 in the large tiles and 11 in the
// launch of the last 32 in quarters; 8192 x 1600 x 6400 79 us, 2120, its last
// column of tiles three quarters empty.
template <int kBM_, int kBN_, int kWM_, int kWN_, int kS_>
struct Shape {
    static constexpr int kBM = kBM_, kBN = kBN_, kWM = kWM_, kWN = kWN_, kS = kS_;
    static constexpr int kThreads = 64 * kWM * kWN;
    static constexpr int kFM = kBM / kWM / 32, kFN = kBN / kWN / 32;
    static constexpr int kRows = kBM + kBN;
    static constexpr int kLoadsA = kBM * 8 / kThreads, kLoadsB = kBN * 8 / kThreads;
    static_assert(kThreads % 128 == 0 && kBM * 8 % kThreads == 0 && kBN * 8 % kThreads == 0, "whole loads");
    static constexpr int kScalesA = (kBM + kThreads - 1) / kThreads, kScalesB = (kBN + kThreads - 1) / kThreads;
    static constexpr int kReads = 2 * (kFM + kFN);  // LDS reads of a half block
    static_assert(kS >= 2 && kS <= 4, "scales of two groups of four blocks are held");
};

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t buffer_of(const uint8_t* p) {
    // offsets are kept in bounds by construction
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0xFFFFFFFFu, 0x00027000);
}

__device__ __forceinline__ int place(int p, int q) { return p * kB8 + ((q ^ (p >> 1 & 7)) << 4); }

// Asks the compiler to deal out a half block's LDS reads, two to a matrix
// instruction until there are no more, and kLoads direct loads, one to each,
// and to keep all of it on this side of what follows.
template <typename S, bool kExact, int kLoads>
__device__ __forceinline__ void interleave() {
    if (!kExact) {
        constexpr int kN = S::kFM * S::kFN, kPer = (kLoads + kN - 1) / kN;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);  // a matrix instruction
            if (i * 2 < S::kReads + (kLoads > 0 ? S::kFM + S::kFN : 0)) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            if (kLoads > 0) __builtin_amdgcn_sched_group_barrier(0x10, kPer, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Waits for this wave's LDS reads and all but its last kFlying direct loads
// (they end in order), then for the workgroup.
template <int kFlying>
__device__ __forceinline__ void arrive() {
    static_assert(kFlying < 64, "the counter's width");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kFlying) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Between lanes of one wave that pass values through LDS: what was written
// before is there afterwards, and what is read before is not overwritten.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The tile whose first element is (m0, n0), over part `part` of k.  The places
// in LDS are objects of their own, so that the compiler sees that loads into
// one do not touch reads of another (p2 and p3 may be null).
template <typename S, int kType, bool kExact>
__device__ __forceinline__ void tile(const ProductArgs& a, int parts, int part, int64_t m0, int64_t n0, uint8_t* p0,
                                     uint8_t* p1, uint8_t* p2, uint8_t* p3, uint32_t* lds_scales) {
    const auto place_of = [&](auto slot) {
        constexpr int i = decltype(slot)::value;
        return i == 0 ? p0 : i == 1 ? p1 : i == 2 ? p2 : p3;
    };
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWN, wn = wave % S::kWN;

    const int blocks = (a.k + kB8 - 1) / kB8;
    // parts begin at a multiple of four blocks (a word of scales)
    const int per = ((blocks + parts - 1) / parts + 3) & ~3;
    const int first = part * per, last = first + per < blocks ? first + per : blocks;

    // Rows past the end repeat the last one (their results are not stored).
    const rsrc_t codes_a = buffer_of(a.a.codes + m0 * a.a.codes_stride);
    const rsrc_t codes_b = buffer_of(a.b.codes + n0 * a.b.codes_stride);
    const int rows_a = a.a.rows - m0 < S::kBM ? static_cast<int>(a.a.rows - m0) : S::kBM;
    const int rows_b = a.b.rows - n0 < S::kBN ? static_cast<int>(a.b.rows - n0) : S::kBN;
    const auto row_of_a = [&](int p) { return p < rows_a ? p : rows_a - 1; };
    const auto row_of_b = [&](int p) {
        const int w = p / (32 * S::kFN), f = p / 32 % S::kFN, n = w * 32 * S::kFN + (p & 31) * S::kFN + f;
        return n < rows_b ? n : rows_b - 1;
    };
    uint32_t off_a[S::kLoadsA], off_b[S::kLoadsB];
    // the piece of its row that a lane loads, the same in all its rows (they are a multiple of 16 apart)
    const uint32_t piece = static_cast<uint32_t>((lane & 7) ^ (threadIdx.x >> 4 & 7)) << 4;
#pragma unroll
    for (int i = 0; i < S::kLoadsA; ++i)
        off_a[i] = static_cast<uint32_t>(row_of_a((i * S::kThreads + static_cast<int>(threadIdx.x)) >> 3)) *
                       a.a.codes_stride + piece;
#pragma unroll
    for (int i = 0; i < S::kLoadsB; ++i)
        off_b[i] = static_cast<uint32_t>(row_of_b((i * S::kThreads + static_cast<int>(threadIdx.x)) >> 3)) *
                       a.b.codes_stride + piece;

    // Loads a block; pieces past the row's end repeat the block's first.
    const auto load = [&](int block, auto slot) {
        const uint32_t k0 = static_cast<uint32_t>(block) * kB8;
        const uint32_t in = (static_cast<uint32_t>(a.k) - k0 + 15) & ~15u;
        const uint32_t back = piece >= in ? piece : 0;
        uint8_t* const to = place_of(slot) + wave * 1024;
#pragma unroll
        for (int i = 0; i < S::kLoadsA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(codes_a, (lds_ptr)(to + i * S::kThreads * 16), 16,
                                                     static_cast<int>(off_a[i] - back), static_cast<int>(k0), 0, 0);
#pragma unroll
        for (int i = 0; i < S::kLoadsB; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(codes_b, (lds_ptr)(to + S::kBM * kB8 + i * S::kThreads * 16), 16,
                                                     static_cast<int>(off_b[i] - back), static_cast<int>(k0), 0, 0);
    };
    // Loads the scales of four blocks; a wave's rows are all a's or all b's.
    const rsrc_t scales_a = buffer_of(scale_row(a.a, m0)), scales_b = buffer_of(scale_row(a.b, n0));
    uint32_t off_sa[S::kScalesA], off_sb[S::kScalesB];
#pragma unroll
    for (int i = 0; i < S::kScalesA; ++i)
        off_sa[i] = scale_offset(a.a, m0, row_of_a(i * S::kThreads + static_cast<int>(threadIdx.x)));
#pragma unroll
    for (int i = 0; i < S::kScalesB; ++i)
        off_sb[i] = scale_offset(a.b, n0, row_of_b(i * S::kThreads + static_cast<int>(threadIdx.x)));
    const auto load_scales = [&](int block) {
        uint32_t* const to = lds_scales + (block >> 2 & 1) * S::kRows + wave * 64;
#pragma unroll
        for (int i = 0; i < S::kScalesA; ++i)
            if ((i + 1) * S::kThreads <= S::kBM || i * S::kThreads + wave * 64 < S::kBM)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(scales_a, (lds_ptr)(to + i * S::kThreads), 4,
                                                         static_cast<int>(off_sa[i]), block, 0, 0);
#pragma unroll
        for (int i = 0; i < S::kScalesB; ++i)
            if ((i + 1) * S::kThreads <= S::kBN || i * S::kThreads + wave * 64 < S::kBN)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(scales_b, (lds_ptr)(to + S::kBM + i * S::kThreads), 4,
                                                         static_cast<int>(off_sb[i]), block, 0, 0);
    };
    const int r32 = lane & 31, g = lane >> 5;
    i32x8 fa[2][S::kFM], fb[2][S::kFN];
    uint32_t wa[S::kFM], wb[S::kFN];
    // Piece 2 g of the lane's rows; the other pieces and the other rows of a wave lie at fixed distances.
    const int at_a = place(wm * 32 * S::kFM + r32, g * 2), at_b = place(S::kBM + wn * 32 * S::kFN + r32, g * 2);
    const auto read_at = [&](const uint8_t* at, auto half) {
        constexpr int kk = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < S::kFM; ++i)
            fa[kk][i] = join(*reinterpret_cast<const i32x4*>(at + (at_a ^ kk * 64) + i * 32 * kB8),
                             *reinterpret_cast<const i32x4*>(at + (at_a ^ (kk * 64 + 16)) + i * 32 * kB8));
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
            fb[kk][j] = join(*reinterpret_cast<const i32x4*>(at + (at_b ^ kk * 64) + j * 32 * kB8),
                             *reinterpret_cast<const i32x4*>(at + (at_b ^ (kk * 64 + 16)) + j * 32 * kB8));
    };
    const auto read = [&](auto slot, auto half) { read_at(place_of(slot), half); };
    // Of half a block in registers, `left` codes of a row count, the others become zeros.
    const auto trim = [&](int left, auto half) {
        constexpr int kk = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < S::kFM; ++i) fa[kk][i] = keep(fa[kk][i], left - g * 32);
#pragma unroll
        for (int j = 0; j < S::kFN; ++j) fb[kk][j] = keep(fb[kk][j], left - g * 32);
    };
    // The words with the scales of a block, and the words shifted to it.
    uint32_t na[S::kFM], nb[S::kFN];
    const auto read_scales = [&](int block) {
        const uint32_t* const at = lds_scales + (block >> 2 & 1) * S::kRows;
#pragma unroll
        for (int i = 0; i < S::kFM; ++i) na[i] = at[wm * 32 * S::kFM + i * 32 + r32];
#pragma unroll
        for (int j = 0; j < S::kFN; ++j) nb[j] = at[S::kBM + wn * 32 * S::kFN + j * 32 + r32];
    };
    const auto take_scales = [&](int block) {
        const int shift = 8 * (block & 3);
#pragma unroll
        for (int i = 0; i < S::kFM; ++i) wa[i] = na[i] >> shift;
#pragma unroll
        for (int j = 0; j < S::kFN; ++j) wb[j] = nb[j] >> shift;
    };

    f32x16 acc[S::kFM][S::kFN];
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const auto multiply = [&](auto half) {
        constexpr int kk = decltype(half)::value;
        if (!kExact) {
#pragma unroll
            for (int i = 0; i < S::kFM; ++i)
#pragma unroll
                for (int j = 0; j < S::kFN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fa[kk][i], fb[kk][j], acc[i][j], 0, 0, 0, static_cast<int>(wa[i]), 0, static_cast<int>(wb[j]));
        } else {
            bf16x8 hb[S::kFN][4];
#pragma unroll
            for (int j = 0; j < S::kFN; ++j) {
                const uint32_t byte = wb[j] & 255u;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    hb[j][t] = widen(poisoned(fb[kk][j][2 * t], byte), fb[kk][j][2 * t + 1], scale_value(byte));
            }
#pragma unroll
            for (int i = 0; i < S::kFM; ++i) {
                const uint32_t byte = wa[i] & 255u;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const bf16x8 ha = widen(poisoned(fa[kk][i][2 * t], byte), fa[kk][i][2 * t + 1], scale_value(byte));
#pragma unroll
                    for (int j = 0; j < S::kFN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ha, hb[j][t], acc[i][j], 0, 0, 0);
                }
            }
        }
    };

    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    constexpr std::integral_constant<int, 3> k3{};
    if (first < last) {
        constexpr int kLoads = S::kLoadsA + S::kLoadsB;
        const bool ragged = last == blocks && (a.k & (kB8 - 1)) != 0;
        const int full = last - (ragged ? 1 : 0);
        // Loads past the last block repeat it, into a place that nobody reads any more.
        const auto load_ahead = [&](int block, auto slot) { load(block < last ? block : last - 1, slot); };
        const auto step = [&](int block, auto slot) {
            constexpr std::integral_constant<int, (decltype(slot)::value + 1) % S::kS> next{};
            if ((block + S::kS & 3) == 0 && block + S::kS < last) load_scales(block + S::kS);
            read(slot, k1);
            multiply(k0);
            interleave<S, kExact, 0>();
            arrive<(S::kS - 2) * kLoads>();
            load_ahead(block + S::kS, slot);
            read(next, k0);  // (past the last block: what is there, and not used)
            read_scales(block + 1);
            multiply(k1);
            interleave<S, kExact, kLoads>();
            take_scales(block + 1);
        };
        load_scales(first);
        load(first, k0);
        load_ahead(first + 1, k1);
        if (S::kS > 2) load_ahead(first + 2, k2);
        if (S::kS > 3) load_ahead(first + 3, k3);
        arrive<(S::kS - 1) * kLoads>();
        read(k0, k0);
        read_scales(first);
        take_scales(first);
        int block = first;
        for (; block + S::kS <= full; block += S::kS) {
            step(block, k0);
            step(block + 1, k1);
            if (S::kS > 2) step(block + 2, k2);
            if (S::kS > 3) step(block + 3, k3);
        }
        uint8_t* at = p0;  // the place of block `block`
        if (block < full) {
            step(block++, k0);
            at = p1;
            if (S::kS > 2 && block < full) {
                step(block++, k1);
                at = p2;
                if (S::kS > 3 && block < full) {
                    step(block++, k2);
                    at = p3;
                }
            }
        }
        if (ragged) {  // its first half has been read
            const int left = a.k - block * kB8;
            if (left < kB8 / 2) trim(left, k0);
            multiply(k0);
            if (left > kB8 / 2) {
                read_at(at, k1);
                trim(left - kB8 / 2, k1);
                multiply(k1);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may outlive the workgroup's LDS
    }

    // A lane has kFN neighbouring columns of 16 rows of each of its squares.
    typedef typename Out<kType>::T T;
    const int64_t corner = n0 + wn * 32 * S::kFN;
    if (parts > 1) {
        // the parts' sums are kept by whole tiles
        float* to = a.part + (part * a.part_rows + m0 + wm * 32 * S::kFM + g * 4) * a.part_stride + corner + r32 * S::kFN;
#pragma unroll
        for (int i = 0; i < S::kFM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float v[S::kFN];
#pragma unroll
                for (int j = 0; j < S::kFN; ++j) v[j] = acc[i][j][e];
                store_whole<float, S::kFN, false>(to, v, nullptr);
                to += ((e & 3) == 3 ? 5 : 1) * a.part_stride;
            }
        return;
    }
    if (rows_a == S::kBM && rows_b == S::kBN) {
        // a whole tile: straight out of the registers
        T* to = static_cast<T*>(a.out) + (m0 + wm * 32 * S::kFM + g * 4) * a.out_stride + corner + r32 * S::kFN;
        const T* add = static_cast<const T*>(a.add) + (m0 + wm * 32 * S::kFM + g * 4) * a.add_stride + corner +
                       r32 * S::kFN;
        const auto store = [&](auto with) {
            constexpr bool kAdd = decltype(with)::value;
            constexpr int kAhead = 8;  // rows whose addends are read at once (out may be the same memory)
            typedef typename Pack<T, S::kFN>::V V;
#pragma unroll
            for (int i = 0; i < S::kFM; ++i)
#pragma unroll
                for (int e0 = 0; e0 < 16; e0 += kAhead) {
                    V y[kAhead];
#pragma unroll
                    for (int e = 0; e < kAhead; ++e) {
                        y[e] = V{};
                        if (kAdd) y[e] = *reinterpret_cast<const V*>(add);
                        add += ((e & 3) == 3 ? 5 : 1) * a.add_stride;
                    }
#pragma unroll
                    for (int e = 0; e < kAhead; ++e) {
                        V x;
#pragma unroll
                        for (int j = 0; j < S::kFN; ++j)
                            x[j] = static_cast<T>(kAdd ? acc[i][j][e0 + e] + static_cast<float>(y[e][j])
                                                       : acc[i][j][e0 + e]);
                        *reinterpret_cast<V*>(to) = x;
                        to += ((e & 3) == 3 ? 5 : 1) * a.out_stride;
                    }
                }
        };
        if (a.add == nullptr)
            store(std::false_type());
        else
            store(std::true_type());
        return;
    }
    // Else 32 rows at a time through LDS, each wave in a place of its own, so
    // that the masks and the addend come in a short loop.
    constexpr int kWide = 32 * S::kFN;
    constexpr int kHalf = S::kWM * S::kWN / 2;
    static_assert(kWide * 32 * 4 * kHalf <= S::kRows * kB8, "room for the waves' squares");
    __syncthreads();  // the last block's reads
    float* const mine = reinterpret_cast<float*>(wave < kHalf ? p0 : p1) + wave % kHalf * kWide * 32;
    const int64_t left = a.b.rows - corner - r32 * S::kFN;
#pragma unroll
    for (int i = 0; i < S::kFM; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            typedef float V __attribute__((ext_vector_type(S::kFN)));
            V v;
#pragma unroll
            for (int j = 0; j < S::kFN; ++j) v[j] = acc[i][j][e];
            *reinterpret_cast<V*>(mine + ((e >> 2) * 8 + g * 4 + (e & 3)) * kWide + r32 * S::kFN) = v;
        }
        wave_exchange();
        const int p0 = wm * 32 * S::kFM + i * 32;
        constexpr int kAhead = 4;  // rows whose addends are read at once
        for (int t = 0; t < 16 && p0 + 2 * t < rows_a; t += kAhead) {
            float v[kAhead][S::kFN];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int j = 0; j < S::kFN; ++j) v[u][j] = mine[(2 * (t + u) + g) * kWide + r32 * S::kFN + j];
            if (a.add != nullptr) {
                float y[kAhead][S::kFN];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    // (rows and columns past the end: the last ones stand in)
                    const int p = p0 + 2 * (t + u) + g;
                    const T* add = static_cast<const T*>(a.add) + (m0 + (p < rows_a ? p : rows_a - 1)) * a.add_stride;
#pragma unroll
                    for (int j = 0; j < S::kFN; ++j)
                        y[u][j] = static_cast<float>(add[j < left ? corner + r32 * S::kFN + j : a.b.rows - 1]);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int j = 0; j < S::kFN; ++j) v[u][j] += y[u][j];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int p = p0 + 2 * (t + u) + g;
                if (p >= rows_a || left <= 0) continue;
                const int64_t row = m0 + p, col = corner + r32 * S::kFN;
                store_run<T, S::kFN>(static_cast<T*>(a.out) + row * a.out_stride + col, v[u], nullptr, left);
            }
        }
        wave_exchange();
    }
}

// Tile `id` of tiles of `high` x `wide`: in bands of 8 tile rows, column by column.
__device__ __forceinline__ void corner_of(uint32_t id, const ProductArgs& a, int high, int wide, int64_t& m0,
                                          int64_t& n0) {
    const uint32_t tm = static_cast<uint32_t>((a.a.rows + high - 1) / high);
    const uint32_t tn = static_cast<uint32_t>((a.b.rows + wide - 1) / wide);
    const uint32_t band = id / (8 * tn), in_band = id - band * 8 * tn;
    const uint32_t rows = tm - band * 8 < 8 ? tm - band * 8 : 8, across = in_band / rows;
    m0 = static_cast<int64_t>(band * 8 + in_band - across * rows) * high;
    n0 = static_cast<int64_t>(across) * wide;
}

// The places of a workgroup in LDS, each an object of its own.
#define ZDP_PLACES(S)                                                                              \
    __shared__ __attribute__((aligned(1024))) uint8_t place0[S::kRows * kB8];                      \
    __shared__ __attribute__((aligned(1024))) uint8_t place1[S::kRows * kB8];                      \
    __shared__ __attribute__((aligned(1024))) uint8_t place2[S::kS > 2 ? S::kRows * kB8 : 1];      \
    __shared__ __attribute__((aligned(1024))) uint8_t place3[S::kS > 3 ? S::kRows * kB8 : 1];      \
    __shared__ uint32_t lds_scales[2 * S::kRows];

// The first `count` tiles of shape S.  Consecutive workgroups go to the eight
// dies in turn; each die takes a run of neighbouring tiles, whose operands
// then meet in its L2.
template <typename S, int kType>
__global__ __launch_bounds__(S::kThreads) void product_kernel(ProductArgs a, int parts, uint32_t count) {
    ZDP_PLACES(S)
    const uint32_t die = blockIdx.x & 7, more = count & 7;
    int64_t m0, n0;
    corner_of(die * (count >> 3) + (die < more ? die : more) + (blockIdx.x >> 3), a, S::kBM, S::kBN, m0, n0);
    tile<S, kType, kType == ZERO_TYPE_F32>(a, parts, blockIdx.y, m0, n0, place0, place1, place2, place3, lds_scales);
}

// The tiles from `first` on of twice S's size, each as four of shape S.
template <typename S, int kType>
__global__ __launch_bounds__(S::kThreads) void product_rest_kernel(ProductArgs a, uint32_t first) {
    ZDP_PLACES(S)
    int64_t m0, n0;
    corner_of(first + (blockIdx.x >> 2), a, 2 * S::kBM, 2 * S::kBN, m0, n0);
    m0 += (blockIdx.x >> 1 & 1) * S::kBM;
    n0 += (blockIdx.x & 1) * S::kBN;
    if (m0 < a.a.rows && n0 < a.b.rows)
        tile<S, kType, kType == ZERO_TYPE_F32>(a, 1, 0, m0, n0, place0, place1, place2, place3, lds_scales);
}
#undef ZDP_PLACES

// The parts' sum, in order, and the addend; a lane takes four columns.
template <int kType>
__global__ __launch_bounds__(256) void join_parts_kernel(ProductArgs a, int parts) {
    typedef typename Out<kType>::T T;
    const uint32_t across = static_cast<uint32_t>((a.b.rows + 3) / 4);
    const uint32_t units = static_cast<uint32_t>(a.a.rows) * across;  // (of at most 256 tiles)
    const int64_t apart = a.part_rows * a.part_stride;
    for (uint32_t u = blockIdx.x * 256 + threadIdx.x; u < units; u += gridDim.x * 256) {
        const uint32_t row = u / across, c = (u - row * across) * 4;
        const float* from = a.part + row * a.part_stride + c;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int p = 0; p < parts; ++p) x += *reinterpret_cast<const f32x4*>(from + p * apart);
        const float v[4] = {x[0], x[1], x[2], x[3]};
        store_run<T, 4>(static_cast<T*>(a.out) + row * a.out_stride + c, v,
                        a.add == nullptr ? nullptr : static_cast<const T*>(a.add) + row * a.add_stride + c,
                        a.b.rows - c);
    }
}

// --------------------------------------------------------------- few rows
// Products whose time is latency or the reading of one operand: no LDS on the
// way in.  A workgroup takes 16 rows of the one operand (the stream, read
// once) against 16 kT of the other, its waves blocks of k in turn, straight
// into registers; the waves' sums meet in LDS.  b's rows are the instruction's
// first operand, whichever the stream is, so that a lane holds four
// neighbouring columns of out.  1 x 6400 x 1600 bf16: 4.5 us (2.3 TB/s, of
// which 2 to 3 us are a launch's own); 8 x 8192 x 8192: 17 us, 3.9 TB/s.
//
// The matrix instructions' rate bounds little of it, so sums are in fp32 for every
// type of out, over the bf16 instructions, at 0 to 10 % (1 x 6400 x 1600: 4.3 us
// over the 8-bit ones; 267 x 1327 x 826: 5.8 and 5.5; 1034 x 165 x 4042: 11.7 and
// 10.8; 8 x 8192 x 8192: 17.1 and 16.9).  A 16-bit out takes the 8-bit ones for a block with a
// scale whose values bf16 does not hold.
constexpr int kFewWaves = 8;

// Whether bf16 holds every e4m3 value under a scale byte: 2^-9 at 10 is 2^-126,
// 448 at 246 is 1.75 * 2^127.
__device__ __forceinline__ bool fits_bf16(uint32_t byte) { return (byte >= 10u && byte <= 246u) || byte == 255u; }

template <int kType, bool kStreamA, int kT>
__global__ __launch_bounds__(kFewWaves * 64) void product_few_kernel(ProductArgs a) {
    constexpr bool kExact = kType == ZERO_TYPE_F32;
    __shared__ f32x4 sums[kFewWaves][kT][64];
    const ProductSide& stream = kStreamA ? a.a : a.b;
    const ProductSide& other = kStreamA ? a.b : a.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t s0 = static_cast<int64_t>(blockIdx.x) * 16, t0 = static_cast<int64_t>(blockIdx.y) * 16 * kT;
    // rows past the end repeat the last one
    const int64_t row_s = s0 + r < stream.rows ? s0 + r : stream.rows - 1;
    const uint8_t* const ps = stream.codes + row_s * stream.codes_stride;
    const uint8_t* const ss = scale_row(stream, row_s);
    const uint8_t *pt[kT], *st[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
        const int64_t row = t0 + t * 16 + r < other.rows ? t0 + t * 16 + r : other.rows - 1;
        pt[t] = other.codes + row * other.codes_stride;
        st[t] = scale_row(other, row);
    }
    f32x4 acc[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int blocks = (a.k + kB8 - 1) / kB8;
    for (int block = wave; block < blocks; block += kFewWaves) {
        // of a row's eight pieces of 16 a lane takes g and g + 4: each load reads half rows, whole
        const int k = block * kB8 + g * 16, left = a.k - k;
        // pieces past the row's end repeat its first
        const int o0 = left > 0 ? k : 0, o1 = left > 64 ? k + 64 : 0;
        i32x4 x[2], y[kT][2];
        uint32_t et[kT];
        x[0] = *reinterpret_cast<const i32x4*>(ps + o0);
        x[1] = *reinterpret_cast<const i32x4*>(ps + o1);
        const uint32_t es = ss[block];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            y[t][0] = *reinterpret_cast<const i32x4*>(pt[t] + o0);
            y[t][1] = *reinterpret_cast<const i32x4*>(pt[t] + o1);
            et[t] = st[t][block];
        }
        if ((block + 1) * kB8 > a.k) {
            x[0] = keep(x[0], left);
            x[1] = keep(x[1], left - 64);
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                y[t][0] = keep(y[t][0], left);
                y[t][1] = keep(y[t][1], left - 64);
            }
        }
        const i32x8 fs = join(x[0], x[1]);
        bool fits = fits_bf16(es);
#pragma unroll
        for (int t = 0; t < kT; ++t) fits = fits && fits_bf16(et[t]);
        if (!kExact && !__all(fits)) {
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                const i32x8 ft = join(y[t][0], y[t][1]), u = kStreamA ? ft : fs, v = kStreamA ? fs : ft;
                const int eu = static_cast<int>(kStreamA ? et[t] : es), ev = static_cast<int>(kStreamA ? es : et[t]);
                acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v, acc[t], 0, 0, 0, eu, 0, ev);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 hs = widen(poisoned(fs[2 * j], es), fs[2 * j + 1], scale_value(es));
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    const i32x4 ft = y[t][j >> 1];
                    const bf16x8 ht =
                        widen(poisoned(ft[2 * (j & 1)], et[t]), ft[2 * (j & 1) + 1], scale_value(et[t]));
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kStreamA ? ht : hs, kStreamA ? hs : ht, acc[t], 0,
                                                                     0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) sums[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= kT) return;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        const f32x4 x = sums[w][wave][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[i];
    }
    const int64_t t1 = t0 + wave * 16;
    const int64_t row = kStreamA ? s0 + r : t1 + r, c = (kStreamA ? t1 : s0) + g * 4;
    if (row >= a.a.rows || c >= a.b.rows) return;
    typedef typename Out<kType>::T T;
    store_run<T, 4>(static_cast<T*>(a.out) + row * a.out_stride + c, v,
                    a.add == nullptr ? nullptr : static_cast<const T*>(a.add) + row * a.add_stride + c, a.b.rows - c);
}

// --------------------------------------------------------------- launchers
int finish() {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return ZERO_OK;
    zdp::set_last_hip_error(static_cast<int>(e));
    return ZERO_EHIP;
}

template <int kType, bool kStreamA>
void launch_few(const ProductArgs& a, hipStream_t s) {
    const int64_t stream = kStreamA ? a.a.rows : a.b.rows, other = kStreamA ? a.b.rows : a.a.rows;
    const int64_t t = zdp::product_few_rows(other);
    const dim3 grid(static_cast<unsigned>((stream + 15) / 16), static_cast<unsigned>((other + 16 * t - 1) / (16 * t)));
    if (t == 1)
        product_few_kernel<kType, kStreamA, 1><<<grid, kFewWaves * 64, 0, s>>>(a);
    else if (t == 2)
        product_few_kernel<kType, kStreamA, 2><<<grid, kFewWaves * 64, 0, s>>>(a);
    else
        product_few_kernel<kType, kStreamA, 4><<<grid, kFewWaves * 64, 0, s>>>(a);
}

typedef Shape<256, 256, 2, 4, 2> Large;
typedef Shape<192, 256, 2, 4, 2> Medium;
typedef Shape<128, 128, 2, 2, 4> Small;
static_assert(Large::kBM == 2 * Small::kBM && Large::kBN == 2 * Small::kBN, "a large tile is four small ones");

template <typename S, int kType>
void launch_tiles(const ProductArgs& a, int parts, hipStream_t s) {
    const int64_t tiles = ((a.a.rows + S::kBM - 1) / S::kBM) * ((a.b.rows + S::kBN - 1) / S::kBN);
    const int64_t rest = std::is_same<S, Large>::value ? zdp::product_rest(tiles) : 0;
    const uint32_t count = static_cast<uint32_t>(tiles - rest);
    product_kernel<S, kType><<<dim3(count, static_cast<unsigned>(parts)), S::kThreads, 0, s>>>(a, parts, count);
    if (rest > 0)
        product_rest_kernel<Small, kType><<<static_cast<unsigned>(4 * rest), Small::kThreads, 0, s>>>(a, count);
    if (parts > 1) {
        const int64_t units = (a.a.rows * ((a.b.rows + 3) / 4) + 255) / 256;
        join_parts_kernel<kType><<<static_cast<unsigned>(units < 8192 ? units : 8192), 256, 0, s>>>(a, parts);
    }
}

template <int kType>
void launch_typed(const ProductArgs& a, int parts, hipStream_t s) {
    switch (zdp::product_shape(a.a.rows, a.b.rows, a.k, kType == ZERO_TYPE_F32)) {
        case zdp::kProductFewB: launch_few<kType, false>(a, s); break;
        case zdp::kProductFewA: launch_few<kType, true>(a, s); break;
        case zdp::kProductSmall: launch_tiles<Small, kType>(a, parts, s); break;
        case zdp::kProductMedium: launch_tiles<Medium, kType>(a, parts, s); break;
        default: launch_tiles<Large, kType>(a, parts, s); break;
    }
}

}  // namespace

namespace zdp {

int launch_block8_product(const ProductArgs& a, int parts, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.type == ZERO_TYPE_F32)
        launch_typed<ZERO_TYPE_F32>(a, parts, s);
    else if (a.type == ZERO_TYPE_F16)
        launch_typed<ZERO_TYPE_F16>(a, parts, s);
    else
        launch_typed<ZERO_TYPE_BF16>(a, parts, s);
    return finish();
}

}  // namespace zdp
