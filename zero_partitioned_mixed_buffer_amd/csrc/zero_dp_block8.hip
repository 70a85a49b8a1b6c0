// Device side of the 8-bit layer operators for CDNA4 (gfx950): the encode of a
// matrix, and the root-mean-square norm with its gradients.
//
//   norm      h = T(x + r);  rstd = 1 / sqrt(mean h^2 + eps);  y = (h rstd) w, in
//             the 8-bit form by rows
//   backward  xh = h rstd;  g = dy w;  c = mean(g xh);
//             dx = (g - xh c) rstd + dh;  dw = sum over rows of dy xh
//   encode    x, or x row_mul col_mul, in the 8-bit form, its transposed, or both
//
// All of it is a stream over memory: each input is read once and each output
// written once.  A lane owns units of 8 consecutive columns (16 bytes of
// 16-bit values, 8 of codes), so that the 16 lanes of a DPP row own one block
// of 128 and its largest magnitude takes four register moves.  No two
// workgroups write the same bytes and every sum has a fixed order, so results
// repeat bit for bit.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/zero_dp.h"
#include "zero_dp_block8.h"
#include "zero_dp_fp8.h"

#pragma clang fp contract(off)

namespace {

using zdp::bits_of;
using zdp::EncodeArgs;
using zdp::float_of;
using zdp::kB8;
using zdp::NormArgs;
using zdp::NormBackArgs;
using zdp::scale_byte;

constexpr int kU = 8;           // columns of a lane's unit
constexpr int kSweep = 64 * kU;  // columns of a wave's sweep: four blocks

// Rows and vectors need only their elements' own alignment.
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------ units of 8 elements
template <int kType>
struct Raw {
    static constexpr int kWords = kType == ZERO_TYPE_F32 ? 8 : 4;
    static constexpr int kSize = kType == ZERO_TYPE_F32 ? 4 : 2;
    uint32_t w[kWords];
};

// Elements c .. c + 7 of a row of n; zeros past its end.
template <int kType>
__device__ __forceinline__ Raw<kType> load_unit(const char* row, int c, int n) {
    Raw<kType> x;
    if (c + kU <= n) {
        if (kType == ZERO_TYPE_F32) {
            const u32x4_4* p = reinterpret_cast<const u32x4_4*>(row + static_cast<int64_t>(c) * 4);
            const u32x4_4 a = p[0], b = p[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x.w[i] = a[i];
                x.w[(4 + i) % Raw<kType>::kWords] = b[i];
            }
        } else {
            const u32x4_2 a = *reinterpret_cast<const u32x4_2*>(row + static_cast<int64_t>(c) * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.w[i] = a[i];
        }
        return x;
    }
#pragma unroll
    for (int i = 0; i < Raw<kType>::kWords; ++i) x.w[i] = 0;
    if (c >= n) return x;
    if (kType == ZERO_TYPE_F32) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < Raw<kType>::kWords; ++i)
            if (c + i < n) x.w[i] = p[i];
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < kU; ++i)
            if (c + i < n) x.w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
    }
    return x;
}

// The same where a unit at the row's end is common (small matrices): its loads
// do not wait for each other, the last element standing in for what is not
// there.  (In the norm's kernels it costs: 8192 x 1600 bf16 19.7 -> 23.5 us.)
template <int kType>
__device__ __forceinline__ Raw<kType> load_end(const char* row, int c, int n) {
    if (c + kU <= n || c >= n) return load_unit<kType>(row, c, n);
    uint32_t e[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        const int at = c + i < n ? c + i : n - 1;
        e[i] = kType == ZERO_TYPE_F32 ? reinterpret_cast<const uint32_t*>(row)[at]
                                      : reinterpret_cast<const uint16_t*>(row)[at];
    }
    Raw<kType> x;
#pragma unroll
    for (int i = 0; i < kU; ++i) e[i] = c + i < n ? e[i] : 0;
#pragma unroll
    for (int i = 0; i < Raw<kType>::kWords; ++i)
        x.w[i] = kType == ZERO_TYPE_F32 ? e[i] : e[2 * i % kU] | e[(2 * i + 1) % kU] << 16;
    return x;
}

template <int kType>
__device__ __forceinline__ void store_unit(char* row, int c, int n, const Raw<kType>& x) {
    if (c + kU <= n) {
        if (kType == ZERO_TYPE_F32) {
            u32x4_4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = x.w[i];
                b[i] = x.w[(4 + i) % Raw<kType>::kWords];
            }
            u32x4_4* p = reinterpret_cast<u32x4_4*>(row + static_cast<int64_t>(c) * 4);
            p[0] = a;
            p[1] = b;
        } else {
            u32x4_2 a;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = x.w[i];
            *reinterpret_cast<u32x4_2*>(row + static_cast<int64_t>(c) * 2) = a;
        }
        return;
    }
    if (kType == ZERO_TYPE_F32) {
        uint32_t* p = reinterpret_cast<uint32_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < Raw<kType>::kWords; ++i)
            if (c + i < n) p[i] = x.w[i];
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < kU; ++i)
            if (c + i < n) p[i] = static_cast<uint16_t>(x.w[i / 2] >> (16 * (i & 1)));
    }
}

template <int kType>
__device__ __forceinline__ void unpack(const Raw<kType>& x, float (&v)[kU]) {
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        if (kType == ZERO_TYPE_F32) {
            v[i] = float_of(x.w[i % Raw<kType>::kWords]);
        } else if (kType == ZERO_TYPE_BF16) {
            v[i] = float_of(i & 1 ? x.w[i / 2] & 0xFFFF0000u : x.w[i / 2] << 16);
        } else {
            v[i] = static_cast<float>(__builtin_bit_cast(f16x2, x.w[i / 2])[i & 1]);
        }
    }
}

// To the type, to nearest even.
template <int kType>
__device__ __forceinline__ Raw<kType> pack(const float (&v)[kU]) {
    Raw<kType> x;
#pragma unroll
    for (int i = 0; i < Raw<kType>::kWords; ++i) {
        if (kType == ZERO_TYPE_F32) {
            x.w[i] = bits_of(v[i]);
        } else if (kType == ZERO_TYPE_BF16) {
            bf16x2 t;
            t[0] = static_cast<__bf16>(v[2 * i % kU]);
            t[1] = static_cast<__bf16>(v[(2 * i + 1) % kU]);
            x.w[i] = __builtin_bit_cast(uint32_t, t);
        } else {
            f16x2 t;
            t[0] = static_cast<_Float16>(v[2 * i % kU]);
            t[1] = static_cast<_Float16>(v[(2 * i + 1) % kU]);
            x.w[i] = __builtin_bit_cast(uint32_t, t);
        }
    }
    return x;
}

// A vector of any of the types (a norm's weight): the branch is the same for
// the whole grid.
__device__ __forceinline__ void load_vector(const void* w, int type, int c, int n, float (&v)[kU]) {
    const char* p = static_cast<const char*>(w);
    if (type == ZERO_TYPE_F32)
        unpack(load_unit<ZERO_TYPE_F32>(p, c, n), v);
    else if (type == ZERO_TYPE_F16)
        unpack(load_unit<ZERO_TYPE_F16>(p, c, n), v);
    else
        unpack(load_unit<ZERO_TYPE_BF16>(p, c, n), v);
}

// ------------------------------------------------------------- reductions
// A register's value in another lane of the same DPP row of 16: lane ^ 1, lane
// ^ 2, the mirrored lane of the 8 and of the 16.
template <int kStep>
__device__ __forceinline__ uint32_t swap16(uint32_t x) {
    constexpr int kCtl = kStep == 0 ? 0xB1 : kStep == 1 ? 0x4E : kStep == 2 ? 0x141 : 0x140;
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), kCtl, 0xF, 0xF, true));
}
template <int kStep>
__device__ __forceinline__ float swap16(float x) {
    return float_of(swap16<kStep>(bits_of(x)));
}
template <int kStep>
__device__ __forceinline__ double swap16(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint64_t lo = swap16<kStep>(static_cast<uint32_t>(b)), hi = swap16<kStep>(static_cast<uint32_t>(b >> 32));
    return __builtin_bit_cast(double, hi << 32 | lo);
}

__device__ __forceinline__ uint32_t lane_of(uint32_t x, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}
__device__ __forceinline__ float lane_of(float x, int lane) { return float_of(lane_of(bits_of(x), lane)); }
__device__ __forceinline__ double lane_of(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint64_t lo = lane_of(static_cast<uint32_t>(b), lane), hi = lane_of(static_cast<uint32_t>(b >> 32), lane);
    return __builtin_bit_cast(double, hi << 32 | lo);
}

// Largest value over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = max(x, swap16<0>(x));
    x = max(x, swap16<1>(x));
    x = max(x, swap16<2>(x));
    return max(x, swap16<3>(x));
}

// Sum over a row's waves, the same in every lane.  `turn` counts the
// workgroup's sums: two places in LDS, used in turn, need one barrier a sum.
template <int kWaves, typename F>
__device__ __forceinline__ F row_sum(F x, int turn) {
    x += swap16<0>(x);
    x += swap16<1>(x);
    x += swap16<2>(x);
    x += swap16<3>(x);
    x = (lane_of(x, 0) + lane_of(x, 16)) + (lane_of(x, 32) + lane_of(x, 48));
    if (kWaves > 1) {
        __shared__ F s[2][kWaves];
        F* const at = s[turn & 1];
        if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = x;
        __syncthreads();
        x = at[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) x += at[w];
    }
    return x;
}

// ------------------------------------------------------------------- codes
__device__ __forceinline__ uint32_t magnitude(const float (&v)[kU]) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < kU; ++i) big = max(big, bits_of(v[i]) & 0x7FFFFFFFu);
    return big;
}

// The codes of four values under their block's scale byte.  The largest
// scale's codes end at 240: 256 * 2^120 would read as inf.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, uint32_t byte) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    constexpr float most = 0x1.Ep127f;
    const float scale = float_of(byte << 23);
    a = __builtin_amdgcn_fmed3f(a, -most, most);
    b = __builtin_amdgcn_fmed3f(b, -most, most);
    c = __builtin_amdgcn_fmed3f(c, -most, most);
    d = __builtin_amdgcn_fmed3f(d, -most, most);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
    return byte == 255u ? 0x7F7F7F7Fu : __builtin_bit_cast(uint32_t, r);
}

// A unit's codes; rows of codes start on 16 bytes.
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int n, uint32_t lo, uint32_t hi) {
    if (c + kU <= n) {
        u32x2 x;
        x[0] = lo;
        x[1] = hi;
        *reinterpret_cast<u32x2*>(row + c) = x;
        return;
    }
#pragma unroll
    for (int i = 0; i < kU; ++i)
        if (c + i < n) row[c + i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

// The scale bytes of a wave's sweep, whose first column is c0: one word, or
// single bytes at the end of the row.
__device__ __forceinline__ void store_scales(uint8_t* row, int c0, int n, uint32_t byte) {
    const int lane = threadIdx.x & 63, b0 = c0 / kB8, nb = (n + kB8 - 1) / kB8;
    if (b0 + 4 <= nb) {
        const uint32_t word =
            lane_of(byte, 0) | lane_of(byte, 16) << 8 | lane_of(byte, 32) << 16 | lane_of(byte, 48) << 24;
        if (lane == 0) *reinterpret_cast<uint32_t*>(row + b0) = word;
    } else if ((lane & 15) == 0 && b0 + (lane >> 4) < nb) {
        row[b0 + (lane >> 4)] = static_cast<uint8_t>(byte);
    }
}

// A unit of values, in the 8-bit form by rows.
__device__ __forceinline__ void emit(uint8_t* codes, uint8_t* scales, int c, int n, const float (&v)[kU]) {
    const uint32_t byte = scale_byte(max16(magnitude(v)));
    store_codes(codes, c, n, codes4(v[0], v[1], v[2], v[3], byte), codes4(v[4], v[5], v[6], v[7], byte));
    store_scales(scales, c & ~(kSweep - 1), n, byte);
}

template <int kType>
__device__ __forceinline__ const char* row_of(const void* p, int64_t row, int64_t stride) {
    return static_cast<const char*>(p) + row * stride * Raw<kType>::kSize;
}
template <int kType>
__device__ __forceinline__ char* row_of(void* p, int64_t row, int64_t stride) {
    return static_cast<char*>(p) + row * stride * Raw<kType>::kSize;
}

// h = T(x + r) of a unit: what is stored, and its values.
template <int kType>
__device__ __forceinline__ Raw<kType> add_units(const Raw<kType>& x, const Raw<kType>& r, float (&v)[kU]) {
    float b[kU];
    unpack(x, v);
    unpack(r, b);
#pragma unroll
    for (int i = 0; i < kU; ++i) v[i] += b[i];
    const Raw<kType> h = pack<kType>(v);
    unpack(h, v);
    return h;
}

__device__ __forceinline__ double square_sum(const float (&v)[kU], double s) {
#pragma unroll
    for (int i = 0; i < kU; ++i) s = __builtin_fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
    return s;
}

__device__ __forceinline__ float rstd_of(double sum, int cols, double eps) {
    return static_cast<float>(1.0 / __builtin_sqrt(sum / cols + eps));
}

__device__ __forceinline__ void scaled(const float (&h)[kU], float rstd, const float (&w)[kU], float (&y)[kU]) {
#pragma unroll
    for (int i = 0; i < kU; ++i) y[i] = (h[i] * rstd) * w[i];
}

// ------------------------------------------------------------------- norm
// A row is held in registers, kNS units a lane, by kWaves waves; rows of one
// wave need no barrier, and kPack of them make a workgroup.  A workgroup takes
// rows in turn, the next one's loads under way while this one is worked on,
// and keeps its columns' weights in registers.  Bound by memory: 8192 x 1600
// bf16 with a residual 19.4 us, 4.7 TB/s (a copy reaches 5.2); by instructions
// too without one, where fewer bytes go by: 4099 x 12288 fp16 35 us, 4.3 TB/s (one
// column more, a unit more for every lane: 45).
template <int kWaves>
constexpr int kPack = kWaves == 1 ? 4 : 1;
template <int kWaves>
constexpr int kThreads = 64 * kWaves * kPack<kWaves>;

// A vector's units of a lane.
template <int kNS>
__device__ __forceinline__ void load_weights(const void* w, int type, int c0, int across, int n, float (&v)[kNS][kU]) {
#pragma unroll
    for (int s = 0; s < kNS; ++s) load_vector(w, type, c0 + s * across, n, v[s]);
}

// A row's units of a lane.
template <int kType, int kNS>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int64_t stride, int c0, int across, int n,
                                         Raw<kType> (&x)[kNS]) {
    const char* from = row_of<kType>(p, row, stride);
#pragma unroll
    for (int s = 0; s < kNS; ++s) x[s] = load_unit<kType>(from, c0 + s * across, n);
}

template <int kType, bool kRes, int kWaves, int kNS>
__global__ __launch_bounds__(kThreads<kWaves>) void norm8_kernel(NormArgs a) {
    constexpr int across = kWaves * kSweep;
    const int c0 = (kWaves == 1 ? threadIdx.x & 63 : threadIdx.x) * kU;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPack<kWaves>;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kPack<kWaves> + (kWaves == 1 ? threadIdx.x >> 6 : 0);
    if (row >= a.rows) return;
    Raw<kType> nx[kNS], nr[kNS];
    load_row<kType>(a.x, row, a.x_stride, c0, across, a.cols, nx);
    if (kRes) load_row<kType>(a.r, row, a.r_stride, c0, across, a.cols, nr);
    float w[kNS][kU];
    load_weights(a.w, a.w_type, c0, across, a.cols, w);
    for (int turn = 0; row < a.rows; row += step, ++turn) {
        float v[kNS][kU];
        double sum = 0.0;
        char* h = row_of<kType>(a.h, row, a.h_stride);
#pragma unroll
        for (int s = 0; s < kNS; ++s) {
            const int c = c0 + s * across;
            if (kRes) {
                const Raw<kType> y = add_units(nx[s], nr[s], v[s]);
                if (c < a.cols) store_unit(h, c, a.cols, y);
            } else {
                unpack(nx[s], v[s]);
            }
            sum = square_sum(v[s], sum);
        }
        if (row + step < a.rows) {
            load_row<kType>(a.x, row + step, a.x_stride, c0, across, a.cols, nx);
            if (kRes) load_row<kType>(a.r, row + step, a.r_stride, c0, across, a.cols, nr);
        }
        const float rstd = rstd_of(row_sum<kWaves>(sum, turn), a.cols, a.eps);
        if (c0 == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int s = 0; s < kNS; ++s) {
            const int c = c0 + s * across;
            if ((c & ~(kSweep - 1)) >= a.cols) break;  // the whole wave
            float y[kU];
            scaled(v[s], rstd, w[s], y);
            emit(a.codes + row * a.codes_stride, a.scales + row * a.scales_stride, c, a.cols, y);
        }
    }
}

// Rows longer than the registers of a workgroup: read twice (h again, out of
// the cache; each lane reads what it wrote itself).
constexpr int kLongWaves = 16;

template <int kType, bool kRes>
__global__ __launch_bounds__(kLongWaves * 64) void norm8_long_kernel(NormArgs a) {
    constexpr int kStep = kLongWaves * kSweep;
    const int c0 = threadIdx.x * kU;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
        const char* x = row_of<kType>(a.x, row, a.x_stride);
        const char* r = row_of<kType>(a.r, row, a.r_stride);
        char* h = row_of<kType>(a.h, row, a.h_stride);
        double sum = 0.0;
        for (int c = c0; c < a.cols; c += kStep) {
            float v[kU];
            const Raw<kType> rx = load_unit<kType>(x, c, a.cols);
            if (kRes)
                store_unit(h, c, a.cols, add_units(rx, load_unit<kType>(r, c, a.cols), v));
            else
                unpack(rx, v);
            sum = square_sum(v, sum);
        }
        const float rstd = rstd_of(row_sum<kLongWaves>(sum, turn), a.cols, a.eps);
        if (threadIdx.x == 0) a.rstd[row] = rstd;
        for (int c = c0; (c & ~(kSweep - 1)) < a.cols; c += kStep) {
            float v[kU], w[kU], y[kU];
            unpack(load_unit<kType>(kRes ? h : x, c, a.cols), v);
            load_vector(a.w, a.w_type, c, a.cols, w);
            scaled(v, rstd, w, y);
            emit(a.codes + row * a.codes_stride, a.scales + row * a.scales_stride, c, a.cols, y);
        }
    }
}

// --------------------------------------------------------------- backward
// A unit's xh and g = dy w.
__device__ __forceinline__ void parts_of(const float (&dy)[kU], const float (&h)[kU], const float (&w)[kU], float rstd,
                                         float (&g)[kU], float (&xh)[kU]) {
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        xh[i] = h[i] * rstd;
        g[i] = dy[i] * w[i];
    }
}

template <int kType>
__device__ __forceinline__ Raw<kType> grad_unit(const float (&g)[kU], const float (&xh)[kU], float c, float rstd,
                                                bool has_dh, const Raw<kType>& dh) {
    float v[kU], d[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) v[i] = (g[i] - xh[i] * c) * rstd;
    if (has_dh) {
        unpack(dh, d);
#pragma unroll
        for (int i = 0; i < kU; ++i) v[i] += d[i];
    }
    return pack<kType>(v);
}

// As the norm's kernel; each workgroup keeps its part of dweight in
// registers, one row of `part` at the end.  8192 x 1600 bf16 with dh 27.8 us,
// of which 24 without dweight (4.4 TB/s); 4096 x 8192 fp32 82 and 76 (5.3).
template <int kType, int kWaves, int kNS>
__global__ __launch_bounds__(kThreads<kWaves>) void norm8_backward_kernel(NormBackArgs a) {
    constexpr int across = kWaves * kSweep;
    const int c0 = (kWaves == 1 ? threadIdx.x & 63 : threadIdx.x) * kU;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPack<kWaves>;
    const bool has_dh = a.dh != nullptr;
    float dw[kNS][kU], w[kNS][kU];
#pragma unroll
    for (int s = 0; s < kNS; ++s)
#pragma unroll
        for (int i = 0; i < kU; ++i) dw[s][i] = 0.0f;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kPack<kWaves> + (kWaves == 1 ? threadIdx.x >> 6 : 0);
    Raw<kType> ny[kNS], nh[kNS], nd[kNS];
    float nrstd = 0.0f;
    const auto load = [&](int64_t at) {
        if (at >= a.rows) return;
        load_row<kType>(a.dy, at, a.dy_stride, c0, across, a.cols, ny);
        load_row<kType>(a.h, at, a.h_stride, c0, across, a.cols, nh);
        nrstd = a.rstd[at];
    };
    load(row);
    load_weights(a.w, a.w_type, c0, across, a.cols, w);
    for (int turn = 0; row < a.rows; row += step, ++turn) {
        const float rstd = nrstd;
        if (has_dh) load_row<kType>(a.dh, row, a.dh_stride, c0, across, a.cols, nd);
        float g[kNS][kU], xh[kNS][kU], sum = 0.0f;
#pragma unroll
        for (int s = 0; s < kNS; ++s) {
            float dy[kU], h[kU];
            unpack(ny[s], dy);
            unpack(nh[s], h);
            parts_of(dy, h, w[s], rstd, g[s], xh[s]);
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                sum += g[s][i] * xh[s][i];
                dw[s][i] += dy[i] * xh[s][i];
            }
        }
        load(row + step);
        const float c = row_sum<kWaves>(sum, turn) / static_cast<float>(a.cols);
#pragma unroll
        for (int s = 0; s < kNS; ++s) {
            const int at = c0 + s * across;
            if (at < a.cols)
                store_unit(row_of<kType>(a.dx, row, a.dx_stride), at, a.cols,
                           grad_unit<kType>(g[s], xh[s], c, rstd, has_dh, nd[s]));
        }
    }
    if (a.dw == nullptr) return;
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
    if (kWaves == 1) {
        __shared__ float all[4][kNS * kSweep];
#pragma unroll
        for (int s = 0; s < kNS; ++s)
#pragma unroll
            for (int i = 0; i < kU; ++i) all[threadIdx.x >> 6][s * kSweep + c0 + i] = dw[s][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += kThreads<kWaves>)
            part[c] = (all[0][c] + all[1][c]) + (all[2][c] + all[3][c]);
        return;
    }
#pragma unroll
    for (int s = 0; s < kNS; ++s) {
        const int c = c0 + s * across;
        if (c < a.cols) store_unit(reinterpret_cast<char*>(part), c, a.cols, pack<ZERO_TYPE_F32>(dw[s]));
    }
}

// Rows longer than the registers of a workgroup: dy and h read twice, and the
// workgroup's part of dweight summed up in memory (each lane its own columns).
template <int kType>
__global__ __launch_bounds__(kLongWaves * 64) void norm8_backward_long_kernel(NormBackArgs a) {
    constexpr int kStep = kLongWaves * kSweep;
    const int c0 = threadIdx.x * kU;
    const bool has_dh = a.dh != nullptr;
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
        const float rstd = a.rstd[row];
        const char* dy_row = row_of<kType>(a.dy, row, a.dy_stride);
        const char* h_row = row_of<kType>(a.h, row, a.h_stride);
        float sum = 0.0f;
        for (int c = c0; c < a.cols; c += kStep) {
            float dy[kU], h[kU], w[kU], g[kU], xh[kU];
            unpack(load_unit<kType>(dy_row, c, a.cols), dy);
            unpack(load_unit<kType>(h_row, c, a.cols), h);
            load_vector(a.w, a.w_type, c, a.cols, w);
            parts_of(dy, h, w, rstd, g, xh);
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                sum += g[i] * xh[i];
                if (a.dw != nullptr && c + i < a.cols) part[c + i] = (turn == 0 ? 0.0f : part[c + i]) + dy[i] * xh[i];
            }
        }
        const float mean = row_sum<kLongWaves>(sum, turn) / static_cast<float>(a.cols);
        for (int c = c0; c < a.cols; c += kStep) {
            float dy[kU], h[kU], w[kU], g[kU], xh[kU];
            Raw<kType> rd = {};
            unpack(load_unit<kType>(dy_row, c, a.cols), dy);
            unpack(load_unit<kType>(h_row, c, a.cols), h);
            load_vector(a.w, a.w_type, c, a.cols, w);
            if (has_dh) rd = load_unit<kType>(row_of<kType>(a.dh, row, a.dh_stride), c, a.cols);
            parts_of(dy, h, w, rstd, g, xh);
            store_unit(row_of<kType>(a.dx, row, a.dx_stride), c, a.cols,
                       grad_unit<kType>(g, xh, mean, rstd, has_dh, rd));
        }
    }
}

// dweight = the parts' sum, in float64 and a fixed order: 16 columns and 64
// parts at a time to a workgroup, then a wave for each column.
__global__ __launch_bounds__(1024) void norm8_dweight_kernel(const float* part, int groups, int cols, float* dw) {
    __shared__ double s[64][17];
    const int j = threadIdx.x & 15, g0 = threadIdx.x >> 4, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = blockIdx.x * 16 + j;
    double x = 0.0;
    if (c < cols) {
#pragma unroll 4
        for (int g = g0; g < groups; g += 64) x += part[static_cast<int64_t>(g) * cols + c];
    }
    s[g0][j] = x;
    __syncthreads();
    x = row_sum<1>(s[lane][wave], 0);
    if (lane == 0 && blockIdx.x * 16 + wave < static_cast<unsigned>(cols))
        dw[blockIdx.x * 16 + wave] = static_cast<float>(x);
}

// ----------------------------------------------------------------- encode
__device__ __forceinline__ void multiply(float m, const float (&w)[kU], float (&v)[kU]) {
#pragma unroll
    for (int i = 0; i < kU; ++i) v[i] = (v[i] * m) * w[i];
}

template <bool kMul>
__device__ __forceinline__ void multipliers(const EncodeArgs& a, int c, int n, float (&w)[kU]) {
    if (kMul && a.col_mul != nullptr) {
        load_vector(a.col_mul, a.col_type, c, n, w);
    } else {
#pragma unroll
        for (int i = 0; i < kU; ++i) w[i] = 1.0f;
    }
}

// By rows, as it is: a wave takes sweeps of 512 columns (16384 x 8192 bf16: 75
// us, 5.4 TB/s, memory's rate).
template <int kType, bool kMul>
__global__ __launch_bounds__(256) void encode_rows_kernel(EncodeArgs a) {
    const int cols = static_cast<int>(a.cols);
    const int sweeps = (cols + kSweep - 1) / kSweep;
    const int64_t units = a.rows * sweeps;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units;
         u += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t row = u / sweeps;
        const int c = static_cast<int>(u - row * sweeps) * kSweep + (threadIdx.x & 63) * kU;
        float v[kU], w[kU];
        unpack(load_unit<kType>(row_of<kType>(a.x, row, a.x_stride), c, cols), v);
        if (kMul) {
            multipliers<kMul>(a, c, cols, w);
            multiply(a.row_mul == nullptr ? 1.0f : a.row_mul[row], w, v);
        }
        emit(a.codes + row * a.codes_stride, a.scales + row * a.scales_stride, c, cols, v);
    }
}

// 128 x 128 values to a workgroup: lane group g (16 lanes) holds rows 8 g to
// 8 g + 7, each lane 8 columns of them.  Transposed codes go through LDS,
// where a lane's 8 rows of a column are 8 neighbouring bytes.  16384 x 8192
// bf16: both 117 us (4.6 TB/s), transposed alone 91 (4.4), whose stores are runs
// of 128 bytes; 6400 x 1600 fp16 tiles, both: 11 us, launch and latency, and 650
// tiles where registers let 512 onto the card at once.
constexpr int kTurnStride = 144;

// The first `bytes` (less than all) of kWords words, by halves: few stores, at
// any alignment.
template <int kWords>
__device__ __forceinline__ void store_some(uint8_t* to, const uint32_t (&w)[kWords], int bytes) {
    typedef uint32_t w4 __attribute__((aligned(1)));
    typedef uint16_t w2 __attribute__((aligned(1)));
    int at = 0;
    uint32_t x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) x[i] = w[i];
#pragma unroll
    for (int half = kWords / 2; half > 0; half /= 2) {
        if ((bytes & 4 * half) == 0) continue;
#pragma unroll
        for (int i = 0; i < half; ++i) reinterpret_cast<w4*>(to + at)[i] = x[i];
#pragma unroll
        for (int i = 0; i < kWords - half; ++i) x[i] = x[i + half];
        at += 4 * half;
    }
    if ((bytes & 2) != 0) {
        *reinterpret_cast<w2*>(to + at) = static_cast<uint16_t>(x[0]);
        x[0] >>= 16;
        at += 2;
    }
    if ((bytes & 1) != 0) to[at] = static_cast<uint8_t>(x[0]);
}

// kEnds 0: the tile has all its rows and columns (straight code, a third as
// long); 1: it may not, but no unit of 8 columns is cut; 2: one may be.
template <int kType, bool kMul, bool kTiles, int kEnds>
__device__ __forceinline__ void encode_tile(const EncodeArgs& a, int64_t tr, int tc, uint32_t (&top)[4][kB8],
                                            uint8_t* turned) {
    constexpr bool kWhole = kEnds == 0;
    const int cols = static_cast<int>(a.cols);
    const int64_t rows = a.rows;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t r0 = tr * kB8 + rg * 8;
    const int c = tc * kB8 + cg * kU;
    const int n = kWhole ? c + kU : cols;  // columns, as far as this lane can tell
    {
        Raw<kType> raw[8];
        float rm[8], w[kU], v[8][kU];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t row = kWhole || r0 + j < rows ? r0 + j : rows - 1;
            const char* from = row_of<kType>(a.x, row, a.x_stride);
            // (kEnds 1: a unit past the end reads the row's first in its place)
            raw[j] = kEnds == 2 ? load_end<kType>(from, c, n)
                                : load_unit<kType>(from, kWhole || c < n ? c : 0, kWhole ? n : c + kU);
        }
        if (kMul) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                rm[j] = a.row_mul == nullptr ? 1.0f : a.row_mul[kWhole || r0 + j < rows ? r0 + j : rows - 1];
        }
        multipliers<kMul>(a, c, n, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            unpack(raw[j], v[j]);
            if (kMul) multiply(rm[j], w, v[j]);
            if (!kWhole) {  // rows and units past the end stay out of every scale
#pragma unroll
                for (int i = 0; i < kU; ++i) v[j][i] = r0 + j < rows && c < cols ? v[j][i] : 0.0f;
            }
        }
        uint32_t tile_byte = 0;
        if (kTiles) {
            uint32_t big = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) big = max(big, magnitude(v[j]));
            big = max16(big);
            big = max(big, static_cast<uint32_t>(__shfl_xor(big, 16)));
            big = max(big, static_cast<uint32_t>(__shfl_xor(big, 32)));
            if ((threadIdx.x & 63) == 0) top[wave][0] = big;
            __syncthreads();
            tile_byte = scale_byte(max(max(top[0][0], top[1][0]), max(top[2][0], top[3][0])));
            if (threadIdx.x == 0) {
                if (a.codes != nullptr) a.scales[tr * a.scales_stride + tc] = static_cast<uint8_t>(tile_byte);
                if (a.codes_t != nullptr) a.scales_t[tc * a.scales_t_stride + tr] = static_cast<uint8_t>(tile_byte);
            }
        }
        if (a.codes != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t byte = kTiles ? tile_byte : scale_byte(max16(magnitude(v[j])));
                const int64_t row = r0 + j;
                if (!kWhole && row >= rows) continue;
                const uint32_t w[2] = {codes4(v[j][0], v[j][1], v[j][2], v[j][3], byte),
                                       codes4(v[j][4], v[j][5], v[j][6], v[j][7], byte)};
                if (kWhole || (kEnds == 1 ? c < cols : c + kU <= cols))
                    *reinterpret_cast<u32x2*>(a.codes + row * a.codes_stride + c) = u32x2{w[0], w[1]};
                else if (kEnds == 2 && c < cols)
                    store_some(a.codes + row * a.codes_stride + c, w, cols - c);
                if (!kTiles && cg == 0) a.scales[row * a.scales_stride + tc] = static_cast<uint8_t>(byte);
            }
        }
        if (a.codes_t != nullptr) {
            uint32_t big[kU];
            if (!kTiles) {
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    uint32_t x = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) x = max(x, bits_of(v[j][i]) & 0x7FFFFFFFu);
                    x = max(x, static_cast<uint32_t>(__shfl_xor(x, 16)));
                    x = max(x, static_cast<uint32_t>(__shfl_xor(x, 32)));
                    if ((threadIdx.x & 48) == 0) top[wave][cg * kU + i] = x;
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kU; ++i) {
                    const int k = cg * kU + i;
                    big[i] = max(max(top[0][k], top[1][k]), max(top[2][k], top[3][k]));
                }
            }
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const uint32_t byte = kTiles ? tile_byte : scale_byte(big[i]);
                u32x2 x;
                x[0] = codes4(v[0][i], v[1][i], v[2][i], v[3][i], byte);
                x[1] = codes4(v[4][i], v[5][i], v[6][i], v[7][i], byte);
                *reinterpret_cast<u32x2*>(turned + (cg * kU + i) * kTurnStride + rg * 8) = x;
                if (!kTiles && rg == 0 && (kWhole || c + i < cols))
                    a.scales_t[static_cast<int64_t>(c + i) * a.scales_t_stride + tr] = static_cast<uint8_t>(byte);
            }
            __syncthreads();
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int k = p * 32 + (threadIdx.x >> 3), part = (threadIdx.x & 7) * 16;
                const int64_t col = static_cast<int64_t>(tc) * kB8 + k, r = tr * kB8 + part;
                if (!kWhole && (col >= cols || r >= rows)) continue;
                const u32x4 x = *reinterpret_cast<const u32x4*>(turned + k * kTurnStride + part);
                uint8_t* to = a.codes_t + col * a.codes_t_stride + r;
                if (kWhole || r + 16 <= rows) {
                    *reinterpret_cast<u32x4*>(to) = x;
                } else {
                    const uint32_t piece[4] = {x[0], x[1], x[2], x[3]};
                    store_some(to, piece, static_cast<int>(rows - r));
                }
            }
        }
        __syncthreads();
    }
}

template <int kType, bool kMul, bool kTiles>
__global__ __launch_bounds__(256) void encode_tile_kernel(EncodeArgs a) {
    __shared__ uint32_t top[4][kB8];
    __shared__ __attribute__((aligned(16))) uint8_t turned[kB8 * kTurnStride];
    const int across = static_cast<int>((a.cols + kB8 - 1) / kB8);
    const int64_t tiles = (a.rows + kB8 - 1) / kB8 * across;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t tr = tile / across;
        const int tc = static_cast<int>(tile - tr * across);
        if ((tr + 1) * kB8 <= a.rows && (tc + 1) * static_cast<int64_t>(kB8) <= a.cols)
            encode_tile<kType, kMul, kTiles, 0>(a, tr, tc, top, turned);
        else if (a.cols % kU == 0)
            encode_tile<kType, kMul, kTiles, 1>(a, tr, tc, top, turned);
        else
            encode_tile<kType, kMul, kTiles, 2>(a, tr, tc, top, turned);
    }
}

// --------------------------------------------------------------- launchers
// Grids are capped far below the runtime's limit of 2^32 lanes; the kernels
// take what is left in turn.
constexpr int64_t kMaxGrid = 1 << 20;

unsigned grid_of(int64_t units) { return static_cast<unsigned>(units < kMaxGrid ? units : kMaxGrid); }

int finish() {
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return ZERO_OK;
    zdp::set_last_hip_error(static_cast<int>(e));
    return ZERO_EHIP;
}

// Calls f with the type as a constant.
template <typename F>
void with_type(int type, F f) {
    if (type == ZERO_TYPE_F32)
        f(std::integral_constant<int, ZERO_TYPE_F32>());
    else if (type == ZERO_TYPE_F16)
        f(std::integral_constant<int, ZERO_TYPE_F16>());
    else
        f(std::integral_constant<int, ZERO_TYPE_BF16>());
}

// Calls f with the waves and the units a lane that hold a row of n columns:
// (0, 0) for a row too long for registers.  At most eight waves, two
// workgroups of which fit a CU (4099 x 12289 fp16: 46 us in eight waves of
// four units, 70 in nine of three, which fit once).  Rows of 1025 to 2048 in
// bf16 are faster in two waves forward (8192 x 1600 with a residual: 19.9 us; in
// one 25.1, in four 22.0) and in one backward (27.6 us; 34.1 in two, 45.7 in
// four), at 1032, 1280, 1536, 1792 and 2048 columns too (four waves within 1 % at
// 1536 and 2048 forward).  In fp32 that choice is not the fastest: 8192 x 1600
// takes 38.1 us forward (36.1 in four) and 53.7 backward (47.9 in two).
template <int kType, bool kBack, typename F>
void with_row_shape(int n, F f) {
    using std::integral_constant;
    constexpr integral_constant<int, 0> k0{};
    constexpr integral_constant<int, 1> k1{};
    constexpr integral_constant<int, 2> k2{};
    constexpr integral_constant<int, 3> k3{};
    constexpr integral_constant<int, 4> k4{};
    constexpr integral_constant<int, 8> k8{};
    if (n <= kSweep)
        f(k1, k1);
    else if (n <= 2 * kSweep)
        f(k1, k2);
    else if (n <= 4 * kSweep)
        f(integral_constant<int, kBack ? 1 : 2>(), integral_constant<int, kBack ? 4 : 2>());
    else if (n <= 8 * kSweep)
        f(k4, k2);
    else if (n <= 12 * kSweep)
        f(k4, k3);
    else if (n <= 16 * kSweep)
        f(k8, k2);
    else if (n <= 24 * kSweep)
        f(k8, k3);
    else if (n <= 32 * kSweep && !(kBack && kType == ZERO_TYPE_F32))
        f(k8, integral_constant<int, kBack && kType == ZERO_TYPE_F32 ? 3 : 4>());  // (backward in fp32 does not fit)
    else
        f(k0, k0);
}

// Workgroups of the norm's kernels: enough rows under way to cover memory's
// latency, few enough that each goes on to a next row.
constexpr int kCus = 256;  // of an MI355X; the choice costs time alone
template <int kWaves, int kNS>
constexpr int64_t kNormGroups = kCus * (kNS >= 3 ? 16 : 24) / (kWaves * kPack<kWaves>);
template <int kWaves>
constexpr int64_t kBackGroups = kCus * 8 / (kWaves * kPack<kWaves>);

template <int kWaves>
int64_t groups_of(int64_t rows, int64_t cap) {
    const int64_t most = (rows + kPack<kWaves> - 1) / kPack<kWaves>;
    return most < cap ? most : cap;
}

}  // namespace

namespace zdp {

int launch_norm8(const NormArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(a.type, [&](auto type) {
        constexpr int kType = decltype(type)::value;
        with_row_shape<kType, false>(a.cols, [&](auto waves, auto units) {
            constexpr int kWaves = decltype(waves)::value, kNS = decltype(units)::value;
            if constexpr (kWaves == 0) {
                const unsigned grid = grid_of(a.rows);
                if (a.r != nullptr)
                    norm8_long_kernel<kType, true><<<grid, kLongWaves * 64, 0, s>>>(a);
                else
                    norm8_long_kernel<kType, false><<<grid, kLongWaves * 64, 0, s>>>(a);
            } else {
                const unsigned grid = static_cast<unsigned>(groups_of<kWaves>(a.rows, kNormGroups<kWaves, kNS>));
                if (a.r != nullptr)
                    norm8_kernel<kType, true, kWaves, kNS><<<grid, kThreads<kWaves>, 0, s>>>(a);
                else
                    norm8_kernel<kType, false, kWaves, kNS><<<grid, kThreads<kWaves>, 0, s>>>(a);
            }
        });
    });
    return finish();
}

int launch_norm8_backward(const NormBackArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    int64_t groups = norm_back_groups(a.rows, a.cols);
    if (a.rows > 0) {
        with_type(a.type, [&](auto type) {
            constexpr int kType = decltype(type)::value;
            with_row_shape<kType, true>(a.cols, [&](auto waves, auto units) {
                constexpr int kWaves = decltype(waves)::value, kNS = decltype(units)::value;
                if constexpr (kWaves == 0) {
                    norm8_backward_long_kernel<kType><<<static_cast<unsigned>(groups), kLongWaves * 64, 0, s>>>(a);
                } else {
                    const int64_t most = groups_of<kWaves>(a.rows, kBackGroups<kWaves>);
                    groups = groups < most ? groups : most;
                    norm8_backward_kernel<kType, kWaves, kNS>
                        <<<static_cast<unsigned>(groups), kThreads<kWaves>, 0, s>>>(a);
                }
            });
        });
        const int rc = finish();
        if (rc != ZERO_OK) return rc;
    }
    if (a.dw == nullptr) return ZERO_OK;
    norm8_dweight_kernel<<<static_cast<unsigned>((a.cols + 15) / 16), 1024, 0, s>>>(
        a.part, a.rows > 0 ? static_cast<int>(groups) : 0, a.cols, a.dw);
    return finish();
}

int launch_block8_encode(const EncodeArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool mul = a.row_mul != nullptr || a.col_mul != nullptr;
    with_type(a.type, [&](auto type) {
        constexpr int kType = decltype(type)::value;
        if (!a.tiles && a.codes_t == nullptr) {
            const unsigned grid = grid_of((a.rows * ((a.cols + kSweep - 1) / kSweep) + 3) / 4);
            if (mul)
                encode_rows_kernel<kType, true><<<grid, 256, 0, s>>>(a);
            else
                encode_rows_kernel<kType, false><<<grid, 256, 0, s>>>(a);
            return;
        }
        const unsigned grid = grid_of(b8_blocks(a.rows) * b8_blocks(a.cols));
        if (a.tiles) {
            if (mul)
                encode_tile_kernel<kType, true, true><<<grid, 256, 0, s>>>(a);
            else
                encode_tile_kernel<kType, false, true><<<grid, 256, 0, s>>>(a);
        } else {
            if (mul)
                encode_tile_kernel<kType, true, false><<<grid, 256, 0, s>>>(a);
            else
                encode_tile_kernel<kType, false, false><<<grid, 256, 0, s>>>(a);
        }
    });
    return finish();
}

}  // namespace zdp
