// Device side of the tensor-list operators for CDNA4 (gfx950): the optimizer
// step of parameters that are separate tensors.
//
//   norm     *sumsq = sum over the list of g^2, g = raw * (1/L) (float64, fixed
//            order); *overflow = the sum is inf or NaN
//   adam     the Adam/AdamW sequence of the fused step, in place, g = raw *
//            (coef / L):
//              m' = b1*m + (1-b1)*g          v' = b2*v + (1-b2)*(g*g)
//              d  = sqrt(v') * (1/sqrt(1-b2^t)) + eps
//              p' = p*(1-lr*wd) - (lr/(1-b1^t)) * (m'/d)
//            fp32 states: one IEEE float64 operation at a time, rounded once
//            to fp32.  8-bit states: m' and v' as above, rounded to fp32; r =
//            sqrt(v'); m' and r encoded as below, and the update in fp32:
//              p' = p - (lr*wd*p + lr/(1-b1^t) * m' / (r/sqrt(1-b2^t) + eps))
//            (the states carry 4 significant bits, so the update term needs
//            no more than fp32's 24; the codes come from the float64 sums,
//            which puts a value beside a border on the right side)
//   encode   blocks of 32 fp32 values: scale 2^(e-127) with the smallest e >= 1
//            that keeps the largest magnitude within 448 scales, each value
//            over the scale in e4m3 (nearest, or stochastic: the random word's
//            top 20 bits, for a root its low 16 with four zeros behind, added
//            to the 20 bits that are cut off), at most 240 at scale 2^120
//   decode   value = code * scale, squared for a root
//
// Everything here is a stream over memory.  No two workgroups write the same
// bytes, and every sum has a fixed order, so results repeat bit for bit.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/zero_dp.h"
#include "zero_dp_tensors.h"

#pragma clang fp contract(off)

namespace {

using zdp::ChunkRef;
using zdp::kBlock;
using zdp::kChunk;
using zdp::kWaves;
using zdp::ListArgs;
using zdp::Partials;
using zdp::TensorDesc;
using zdp::TensorStepArgs;

constexpr uint32_t kSubTickets = zdp::kSubTickets;

// Elements per lane per row of a chunk: a 16-byte fp32 vector, an 8-byte
// 16-bit vector, a 4-byte vector of codes.  Tensors need only their
// elements' own alignment; the hardware takes vector accesses at any
// address, so the vector types below claim no more.
constexpr int kV = 4;
constexpr int kRow = kBlock * kV;
constexpr int kRows = kChunk / kRow;
typedef float fvec __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t hvec __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t cvec __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Global and constant address spaces: a list's pointers come out of memory,
// where the compiler cannot tell what they point to, and a flat access
// would wait on two counters; the table itself never changes under a launch,
// so it is read through the scalar cache.
#define ZDP_GLOBAL __attribute__((address_space(1)))
#define ZDP_CONST __attribute__((address_space(4)))
typedef ZDP_GLOBAL const float* gcf32;
typedef ZDP_GLOBAL float* gf32;
typedef ZDP_GLOBAL const uint16_t* gcu16;
typedef ZDP_GLOBAL uint16_t* gu16;
typedef ZDP_GLOBAL const uint8_t* gcu8;
typedef ZDP_GLOBAL uint8_t* gu8;

// Streaming (non-temporal) accesses, unless a load is meant to stay in cache.
template <bool kNt = true, typename T>
__device__ __forceinline__ T ldg(ZDP_GLOBAL const T* p) {
    if (kNt) return __builtin_nontemporal_load(p);
    return *p;
}

template <typename T>
__device__ __forceinline__ void stg(ZDP_GLOBAL T* p, const T& v) {
    __builtin_nontemporal_store(v, p);
}

// ------------------------------------------------------------- reductions
// Sum over the workgroup in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double s[kWaves];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        x = s[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) x += s[w];
    }
    __syncthreads();
    return x;
}

// Largest value over the 8 lanes whose vectors make up one block of 32.
__device__ __forceinline__ uint32_t max8(uint32_t x) {
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true)));   // lane ^ 1
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true)));   // lane ^ 2
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x141, 0xF, 0xF, true)));  // other half of 8
    return x;
}

// Draws a ticket for the workgroup (one thread of it): true for the last of
// the grid, which leaves the counters at zero.  Draws on one address follow
// each other at about 10 ns, so the workgroups draw from 32 counters, and
// the last of each draws from the one behind them (755 workgroups: 15.9 us
// of kernel on one counter, 12.5 on 33).  The order is relaxed: what has
// to be seen by the last workgroup has to be performed before the draw.
__device__ __forceinline__ bool last_to_draw(uint32_t* ticket) {
    const uint32_t s = blockIdx.x % kSubTickets;
    const uint32_t members = (gridDim.x - s + kSubTickets - 1) / kSubTickets;
    uint32_t* const sub = ticket + (zdp::kWsSubTickets - zdp::kWsTicket) / 4 + s;
    if (__hip_atomic_fetch_add(sub, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != members - 1) return false;
    __hip_atomic_store(sub, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t subs = gridDim.x < kSubTickets ? gridDim.x : kSubTickets;
    if (__hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != subs - 1) return false;
    __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// ------------------------------------------------------------- random bits
// A 32-bit mixing function: two odd multiplications between folds.  The
// multipliers are the best of 60 random pairs by how evenly one input bit
// flips every output bit (worst probability 0.494 to 0.506).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x, uint32_t k) {
    x = (x ^ (x >> 16)) * 0xACE5F457u;
    x = (x ^ (x >> 15) ^ k) * 0x7B639EB3u;
    return x ^ (x >> 16);
}

struct RandomKey {
    uint32_t k1, k2;
};

__host__ __device__ __forceinline__ RandomKey random_key(uint64_t seed, uint32_t step) {
    const uint32_t k1 =
        mix(mix(mix(step, 0) ^ static_cast<uint32_t>(seed >> 32), 0) ^ static_cast<uint32_t>(seed), 0);
    return RandomKey{k1, mix(~k1, 0)};
}

// The random word of counter c (the low 32 bits of flat_off + index).
__device__ __forceinline__ uint32_t random_word(const RandomKey& k, uint32_t c) { return mix(c ^ k.k1, k.k2); }

// ------------------------------------------------------------ 8-bit blocks
// Scale byte of a block whose largest magnitude has the bits `big`: the
// exponent, one more where the mantissa passes 448 = 1.75 * 2^8.  255 for a
// block that holds an inf or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t big) {
    int e = static_cast<int>((big + 0x1FFFFFu) >> 23) - 8;
    e = e < 1 ? 1 : e;
    return big >= 0x7F800000u ? 255u : static_cast<uint32_t>(e);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    const uint32_t bits = byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23;
    return __builtin_bit_cast(float, bits);
}

__device__ __forceinline__ fvec decode4(uint32_t codes, float scale) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
    fvec r;
    r[0] = a[0] * scale;
    r[1] = a[1] * scale;
    r[2] = b[0] * scale;
    r[3] = b[1] * scale;
    return r;
}

__device__ __forceinline__ uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float float_of(uint32_t x) { return __builtin_bit_cast(float, x); }

// Correctly rounded square roots of four fp32 values.  The hardware's root s
// is off by at most one step u; x lies above the midpoint (s - u/2)^2 =
// s (s - u) + u^2/4 exactly where x > s (s - u), since both sides of that are
// multiples of a unit larger than u^2/4, and likewise at s + u/2; one fused
// multiply-add gives the sign.  Nothing underflows in it from 2^-96 up (and
// at 0); a wave that holds a smaller value takes the library's root, which
// scales first.  (The compiler's own expansion of a correctly rounded root
// takes the same correction, after a scaling that few values here need.)
__device__ __forceinline__ void roots4(fvec& x) {
    uint32_t least = 0xFFFFFFFFu;
#pragma unroll
    for (int e = 0; e < kV; ++e) least = min(least, bits_of(x[e]) - 1u);
    if (__any(least < bits_of(0x1p-96f) - 1u)) {
#pragma unroll
        for (int e = 0; e < kV; ++e) x[e] = __builtin_sqrtf(x[e]);
        return;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        const float s = __builtin_amdgcn_sqrtf(x[e]);
        const float down = float_of(bits_of(s) - 1u), up = float_of(bits_of(s) + 1u);
        const bool lower = __builtin_fmaf(-down, s, x[e]) <= 0.0f, upper = __builtin_fmaf(-up, s, x[e]) > 0.0f;
        x[e] = upper ? up : lower ? down : s;
    }
}

// Roots of the variances v, given in float64: those of their fp32 values, and
// past fp32's range those of v itself, whose roots fp32 still holds (one
// huge gradient would else turn its block, and 32 weights, into NaN).
// wide: some lane of the wave holds such a variance.
__device__ __forceinline__ fvec wide_roots4(const double (&v)[kV], bool& wide) {
    fvec x;
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        x[e] = static_cast<float>(v[e]);
        most = max(most, bits_of(x[e]));
    }
    wide = __any(most >= 0x7F800000u);
    if (wide) {
#pragma unroll
        for (int e = 0; e < kV; ++e)
            x[e] = bits_of(x[e]) >= 0x7F800000u ? static_cast<float>(__builtin_sqrt(v[e])) : __builtin_sqrtf(x[e]);
        return x;
    }
    roots4(x);
    return x;
}

// The four codes of x under their block's scale byte.  The conversions take
// the scale as an operand.  Their stochastic form adds the top 20 bits of
// its random operand to the mantissa's last 20 bits and cuts them off,
// counted in the target's subnormal steps below 2^-6.
template <bool kStoch>
__device__ __forceinline__ uint32_t codes4(const fvec& x, float scale, const uint32_t (&bits)[kV]) {
    if (kStoch) {
        int c = 0;
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[0], bits[0], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[1], bits[1], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[2], bits[2], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, x[3], bits[3], scale, 3);
        return static_cast<uint32_t>(c);
    }
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 c = {0, 0};
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[0], x[1], scale, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[2], x[3], scale, true);
    return __builtin_bit_cast(uint32_t, c);
}

// Encodes a lane's four elements of a block (8 lanes, all of them here, with
// zeros for elements that are not).  kRoot: x are roots.
template <bool kRoot, bool kStoch>
__device__ __forceinline__ uint32_t encode4(const fvec& x, const uint32_t (&word)[kV], uint32_t& byte) {
    uint32_t big = 0;
    uint32_t bits[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        big = max(big, bits_of(x[e]) & 0x7FFFFFFFu);
        bits[e] = kRoot ? word[e] << 16 : word[e];
    }
    byte = scale_byte(max8(big));
    // the largest scale's codes end at 240: 256 * 2^120 would read as inf
    constexpr float most = 0x1.Ep127f;
    // a positive root keeps at least the smallest code: rounded to zero it
    // would turn its weight's next update into m/eps
    const float least = __builtin_bit_cast(float, byte << 23) * 0x1p-9f;
    fvec y;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        if (kRoot)
            y[e] = x[e] > 0.0f ? __builtin_amdgcn_fmed3f(x[e], least, most) : static_cast<float>(x[e]);
        else
            y[e] = __builtin_amdgcn_fmed3f(x[e], -most, most);
    }
    const uint32_t c = codes4<kStoch>(y, __builtin_bit_cast(float, byte << 23), bits);
    return byte == 255u ? 0x7F7F7F7Fu : c;
}

// ------------------------------------------------------- loads and stores
// A lane's kV elements of an array at element j of n; a row that is not
// `full` is loaded and stored element by element, with zeros for the
// elements past n (a lane at the end of a tensor).
template <bool kFull, bool kNt = true>
__device__ __forceinline__ fvec load_f32(gcf32 p, int j, int n) {
    if (kFull) return ldg<kNt>(reinterpret_cast<ZDP_GLOBAL const fvec*>(p + j));
    fvec x;
#pragma unroll
    for (int e = 0; e < kV; ++e) x[e] = j + e < n ? p[j + e] : 0.0f;
    return x;
}

template <bool kFull, bool kNt = true>
__device__ __forceinline__ hvec load_16(gcu16 p, int j, int n) {
    if (kFull) return ldg<kNt>(reinterpret_cast<ZDP_GLOBAL const hvec*>(p + j));
    hvec x = {0, 0};
#pragma unroll
    for (int e = 0; e < kV; ++e)
        if (j + e < n) x[e >> 1] |= static_cast<uint32_t>(p[j + e]) << (16 * (e & 1));
    return x;
}

template <bool kFull>
__device__ __forceinline__ uint32_t load_8(gcu8 p, int j, int n) {
    if (kFull) return ldg(reinterpret_cast<ZDP_GLOBAL const cvec*>(p + j));
    uint32_t x = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e)
        if (j + e < n) x |= static_cast<uint32_t>(p[j + e]) << (8 * e);
    return x;
}

template <bool kFull>
__device__ __forceinline__ void store_f32(gf32 p, int j, int n, const fvec& x) {
    if (kFull) {
        stg(reinterpret_cast<ZDP_GLOBAL fvec*>(p + j), x);
        return;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e)
        if (j + e < n) p[j + e] = x[e];
}

template <bool kFull>
__device__ __forceinline__ void store_16(gu16 p, int j, int n, const hvec& x) {
    if (kFull) {
        stg(reinterpret_cast<ZDP_GLOBAL hvec*>(p + j), x);
        return;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e)
        if (j + e < n) p[j + e] = static_cast<uint16_t>(x[e >> 1] >> (16 * (e & 1)));
}

template <bool kFull>
__device__ __forceinline__ void store_8(gu8 p, int j, int n, uint32_t x) {
    if (kFull) {
        stg(reinterpret_cast<ZDP_GLOBAL cvec*>(p + j), static_cast<cvec>(x));
        return;
    }
#pragma unroll
    for (int e = 0; e < kV; ++e)
        if (j + e < n) p[j + e] = static_cast<uint8_t>(x >> (8 * e));
}

// The gradient's kV raw values.
template <int kType>
struct GradVec {
    hvec h;
    __device__ __forceinline__ void zero() { h = hvec{0, 0}; }
    __device__ __forceinline__ double at(int e) const {
        const uint32_t w = h[e >> 1];
        if (kType == ZERO_TYPE_BF16)
            return static_cast<double>(__builtin_bit_cast(float, (e & 1) ? w & 0xFFFF0000u : w << 16));
        const f16x2 v = __builtin_bit_cast(f16x2, w);
        return static_cast<double>(static_cast<float>(v[e & 1]));
    }
    template <bool kFull, bool kNt = true>
    __device__ __forceinline__ void load(gcu8 p, int j, int n) {
        h = load_16<kFull, kNt>(reinterpret_cast<gcu16>(p), j, n);
    }
};
template <>
struct GradVec<ZERO_TYPE_F32> {
    fvec f;
    __device__ __forceinline__ void zero() { f = fvec{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ double at(int e) const { return static_cast<double>(static_cast<float>(f[e])); }
    template <bool kFull, bool kNt = true>
    __device__ __forceinline__ void load(gcu8 p, int j, int n) {
        f = load_f32<kFull, kNt>(reinterpret_cast<gcf32>(p), j, n);
    }
};

template <int kType>
constexpr int grad_size() {
    return kType == ZERO_TYPE_F32 ? 4 : 2;
}

template <int kType>
__device__ __forceinline__ hvec pack_param(const fvec& x) {
    hvec h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (kType == ZERO_TYPE_BF16) {
            const bf16x2 b = {static_cast<__bf16>(x[2 * i]), static_cast<__bf16>(x[2 * i + 1])};
            h[i] = __builtin_bit_cast(uint32_t, b);
        } else {
            const f16x2 b = {static_cast<_Float16>(x[2 * i]), static_cast<_Float16>(x[2 * i + 1])};
            h[i] = __builtin_bit_cast(uint32_t, b);
        }
    }
    return h;
}

// A chunk's tensor and its first element there.
struct Place {
    ZDP_CONST const TensorDesc* desc;
    int64_t base;
    __device__ __forceinline__ int count() const {
        const int64_t rest = desc->n - base;
        return static_cast<int>(rest < kChunk ? rest : kChunk);
    }
    // The chunk's first element of an array of `size` bytes an element.
    template <typename T>
    __device__ __forceinline__ gu8 bytes(T* p, int size) const {
        return (gu8)(uintptr_t)p + base * size;
    }
};

__device__ __forceinline__ Place place_of(const ListArgs& list, int64_t c) {
    ZDP_CONST const ChunkRef* refs = (ZDP_CONST const ChunkRef*)(uintptr_t)list.chunks;
    ZDP_CONST const TensorDesc* desc = (ZDP_CONST const TensorDesc*)(uintptr_t)list.desc;
    return Place{desc + refs[c].tensor, static_cast<int64_t>(refs[c].chunk) * kChunk};
}

// ------------------------------------------------------------------- norm
template <int kGrad, bool kNt>
__device__ __forceinline__ void load_grads(GradVec<kGrad> (&v)[kRows], gcu8 g, int n) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int j = k * kRow + static_cast<int>(threadIdx.x) * kV;
        v[k].zero();
        if (j + kV <= n)
            v[k].template load<true, kNt>(g, j, n);
        else if (j < n)
            v[k].template load<false>(g, j, n);
    }
}

// The list is walked from its end, and its first kKeep bytes of gradients
// are read with ordinary loads, so that the step that follows finds them in
// the 256 MB Infinity Cache: for GPT-2 small the norm takes 50 us instead of
// 44, and norm and step together 624 instead of 650 (32-bit states) and 400
// instead of 424 (8-bit); the GPT-2 XL norm 453 instead of 448.
constexpr int64_t kKeep = 192ll << 20;

// Sum of squares of a list.  Bound by HBM reads: one load, two conversions and
// a fused multiply-add an element.  A chunk at a time per workgroup, its
// rows' loads issued together (1.56e9 bf16 gradients: 453 us, 6.9 TB/s;
// 1.2e8 fp16: 49 us, 5.1 TB/s; 1536 fp32: 4.3 us of kernel).
template <int kGrad>
__global__ void __launch_bounds__(kBlock) tensors_norm_kernel(ListArgs list, double inv_scale,
                                                              const zero_step_ctl* dyn, int32_t* overflow,
                                                              double* sumsq, Partials ws) {
    double sq = 0.0;
    for (int64_t i = blockIdx.x; i < list.n_chunks; i += gridDim.x) {
        const int64_t c = list.n_chunks - 1 - i;
        const Place at = place_of(list, c);
        const gcu8 g = at.bytes(at.desc->g, grad_size<kGrad>());
        GradVec<kGrad> v[kRows];
        if (c < kKeep / (kChunk * grad_size<kGrad>()))
            load_grads<kGrad, false>(v, g, at.count());
        else
            load_grads<kGrad, true>(v, g, at.count());
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const double x = v[k].at(e);
                sq = __builtin_fma(x, x, sq);
            }
        }
    }
    // the last workgroup sums the workgroups' parts in a fixed order
    __shared__ int s_last;
    sq = block_sum(sq);
    // (an agent-scope release would write back the XCD's whole L2, once per
    // workgroup, 80 us a launch of 2048: the part goes out by an exchange
    // instead, whose returned value says that it has been performed before
    // the ticket is drawn)
    uint64_t* const parts = reinterpret_cast<uint64_t*>(ws.sq);
    if (threadIdx.x == 0) {
        uint64_t done = __hip_atomic_exchange(parts + blockIdx.x, __builtin_bit_cast(uint64_t, sq), __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" : "+v"(done) : : "memory");
        s_last = last_to_draw(ws.ticket);
    }
    __syncthreads();
    if (!s_last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kBlock)
        t += __builtin_bit_cast(double, __hip_atomic_load(parts + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    t = block_sum(t);
    if (threadIdx.x == 0) {
        // any inf or NaN among the gradients, or a loss scale without a
        // finite reciprocal, leaves the sum inf or NaN
        const double inv = dyn != nullptr ? 1.0 / dyn->loss_scale : inv_scale;
        const double total = t * inv * inv;
        *sumsq = total;
        *overflow = __builtin_isfinite(total) ? 0 : 1;
    }
}

// ------------------------------------------------------------------- adam
// Scalars of the step taken, t = committed + 1.
struct AdamScalars {
    double b1, b2, omb1, omb2, ss, isb, dcy, eps, factor;
    float ssf, isbf, lrwdf, epsf;
};

__device__ __forceinline__ double clip_coef(const TensorStepArgs& a) {
    if (!(a.max_norm > 0.0)) return 1.0;
    const double r = a.max_norm / (__builtin_sqrt(*a.sumsq) + 1e-6);
    return r < 1.0 ? r : 1.0;
}

__device__ __forceinline__ AdamScalars step_scalars(const TensorStepArgs& a) {
    const zero_step_ctl* ctl = a.ctl;
    AdamScalars c;
    c.b1 = a.b1;
    c.b2 = a.b2;
    c.omb1 = 1.0 - a.b1;
    c.omb2 = 1.0 - a.b2;
    c.ss = a.lr / (1.0 - ctl->beta1_pow * a.b1);
    c.isb = 1.0 / __builtin_sqrt(1.0 - ctl->beta2_pow * a.b2);
    c.dcy = 1.0 - a.lr * a.wd;
    c.eps = a.eps;
    c.ssf = static_cast<float>(c.ss);
    c.isbf = static_cast<float>(c.isb);
    c.lrwdf = static_cast<float>(a.lr * a.wd);
    c.epsf = __builtin_fmaxf(static_cast<float>(a.eps), 0x1p-126f);
    c.factor = clip_coef(a) * (a.interval > 0 ? 1.0 / ctl->loss_scale : a.inv_scale);
    return c;
}

// Records the step, or the skip, and advances the dynamic loss scale.
__device__ __forceinline__ void commit(const TensorStepArgs& a, bool skip) {
    zero_step_ctl* w = a.ctl;
    w->overflow = skip ? 1 : 0;
    if (a.sumsq != nullptr) w->sumsq = *a.sumsq;
    if (!skip) {
        w->clip_coef = clip_coef(a);
        w->t = w->t + 1;
        w->beta1_pow = w->beta1_pow * a.b1;
        w->beta2_pow = w->beta2_pow * a.b2;
    } else {
        w->skipped = w->skipped + 1;
    }
    if (a.interval > 0) {
        if (skip) {
            w->loss_scale = w->loss_scale * a.backoff;
            w->good_steps = 0;
        } else {
            int g = w->good_steps + 1;
            if (g == a.interval) {
                // a growth that overflows keeps the scale
                const double grown = w->loss_scale * a.growth;
                if (__builtin_isfinite(grown)) w->loss_scale = grown;
                g = 0;
            }
            w->good_steps = g;
        }
    }
}

__device__ __forceinline__ void adam1(const AdamScalars& c, double g, float p, float m, float v, float& po, float& mo,
                                      float& vo) {
    const double m1 = (c.b1 * static_cast<double>(m)) + (c.omb1 * g);
    const double v1 = (c.b2 * static_cast<double>(v)) + (c.omb2 * (g * g));
    const double d = (__builtin_sqrt(v1) * c.isb) + c.eps;
    const double q = m1 / d;
    const double p1 = (static_cast<double>(p) * c.dcy) - (c.ss * q);
    mo = static_cast<float>(m1);
    vo = static_cast<float>(v1);
    po = static_cast<float>(p1);
}

// One chunk's arrays.
struct Chunk {
    gu8 g, p, w, m, v, ms, vs;
    int n;
    uint32_t counter;
};

template <int kGrad, bool kMx>
__device__ __forceinline__ Chunk chunk_at(const ListArgs& list, int64_t c) {
    const Place at = place_of(list, c);
    ZDP_CONST const TensorDesc* d = at.desc;
    Chunk k;
    k.g = at.bytes(d->g, grad_size<kGrad>());
    k.p = at.bytes(d->p, 4);
    k.w = at.bytes(d->w, 2);
    k.m = at.bytes(d->m, kMx ? 1 : 4);
    k.v = at.bytes(d->v, kMx ? 1 : 4);
    k.ms = (gu8)(uintptr_t)d->ms + at.base / zdp::kMxBlock;
    k.vs = (gu8)(uintptr_t)d->vs + at.base / zdp::kMxBlock;
    k.n = at.count();
    k.counter = static_cast<uint32_t>(d->flat_off) + static_cast<uint32_t>(at.base);
    return k;
}

// A lane's part of one row.
template <int kGrad, bool kMx>
struct Row {
    GradVec<kGrad> g;
    fvec p, m, v;            // 32-bit states
    uint32_t mc, vc, mb, vb;  // 8-bit states: codes and scale bytes

    template <bool kFull>
    __device__ __forceinline__ void load_part(const Chunk& k, int j) {
        g.template load<kFull>(k.g, j, k.n);
        p = load_f32<kFull>(reinterpret_cast<gcf32>(k.p), j, k.n);
        if (kMx) {
            mc = load_8<kFull>(k.m, j, k.n);
            vc = load_8<kFull>(k.v, j, k.n);
            mb = k.ms[j / zdp::kMxBlock];
            vb = k.vs[j / zdp::kMxBlock];
        } else {
            m = load_f32<kFull>(reinterpret_cast<gcf32>(k.m), j, k.n);
            v = load_f32<kFull>(reinterpret_cast<gcf32>(k.v), j, k.n);
        }
    }

    // kFull: the row lies inside the chunk; else a lane that is past the
    // end has zeros (and scale bytes of a block of zeros).
    template <bool kFull>
    __device__ __forceinline__ void load(const Chunk& k, int j) {
        if (kFull) {
            load_part<true>(k, j);
            return;
        }
        g.zero();
        p = m = v = fvec{0.0f, 0.0f, 0.0f, 0.0f};
        mc = vc = 0;
        mb = vb = 1;
        if (j + kV <= k.n)
            load_part<true>(k, j);
        else if (j < k.n)
            load_part<false>(k, j);
    }

    template <bool kFull, int kParam>
    __device__ __forceinline__ void store_part(const Chunk& k, int j, const fvec& po, const fvec& mo, const fvec& vo,
                                               uint32_t m4, uint32_t v4) {
        if (kMx) {
            store_8<kFull>(k.m, j, k.n, m4);
            store_8<kFull>(k.v, j, k.n, v4);
        } else {
            store_f32<kFull>(reinterpret_cast<gf32>(k.m), j, k.n, mo);
            store_f32<kFull>(reinterpret_cast<gf32>(k.v), j, k.n, vo);
        }
        store_f32<kFull>(reinterpret_cast<gf32>(k.p), j, k.n, po);
        if (kParam != ZERO_TYPE_NONE) store_16<kFull>(reinterpret_cast<gu16>(k.w), j, k.n, pack_param<kParam>(po));
    }

    template <bool kFull, int kParam, bool kStoch>
    __device__ __forceinline__ void finish(const Chunk& k, int j, const AdamScalars& c, const RandomKey& key) {
        fvec po, mo, vo;
        uint32_t m4 = 0, v4 = 0;
        if (kMx) {
            m = decode4(mc, scale_value(mb));
            v = decode4(vc, scale_value(vb));  // roots: four significant bits, so their squares are exact
            double v1[kV];
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const double g1 = g.at(e) * c.factor;
                const double m1 = (c.b1 * static_cast<double>(m[e])) + (c.omb1 * g1);
                const double r = static_cast<double>(v[e]);
                v1[e] = (c.b2 * (r * r)) + (c.omb2 * (g1 * g1));
                mo[e] = static_cast<float>(m1);
            }
            bool wide;
            vo = wide_roots4(v1, wide);
            uint32_t word[kV] = {0, 0, 0, 0};
            if (kStoch) {
#pragma unroll
                for (int e = 0; e < kV; ++e) word[e] = random_word(key, k.counter + static_cast<uint32_t>(j + e));
            }
            uint32_t mbyte, vbyte;
            m4 = encode4<false, kStoch>(mo, word, mbyte);
            v4 = encode4<true, kStoch>(vo, word, vbyte);
            if ((threadIdx.x & 7) == 0 && (kFull || j < k.n)) {
                k.ms[j / zdp::kMxBlock] = static_cast<uint8_t>(mbyte);
                k.vs[j / zdp::kMxBlock] = static_cast<uint8_t>(vbyte);
            }
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float q = mo[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(vo[e], c.isbf, c.epsf));
                po[e] = p[e] - __builtin_fmaf(c.lrwdf, p[e], c.ssf * q);
            }
            // The hardware's reciprocal has no denormal results: above 2^126
            // it is 0 and the weight would stay.  1/sqrt(1-b2^t) <= 2^26.5,
            // so such a denominator has a root above 2^98, whose variance is
            // past fp32's range, or a huge eps.  Its element takes float64.
            if (wide || c.epsf >= 0x1p124f) {
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    if (!(__builtin_fmaf(vo[e], c.isbf, c.epsf) >= 0x1p125f)) continue;
                    const double q = static_cast<double>(mo[e]) / (static_cast<double>(vo[e]) * c.isb + c.eps);
                    po[e] = static_cast<float>((static_cast<double>(p[e]) * c.dcy) - (c.ss * q));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                float a, b, d;
                adam1(c, g.at(e) * c.factor, p[e], m[e], v[e], a, b, d);
                po[e] = a;
                mo[e] = b;
                vo[e] = d;
            }
        }
        if (kFull || j + kV <= k.n)
            store_part<true, kParam>(k, j, po, mo, vo, m4, v4);
        else if (j < k.n)
            store_part<false, kParam>(k, j, po, mo, vo, m4, v4);
    }
};

// All rows of a chunk.
template <int kGrad, bool kMx>
__device__ __forceinline__ void load_chunk(Row<kGrad, kMx> (&r)[kRows], const Chunk& k) {
    const int j = static_cast<int>(threadIdx.x) * kV;
    if (k.n == kChunk) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) r[u].template load<true>(k, j + u * kRow);
    } else {
#pragma unroll
        for (int u = 0; u < kRows; ++u) r[u].template load<false>(k, j + u * kRow);
    }
}

template <int kGrad, int kParam, bool kMx, bool kStoch>
__device__ __forceinline__ void finish_chunk(Row<kGrad, kMx> (&r)[kRows], const Chunk& k, const AdamScalars& c,
                                             const RandomKey& key) {
    const int j = static_cast<int>(threadIdx.x) * kV;
    if (k.n == kChunk) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) r[u].template finish<true, kParam, kStoch>(k, j + u * kRow, c, key);
    } else {
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (u * kRow < k.n) r[u].template finish<false, kParam, kStoch>(k, j + u * kRow, c, key);
    }
}

// One step of the list's chunks [from, to), in place.  Bound by HBM's mixed
// rate (a copy reaches 5.2 to 5.4 TB/s).  Chunks are dealt to the workgroups
// in rounds of the grid, so that all of them walk the arrays side by side;
// each workgroup takes a chunk's four rows from registers while the next
// chunk's are on their way (kPipe).  4096 elements a chunk: 2048 measured 6%
// (fp32 states) and 2% (8-bit) slower, 8192 4% and 12%.
//   fp32 states, f16 gradients and copy: 28 bytes an element, GPT-2 small
//     575 us, 6.1 TB/s, VALU 37% busy
//   8-bit states, bf16 gradients and copy: 16.1 bytes, GPT-2 small 372 us, 5.4
//     TB/s, VALU 69% busy; a quarter of GPT-2 XL 1216 us, 5.2 TB/s
// Short lists are bound by latency: table, descriptor and data in turn, then
// the stores (400 tensors: 14.3 us of kernel for 1.4e6 elements with fp32
// states, 12.1 for 1.8e6 with 8-bit ones).
template <int kGrad, int kParam, bool kMx, bool kStoch, bool kPipe>
__global__ void __launch_bounds__(kBlock) tensors_adam_kernel(ListArgs list, TensorStepArgs a, int64_t from, int64_t to) {
    const bool skip = a.overflow != nullptr && *a.overflow != 0;
    if (!skip) {
        Row<kGrad, kMx> r[kRows];
        Chunk k;
        int64_t i = from + blockIdx.x;
        if (i < to) {
            k = chunk_at<kGrad, kMx>(list, i);
            load_chunk(r, k);
        }
        const AdamScalars c = step_scalars(a);
        const RandomKey key = random_key(a.seed, static_cast<uint32_t>(a.ctl->t) + 1u);
        while (i < to) {
            const int64_t i2 = i + gridDim.x;
            if (kPipe) {
                Chunk k2 = k;
                Row<kGrad, kMx> r2[kRows];
                if (i2 < to) {
                    k2 = chunk_at<kGrad, kMx>(list, i2);
                    load_chunk(r2, k2);
                }
                __builtin_amdgcn_sched_barrier(0);
                finish_chunk<kGrad, kParam, kMx, kStoch>(r, k, c, key);
#pragma unroll
                for (int u = 0; u < kRows; ++u) r[u] = r2[u];
                k = k2;
            } else {
                finish_chunk<kGrad, kParam, kMx, kStoch>(r, k, c, key);
                if (i2 < to) {
                    k = chunk_at<kGrad, kMx>(list, i2);
                    load_chunk(r, k);
                }
            }
            i = i2;
        }
    }
    if (to < list.n_chunks) return;  // the list's last launch commits
    // its last workgroup does: every workgroup has read the control block by
    // the barrier before its ticket, and nothing it wrote is read here, so
    // the ticket orders no other memory
    __syncthreads();
    if (threadIdx.x == 0 && last_to_draw(a.ticket)) commit(a, skip);
}

// ------------------------------------------------------- encode and decode
// Both bound by HBM: 5.03 bytes an element (1.2e8 values: encode 110 us, 5.7
// TB/s; decode 115 us, 5.4 TB/s, four fifths of it writes).
// Rows whose loads are under way together; GPT-2-small-sized arrays, eight
// workgroups per CU: one row 116 us to encode and 113 to decode, four 110
// and 115.
constexpr int kMxRows = 4;

template <bool kRoot, bool kStoch>
__global__ void __launch_bounds__(kBlock) mx8_encode_kernel(const float* x_in, int64_t n, uint8_t* codes_out,
                                                            uint8_t* scales_out, RandomKey key,
                                                            uint32_t counter) {
    constexpr int kSpan = kMxRows * kRow;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kSpan; base < n;
         base += static_cast<int64_t>(gridDim.x) * kSpan) {
        const gcf32 x = (gcf32)x_in + base;
        const gu8 codes = (gu8)codes_out + base, scales = (gu8)scales_out + base / zdp::kMxBlock;
        const int rest = static_cast<int>(n - base < kSpan ? n - base : kSpan);
        fvec v[kMxRows];
#pragma unroll
        for (int u = 0; u < kMxRows; ++u) {
            const int j = u * kRow + static_cast<int>(threadIdx.x) * kV;
            v[u] = fvec{0.0f, 0.0f, 0.0f, 0.0f};
            if (j + kV <= rest)
                v[u] = load_f32<true>(x, j, rest);
            else if (j < rest)
                v[u] = load_f32<false>(x, j, rest);
        }
#pragma unroll
        for (int u = 0; u < kMxRows; ++u) {
            if (u * kRow >= rest) break;
            const int j = u * kRow + static_cast<int>(threadIdx.x) * kV;
            uint32_t word[kV] = {0, 0, 0, 0};
            if (kStoch) {
#pragma unroll
                for (int e = 0; e < kV; ++e)
                    word[e] = random_word(key, counter + static_cast<uint32_t>(base) + static_cast<uint32_t>(j + e));
            }
            if (kRoot) roots4(v[u]);
            uint32_t byte;
            const uint32_t c = encode4<kRoot, kStoch>(v[u], word, byte);
            if (j + kV <= rest)
                store_8<true>(codes, j, rest, c);
            else if (j < rest)
                store_8<false>(codes, j, rest, c);
            if ((threadIdx.x & 7) == 0 && j < rest) scales[j / zdp::kMxBlock] = static_cast<uint8_t>(byte);
        }
    }
}

template <bool kRoot>
__global__ void __launch_bounds__(kBlock) mx8_decode_kernel(const uint8_t* codes_in, const uint8_t* scales_in,
                                                            int64_t n, float* x_out) {
    constexpr int kSpan = kMxRows * kRow;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kSpan; base < n;
         base += static_cast<int64_t>(gridDim.x) * kSpan) {
        const gcu8 codes = (gcu8)codes_in + base, scales = (gcu8)scales_in + base / zdp::kMxBlock;
        const gf32 x = (gf32)x_out + base;
        const int rest = static_cast<int>(n - base < kSpan ? n - base : kSpan);
        uint32_t c[kMxRows], e[kMxRows];
#pragma unroll
        for (int u = 0; u < kMxRows; ++u) {
            const int j = u * kRow + static_cast<int>(threadIdx.x) * kV;
            c[u] = 0;
            e[u] = 1;
            if (j < rest) e[u] = scales[j / zdp::kMxBlock];
            if (j + kV <= rest)
                c[u] = load_8<true>(codes, j, rest);
            else if (j < rest)
                c[u] = load_8<false>(codes, j, rest);
        }
#pragma unroll
        for (int u = 0; u < kMxRows; ++u) {
            const int j = u * kRow + static_cast<int>(threadIdx.x) * kV;
            fvec v = decode4(c[u], scale_value(e[u]));
            if (kRoot) v = v * v;
            if (j + kV <= rest)
                store_f32<true>(x, j, rest, v);
            else if (j < rest)
                store_f32<false>(x, j, rest, v);
        }
    }
}

// --------------------------------------------------------------- launchers
constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];

// Compute units of the current device (256 if the runtime does not say).
int cu_count() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
    int n = g_cus[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) {
        (void)hipGetLastError();
        return 256;
    }
    g_cus[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Workgroups for `units` units of work, at most per_cu to a CU.
int grid_of(int64_t units, int per_cu) {
    int64_t cap = static_cast<int64_t>(cu_count()) * per_cu;
    if (cap > zdp::kMaxBlocks) cap = zdp::kMaxBlocks;
    const int64_t g = units < cap ? units : cap;
    return static_cast<int>(g < 1 ? 1 : g);
}

int finish_launch() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        zdp::set_last_hip_error(static_cast<int>(e));
        return ZERO_EHIP;
    }
    return ZERO_OK;
}

// Workgroups per CU of the long kernels; each was timed against its
// neighbours on the GPT-2 shaped lists.  Grids that are not a multiple of
// the CU count lose 10 to 30%.
//   norm: 5 (1.56e9 bf16 gradients, all streaming: 443 us; 4: 486, 6: 443, 8: 505)
//   adam, fp32 states: 1 with the next chunk's loads under way (GPT-2 small:
//     609 us; 2 such: 656, 4 without the loads ahead: 672)
//   adam, 8-bit states: 3 (a quarter of GPT-2 XL: 1237 us; 2: 1240, 1: 1454).
//     With 16-bit gradients the kernels take up to 168 VGPRs, the most of
//     which three workgroups fit (174: two, and GPT-2 small 449 us for 397);
//     with f32 gradients 182, and two fit (GPT-2 small: 411 us).
constexpr int kNormPerCu = 5;
constexpr int kAdamPerCu = 1;
constexpr int kAdamMxPerCu = 3;
// fp32 states: a list of at most kAdamShortChunks chunks per CU takes more
// workgroups without loads ahead (400 tensors, 673 chunks: 13.9 us; 16.7 on
// kAdamPerCu; 2048 chunks: 44.8 and 47.1; 4096: 85.1 and 85.4).
constexpr int kAdamShortChunks = 8;
constexpr int kAdamShortPerCu = 4;
// A list of more than twice this many chunks is stepped in launches of
// about 2^26 elements (a quarter of GPT-2 XL, one launch against six: 1946
// and 1875 us with fp32 states, 1231 and 1213 with 8-bit ones; GPT-2 small
// in two: within 1%; launches of 2^24: 3% to 8% slower).
constexpr int64_t kPieceChunks = 1 << 14;
constexpr int kMx8PerCu = 8;

// The chunks [0, n_chunks) in launches of whole rounds of the grid.
template <int kGrad, int kParam, bool kMx, bool kStoch, bool kPipe>
int adam_launches(const ListArgs& list, const TensorStepArgs& a, int grid, hipStream_t s) {
    int64_t per = list.n_chunks;
    if (per > 2 * kPieceChunks) {
        const int64_t pieces = (per + kPieceChunks - 1) / kPieceChunks;
        per = ((per + pieces - 1) / pieces + grid - 1) / grid * grid;
    }
    int64_t from = 0;
    do {
        const int64_t to = list.n_chunks - from > per ? from + per : list.n_chunks;
        tensors_adam_kernel<kGrad, kParam, kMx, kStoch, kPipe><<<grid, kBlock, 0, s>>>(list, a, from, to);
        const int rc = finish_launch();
        if (rc != ZERO_OK) return rc;
        from = to;
    } while (from < list.n_chunks);
    return ZERO_OK;
}

template <int kGrad, int kParam>
int adam_with(const ListArgs& list, const TensorStepArgs& a, hipStream_t s) {
    if (list.state_type == ZERO_TYPE_MX8) {
        const int grid = grid_of(list.n_chunks, kAdamMxPerCu);
        return a.stochastic ? adam_launches<kGrad, kParam, true, true, true>(list, a, grid, s)
                            : adam_launches<kGrad, kParam, true, false, true>(list, a, grid, s);
    }
    if (list.n_chunks <= static_cast<int64_t>(cu_count()) * kAdamShortChunks)
        return adam_launches<kGrad, kParam, false, false, false>(list, a, grid_of(list.n_chunks, kAdamShortPerCu), s);
    return adam_launches<kGrad, kParam, false, false, true>(list, a, grid_of(list.n_chunks, kAdamPerCu), s);
}

template <int kGrad>
int adam_of(const ListArgs& list, const TensorStepArgs& a, hipStream_t s) {
    if (list.param_type == ZERO_TYPE_F16) return adam_with<kGrad, ZERO_TYPE_F16>(list, a, s);
    if (list.param_type == ZERO_TYPE_BF16) return adam_with<kGrad, ZERO_TYPE_BF16>(list, a, s);
    return adam_with<kGrad, ZERO_TYPE_NONE>(list, a, s);
}

int mx8_grid(int64_t n) { return grid_of((n - 1) / (kMxRows * kRow) + 1, kMx8PerCu); }

template <bool kRoot>
int encode_of(const float* x, int64_t n, uint8_t* codes, uint8_t* scales, bool stochastic, const RandomKey& key,
              uint32_t counter, hipStream_t s) {
    const int grid = mx8_grid(n);
    if (stochastic)
        mx8_encode_kernel<kRoot, true><<<grid, kBlock, 0, s>>>(x, n, codes, scales, key, counter);
    else
        mx8_encode_kernel<kRoot, false><<<grid, kBlock, 0, s>>>(x, n, codes, scales, key, counter);
    return finish_launch();
}

}  // namespace

namespace zdp {

int launch_tensors_norm(const ListArgs& list, double inv_scale, const zero_step_ctl* dyn, int32_t* overflow,
                        double* sumsq, const Partials& ws, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int grid = grid_of(list.n_chunks, kNormPerCu);
    if (list.grad_type == ZERO_TYPE_F32)
        tensors_norm_kernel<ZERO_TYPE_F32><<<grid, kBlock, 0, s>>>(list, inv_scale, dyn, overflow, sumsq, ws);
    else if (list.grad_type == ZERO_TYPE_F16)
        tensors_norm_kernel<ZERO_TYPE_F16><<<grid, kBlock, 0, s>>>(list, inv_scale, dyn, overflow, sumsq, ws);
    else
        tensors_norm_kernel<ZERO_TYPE_BF16><<<grid, kBlock, 0, s>>>(list, inv_scale, dyn, overflow, sumsq, ws);
    return finish_launch();
}

int launch_tensors_adam(const ListArgs& list, const TensorStepArgs& a, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (list.grad_type == ZERO_TYPE_F32) return adam_of<ZERO_TYPE_F32>(list, a, s);
    if (list.grad_type == ZERO_TYPE_F16) return adam_of<ZERO_TYPE_F16>(list, a, s);
    return adam_of<ZERO_TYPE_BF16>(list, a, s);
}

int launch_mx8_encode(const float* x, int64_t n, bool root, uint8_t* codes, uint8_t* scales, bool stochastic,
                      uint64_t seed, uint32_t step, uint64_t flat_off, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const RandomKey key = random_key(seed, step);
    const uint32_t counter = static_cast<uint32_t>(flat_off);
    return root ? encode_of<true>(x, n, codes, scales, stochastic, key, counter, s)
                : encode_of<false>(x, n, codes, scales, stochastic, key, counter, s);
}

int launch_mx8_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, bool root, float* x, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int grid = mx8_grid(n);
    if (root)
        mx8_decode_kernel<true><<<grid, kBlock, 0, s>>>(codes, scales, n, x);
    else
        mx8_decode_kernel<false><<<grid, kBlock, 0, s>>>(codes, scales, n, x);
    return finish_launch();
}

}  // namespace zdp
