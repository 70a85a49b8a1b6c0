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
//            one IEEE float64 operation at a time, state stored as fp32, or
//            as 8 bits: fp32(m') and sqrt(fp32(v')) encoded as below
//   encode   blocks of 32 fp32 values: scale 2^(e-127) with the smallest e >= 1
//            that keeps the largest magnitude within 448 scales, each value
//            over the scale in e4m3 (nearest, or stochastic: the random word's
//            top 20 bits added to the 20 bits that are cut off)
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

template <typename T>
__device__ __forceinline__ T ldg(ZDP_GLOBAL const T* p) {
    return __builtin_nontemporal_load(p);
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

// The four codes of x, whose block (8 lanes) may lie in any part of the
// wave: all lanes have to be here, with zeros for elements that are not.
// The conversions take the scale as an operand.  Their stochastic form adds
// the top 20 bits of its random operand to the mantissa's last 20 bits and
// cuts them off, counted in the target's subnormal steps below 2^-6.
template <bool kRoot>
__device__ __forceinline__ uint32_t encode4(const fvec& x, bool stochastic, const uint32_t (&word)[kV],
                                            uint32_t& byte) {
    uint32_t big = 0;
#pragma unroll
    for (int e = 0; e < kV; ++e) big = max(big, __builtin_bit_cast(uint32_t, static_cast<float>(x[e])) & 0x7FFFFFFFu);
    big = max8(big);
    byte = scale_byte(big);
    if (byte == 255u) return 0x7F7F7F7Fu;
    const float scale = __builtin_bit_cast(float, byte << 23);
    fvec y = x;
    if (kRoot) {
        // a positive root keeps at least the smallest code: rounded to zero
        // it would turn its weight's next update into m/eps
        const float least = scale * 0x1p-9f;
#pragma unroll
        for (int e = 0; e < kV; ++e) y[e] = y[e] > 0.0f && y[e] < least ? least : static_cast<float>(y[e]);
    }
    if (stochastic) {
        int c = 0;
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, y[0], kRoot ? word[0] << 16 : word[0], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, y[1], kRoot ? word[1] << 16 : word[1], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, y[2], kRoot ? word[2] << 16 : word[2], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(c, y[3], kRoot ? word[3] << 16 : word[3], scale, 3);
        return static_cast<uint32_t>(c);
    }
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 c = {0, 0};
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, y[0], y[1], scale, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, y[2], y[3], scale, true);
    return __builtin_bit_cast(uint32_t, c);
}

// ------------------------------------------------------- loads and stores
// A lane's kV elements of an array at element j of n; a row that is not
// `full` is loaded and stored element by element, with zeros for the
// elements past n.
template <bool kFull>
__device__ __forceinline__ fvec load_f32(gcf32 p, int j, int n) {
    if (kFull) return ldg(reinterpret_cast<ZDP_GLOBAL const fvec*>(p + j));
    fvec x;
#pragma unroll
    for (int e = 0; e < kV; ++e) x[e] = j + e < n ? p[j + e] : 0.0f;
    return x;
}

template <bool kFull>
__device__ __forceinline__ hvec load_16(gcu16 p, int j, int n) {
    if (kFull) return ldg(reinterpret_cast<ZDP_GLOBAL const hvec*>(p + j));
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
    __device__ __forceinline__ double at(int e) const {
        const uint32_t w = h[e >> 1];
        if (kType == ZERO_TYPE_BF16)
            return static_cast<double>(__builtin_bit_cast(float, (e & 1) ? w & 0xFFFF0000u : w << 16));
        const f16x2 v = __builtin_bit_cast(f16x2, w);
        return static_cast<double>(static_cast<float>(v[e & 1]));
    }
    template <bool kFull>
    __device__ __forceinline__ void load(gcu8 p, int j, int n) {
        h = load_16<kFull>(reinterpret_cast<gcu16>(p), j, n);
    }
};
template <>
struct GradVec<ZERO_TYPE_F32> {
    fvec f;
    __device__ __forceinline__ double at(int e) const { return static_cast<double>(static_cast<float>(f[e])); }
    template <bool kFull>
    __device__ __forceinline__ void load(gcu8 p, int j, int n) {
        f = load_f32<kFull>(reinterpret_cast<gcf32>(p), j, n);
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
template <int kGrad>
__global__ void __launch_bounds__(kBlock) tensors_norm_kernel(ListArgs list, double inv_scale,
                                                              const zero_step_ctl* dyn, int32_t* overflow,
                                                              double* sumsq, Partials ws) {
    double sq = 0.0;
    for (int64_t c = blockIdx.x; c < list.n_chunks; c += gridDim.x) {
        const Place at = place_of(list, c);
        const int n = at.count();
        const gcu8 g = at.bytes(at.desc->g, grad_size<kGrad>());
        GradVec<kGrad> v[kRows];
        const int full = n / kRow;
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int j = k * kRow + static_cast<int>(threadIdx.x) * kV;
            if (k < full)
                v[k].template load<true>(g, j, n);
            else
                v[k].template load<false>(g, j, n);
        }
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
    if (threadIdx.x == 0) {
        ws.sq[blockIdx.x] = sq;
        const uint32_t prev = __hip_atomic_fetch_add(ws.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        s_last = prev == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kBlock)
        t += __hip_atomic_load(ws.sq + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = block_sum(t);
    if (threadIdx.x == 0) {
        // any inf or NaN among the gradients, or a loss scale without a
        // finite reciprocal, leaves the sum inf or NaN
        const double inv = dyn != nullptr ? 1.0 / dyn->loss_scale : inv_scale;
        const double total = t * (inv * inv);
        *sumsq = total;
        *overflow = __builtin_isfinite(total) ? 0 : 1;
        __hip_atomic_store(ws.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// ------------------------------------------------------------------- adam
// Scalars of the step taken, t = committed + 1.
struct AdamScalars {
    double b1, b2, omb1, omb2, ss, isb, dcy, eps, factor;
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
    __device__ __forceinline__ void load(const Chunk& k, int j) {
        g.template load<kFull>(k.g, j, k.n);
        p = load_f32<kFull>(reinterpret_cast<gcf32>(k.p), j, k.n);
        if (kMx) {
            mc = load_8<kFull>(k.m, j, k.n);
            vc = load_8<kFull>(k.v, j, k.n);
            const bool in = kFull || j < k.n;
            mb = in ? k.ms[j / zdp::kMxBlock] : 1u;
            vb = in ? k.vs[j / zdp::kMxBlock] : 1u;
        } else {
            m = load_f32<kFull>(reinterpret_cast<gcf32>(k.m), j, k.n);
            v = load_f32<kFull>(reinterpret_cast<gcf32>(k.v), j, k.n);
        }
    }

    template <bool kFull, int kParam>
    __device__ __forceinline__ void finish(const Chunk& k, int j, const AdamScalars& c, bool stochastic,
                                           const RandomKey& key) {
        if (kMx) {
            m = decode4(mc, scale_value(mb));
            v = decode4(vc, scale_value(vb));
            v = v * v;
        }
        fvec po, mo, vo;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            float a, b, d;
            adam1(c, g.at(e) * c.factor, p[e], m[e], v[e], a, b, d);
            po[e] = a;
            mo[e] = b;
            vo[e] = d;
        }
        store_f32<kFull>(reinterpret_cast<gf32>(k.p), j, k.n, po);
        if (kParam != ZERO_TYPE_NONE) store_16<kFull>(reinterpret_cast<gu16>(k.w), j, k.n, pack_param<kParam>(po));
        if (kMx) {
            uint32_t word[kV] = {0, 0, 0, 0};
            if (stochastic) {
#pragma unroll
                for (int e = 0; e < kV; ++e) word[e] = random_word(key, k.counter + static_cast<uint32_t>(j + e));
            }
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const bool in = kFull || j + e < k.n;  // elements past the end count as zeros
                mo[e] = in ? static_cast<float>(mo[e]) : 0.0f;
                vo[e] = in ? __builtin_sqrtf(vo[e]) : 0.0f;
            }
            uint32_t mbyte, vbyte;
            const uint32_t m4 = encode4<false>(mo, stochastic, word, mbyte);
            const uint32_t v4 = encode4<true>(vo, stochastic, word, vbyte);
            store_8<kFull>(k.m, j, k.n, m4);
            store_8<kFull>(k.v, j, k.n, v4);
            if ((threadIdx.x & 7) == 0 && (kFull || j < k.n)) {
                k.ms[j / zdp::kMxBlock] = static_cast<uint8_t>(mbyte);
                k.vs[j / zdp::kMxBlock] = static_cast<uint8_t>(vbyte);
            }
        } else {
            store_f32<kFull>(reinterpret_cast<gf32>(k.m), j, k.n, mo);
            store_f32<kFull>(reinterpret_cast<gf32>(k.v), j, k.n, vo);
        }
    }
};

template <int kGrad, int kParam, bool kMx>
__global__ void __launch_bounds__(kBlock) tensors_adam_kernel(ListArgs list, TensorStepArgs a) {
    const bool skip = a.overflow != nullptr && *a.overflow != 0;
    if (!skip) {
        const AdamScalars c = step_scalars(a);
        const RandomKey key = random_key(a.seed, static_cast<uint32_t>(a.ctl->t) + 1u);
        for (int64_t i = blockIdx.x; i < list.n_chunks; i += gridDim.x) {
            const Chunk k = chunk_at<kGrad, kMx>(list, i);
            for (int row = 0; row * kRow < k.n; ++row) {
                const int j = row * kRow + static_cast<int>(threadIdx.x) * kV;
                Row<kGrad, kMx> r;
                if ((row + 1) * kRow <= k.n) {
                    r.template load<true>(k, j);
                    r.template finish<true, kParam>(k, j, c, a.stochastic != 0, key);
                } else {
                    r.template load<false>(k, j);
                    r.template finish<false, kParam>(k, j, c, a.stochastic != 0, key);
                }
            }
        }
    }
    // the last workgroup commits: every workgroup has read the control
    // block by the barrier before its ticket, and nothing it wrote is read
    // here, so the ticket orders no other memory
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t prev = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (prev == gridDim.x - 1) {
            commit(a, skip);
            __hip_atomic_store(a.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// ------------------------------------------------------- encode and decode
template <bool kRoot>
__global__ void __launch_bounds__(kBlock) mx8_encode_kernel(const float* x_in, int64_t n, uint8_t* codes_out,
                                                            uint8_t* scales_out, bool stochastic, RandomKey key,
                                                            uint32_t counter) {
    const gcf32 x = (gcf32)x_in;
    const gu8 codes = (gu8)codes_out, scales = (gu8)scales_out;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kRow; base < n;
         base += static_cast<int64_t>(gridDim.x) * kRow) {
        const int rest = static_cast<int>(n - base < kRow ? n - base : kRow);
        const int j = static_cast<int>(threadIdx.x) * kV;
        const bool full = rest == kRow;
        fvec v = full ? load_f32<true>(x + base, j, rest) : load_f32<false>(x + base, j, rest);
        uint32_t word[kV] = {0, 0, 0, 0};
        if (stochastic) {
#pragma unroll
            for (int e = 0; e < kV; ++e)
                word[e] = random_word(key, counter + static_cast<uint32_t>(base) + static_cast<uint32_t>(j + e));
        }
        if (kRoot) {
#pragma unroll
            for (int e = 0; e < kV; ++e) v[e] = __builtin_sqrtf(v[e]);
        }
        uint32_t byte;
        const uint32_t c = encode4<kRoot>(v, stochastic, word, byte);
        if (full)
            store_8<true>(codes + base, j, rest, c);
        else
            store_8<false>(codes + base, j, rest, c);
        if ((threadIdx.x & 7) == 0 && j < rest) scales[(base + j) / zdp::kMxBlock] = static_cast<uint8_t>(byte);
    }
}

template <bool kRoot>
__global__ void __launch_bounds__(kBlock) mx8_decode_kernel(const uint8_t* codes_in, const uint8_t* scales_in,
                                                            int64_t n, float* x_out) {
    const gcu8 codes = (gcu8)codes_in, scales = (gcu8)scales_in;
    const gf32 x = (gf32)x_out;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kRow; base < n;
         base += static_cast<int64_t>(gridDim.x) * kRow) {
        const int rest = static_cast<int>(n - base < kRow ? n - base : kRow);
        const int j = static_cast<int>(threadIdx.x) * kV;
        if (j >= rest) continue;
        const bool full = rest == kRow;
        const uint32_t c = full ? load_8<true>(codes + base, j, rest) : load_8<false>(codes + base, j, rest);
        fvec v = decode4(c, scale_value(scales[(base + j) / zdp::kMxBlock]));
        if (kRoot) v = v * v;
        if (full)
            store_f32<true>(x + base, j, rest, v);
        else
            store_f32<false>(x + base, j, rest, v);
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

constexpr int kNormPerCu = 8;
constexpr int kAdamPerCu = 4;
constexpr int kMx8PerCu = 8;

template <int kGrad, bool kMx>
int adam_for(const ListArgs& list, const TensorStepArgs& a, hipStream_t s) {
    const int grid = grid_of(list.n_chunks, kAdamPerCu);
    if (list.param_type == ZERO_TYPE_F16)
        tensors_adam_kernel<kGrad, ZERO_TYPE_F16, kMx><<<grid, kBlock, 0, s>>>(list, a);
    else if (list.param_type == ZERO_TYPE_BF16)
        tensors_adam_kernel<kGrad, ZERO_TYPE_BF16, kMx><<<grid, kBlock, 0, s>>>(list, a);
    else
        tensors_adam_kernel<kGrad, ZERO_TYPE_NONE, kMx><<<grid, kBlock, 0, s>>>(list, a);
    return finish_launch();
}

template <int kGrad>
int adam_of(const ListArgs& list, const TensorStepArgs& a, hipStream_t s) {
    return list.state_type == ZERO_TYPE_MX8 ? adam_for<kGrad, true>(list, a, s) : adam_for<kGrad, false>(list, a, s);
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
    const int grid = grid_of((n + kRow - 1) / kRow, kMx8PerCu);
    const RandomKey key = random_key(seed, step);
    const uint32_t counter = static_cast<uint32_t>(flat_off);
    if (root)
        mx8_encode_kernel<true><<<grid, kBlock, 0, s>>>(x, n, codes, scales, stochastic, key, counter);
    else
        mx8_encode_kernel<false><<<grid, kBlock, 0, s>>>(x, n, codes, scales, stochastic, key, counter);
    return finish_launch();
}

int launch_mx8_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, bool root, float* x, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int grid = grid_of((n + kRow - 1) / kRow, kMx8PerCu);
    if (root)
        mx8_decode_kernel<true><<<grid, kBlock, 0, s>>>(codes, scales, n, x);
    else
        mx8_decode_kernel<false><<<grid, kBlock, 0, s>>>(codes, scales, n, x);
    return finish_launch();
}

}  // namespace zdp
