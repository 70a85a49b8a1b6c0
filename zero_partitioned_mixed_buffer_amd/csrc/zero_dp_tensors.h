// Internal declarations of the tensor-list operators (gradient norm, AdamW
// with 32-bit or 8-bit states, the 8-bit form's encode and decode), shared
// by their host unit (zero_dp_tensors.cpp) and their device unit
// (zero_dp_tensors.hip).  Not part of the public ABI.
#pragma once

#include <cstdint>

#include "zero_dp_internal.h"

namespace zdp {

// A list's unit of work: up to kChunk consecutive elements of one tensor,
// by one workgroup at a time (a multiple of 32, so 8-bit blocks never cross
// a chunk's edge).
constexpr int kChunk = 4096;
constexpr int kMxBlock = 32;  // elements that share a scale in the 8-bit form

// Counters of the operators' tickets, beside the workspace's first: in the
// bytes between its element count and its partial sums.  As there, every
// call leaves them at zero.
constexpr int64_t kWsSubTickets = 128;
constexpr uint32_t kSubTickets = 32;
static_assert(kWsRunCount + 8 <= kWsSubTickets && kWsSubTickets + 4 * kSubTickets <= kWsPartSq, "workspace layout");

// Device table of a list: the tensors' descriptors, then one reference per
// chunk, in list order.
struct TensorDesc {
    float* p;          // master
    const void* g;     // gradient
    uint16_t* w;       // 16-bit copy, or null
    void* m;           // float or e4m3 codes
    void* v;           // float or e4m3 codes of the root
    uint8_t* ms;       // block scales (8-bit states)
    uint8_t* vs;
    int64_t n;
    uint64_t flat_off;
    uint64_t reserved;
};
static_assert(sizeof(TensorDesc) == 80, "descriptor layout");
struct ChunkRef {
    int32_t tensor;
    int32_t chunk;
};

struct ListArgs {
    const TensorDesc* desc;
    const ChunkRef* chunks;
    int64_t n_chunks;
    int32_t grad_type, param_type, state_type;
};

struct TensorStepArgs {
    double lr, b1, b2, eps, wd;
    double inv_scale;         // 1/L of a static loss scale
    double max_norm;          // > 0: clip by *sumsq
    double growth, backoff;   // dynamic loss scaling
    int32_t interval;         // > 0: dynamic loss scaling, L = ctl->loss_scale
    int32_t stochastic;       // rounding of 8-bit states
    uint64_t seed;
    zero_step_ctl* ctl;
    const int32_t* overflow;  // null: the step is always taken
    const double* sumsq;      // null: no clipping, no norm recorded
    uint32_t* ticket;
};

// Every argument has been validated by the caller.  Each returns ZERO_OK or
// ZERO_EHIP.
int launch_tensors_norm(const ListArgs& list, double inv_scale, const zero_step_ctl* dyn, int32_t* overflow,
                        double* sumsq, const Partials& ws, void* stream);
int launch_tensors_adam(const ListArgs& list, const TensorStepArgs& a, void* stream);
int launch_mx8_encode(const float* x, int64_t n, bool root, uint8_t* codes, uint8_t* scales, bool stochastic,
                      uint64_t seed, uint32_t step, uint64_t flat_off, void* stream);
int launch_mx8_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, bool root, float* x, void* stream);

}  // namespace zdp
