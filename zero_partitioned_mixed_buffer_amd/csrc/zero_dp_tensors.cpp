// Entry points of the tensor-list operators: the plan of a list (descriptor
// and chunk table), and the argument validation of every asynchronous call
// before its launch.  Plain C++ with no HIP types, so that this unit can
// also be built for the host alone (with sanitizers).
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/zero_dp.h"
#include "zero_dp_tensors.h"

namespace {

using zdp::ChunkRef;
using zdp::kChunk;
using zdp::kMxBlock;
using zdp::ListArgs;
using zdp::TensorDesc;

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
    int64_t out;       // 1: written by a step
};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

Span span_of(const void* p, int64_t bytes, bool out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, lo + static_cast<uintptr_t>(bytes), out};
}

// Sorts the spans and finds a byte that is written through one of them and
// belongs to another too.
bool write_conflict(Span* s, int64_t ns) {
    std::sort(s, s + ns, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t any = 0, out = 0;  // ends of all spans, and of the written ones, so far
    for (int64_t i = 0; i < ns; ++i) {
        if (s[i].lo == s[i].hi) continue;
        if (s[i].lo < (s[i].out ? any : out)) return true;
        any = std::max(any, s[i].hi);
        if (s[i].out) out = std::max(out, s[i].hi);
    }
    return false;
}

int64_t grad_bytes(int32_t type) { return type == ZERO_TYPE_F32 ? 4 : 2; }

constexpr int kSpansPerTensor = 7;

// Checks one tensor and lists the byte spans a step touches.
int check_tensor(const zero_tensor& t, int32_t grad_type, int32_t param_type, int32_t state_type, Span* s, int* ns) {
    *ns = 0;
    int64_t b4 = 0, end = 0;
    if (t.n < 0 || t.flat_off < 0 || t.reserved != 0) return ZERO_EINVAL;
    if (zdp::mul_overflows(t.n, 4, &b4) || zdp::add_overflows(t.flat_off, t.n, &end)) return ZERO_EOVERFLOW;
    if (t.n == 0) return ZERO_OK;
    // a chunk's number inside its tensor is 32 bits wide
    if ((t.n - 1) / kChunk >= INT32_MAX) return ZERO_EOVERFLOW;
    const bool mx = state_type == ZERO_TYPE_MX8;
    if (t.grad == nullptr) return ZERO_EINVAL;
    if (!aligned(t.grad, static_cast<uintptr_t>(grad_bytes(grad_type)))) return ZERO_EALIGN;
    s[(*ns)++] = span_of(t.grad, t.n * grad_bytes(grad_type), false);
    if (state_type == ZERO_TYPE_NONE) return ZERO_OK;
    if (t.master == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr) return ZERO_EINVAL;
    if ((t.param == nullptr) != (param_type == ZERO_TYPE_NONE)) return ZERO_EINVAL;
    if ((t.avg_scale == nullptr) == mx || (t.sq_scale == nullptr) == mx) return ZERO_EINVAL;
    if (!aligned(t.master, 4) || !aligned(t.param, 2)) return ZERO_EALIGN;
    if (!mx && (!aligned(t.exp_avg, 4) || !aligned(t.exp_avg_sq, 4))) return ZERO_EALIGN;
    s[(*ns)++] = span_of(t.master, b4, true);
    s[(*ns)++] = span_of(t.exp_avg, mx ? t.n : b4, true);
    s[(*ns)++] = span_of(t.exp_avg_sq, mx ? t.n : b4, true);
    if (param_type != ZERO_TYPE_NONE) s[(*ns)++] = span_of(t.param, t.n * 2, true);
    if (mx) {
        const int64_t blocks = (t.n - 1) / kMxBlock + 1;
        s[(*ns)++] = span_of(t.avg_scale, blocks, true);
        s[(*ns)++] = span_of(t.sq_scale, blocks, true);
    }
    return ZERO_OK;
}

bool is_grad_type(int32_t t) { return t == ZERO_TYPE_F32 || t == ZERO_TYPE_F16 || t == ZERO_TYPE_BF16; }

int check_list(const zero_tensor_list* l, const void* table, ListArgs* a) {
    if (l == nullptr || l->n_tensors < 0 || l->n_chunks < 0 || l->n_elems < 0 || l->table_bytes < 0 ||
        l->reserved != 0 || !is_grad_type(l->grad_type))
        return ZERO_EINVAL;
    if (table == nullptr && l->n_chunks != 0) return ZERO_EINVAL;
    if (!aligned(table, 16)) return ZERO_EALIGN;
    a->desc = static_cast<const TensorDesc*>(table);
    a->chunks = reinterpret_cast<const ChunkRef*>(a->desc + l->n_tensors);
    a->n_chunks = l->n_chunks;
    a->grad_type = l->grad_type;
    a->param_type = l->param_type;
    a->state_type = l->state_type;
    return ZERO_OK;
}

bool good_scale(double l) { return l > 0.0 && __builtin_isfinite(l) && __builtin_isfinite(1.0 / l); }

uint32_t* ticket_of(void* ws) { return reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + zdp::kWsTicket); }

// The arrays of an encode or a decode.
int check_mx8(const void* x, int64_t n, int32_t root, const uint8_t* codes, const uint8_t* scales) {
    if (n < 0 || (root != 0 && root != 1)) return ZERO_EINVAL;
    int64_t b4 = 0;
    if (zdp::mul_overflows(n, 4, &b4)) return ZERO_EOVERFLOW;
    if (n == 0) return ZERO_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr) return ZERO_EINVAL;
    if (!aligned(x, 4)) return ZERO_EALIGN;
    Span s[3] = {span_of(x, b4, true), span_of(codes, n, true), span_of(scales, (n - 1) / kMxBlock + 1, true)};
    return write_conflict(s, 3) ? ZERO_EALIAS : ZERO_OK;
}

}  // namespace

extern "C" {

int zero_tensors_plan(const zero_tensor* tensors, int32_t n_tensors, int32_t grad_type, int32_t param_type,
                      int32_t state_type, zero_tensor_list* list, void* table, int64_t table_cap) {
    if (list == nullptr || n_tensors < 0 || table_cap < 0 || (n_tensors > 0 && tensors == nullptr) ||
        (table_cap > 0 && table == nullptr))
        return ZERO_EINVAL;
    if (!is_grad_type(grad_type) ||
        (param_type != ZERO_TYPE_NONE && param_type != ZERO_TYPE_F16 && param_type != ZERO_TYPE_BF16) ||
        (state_type != ZERO_TYPE_NONE && state_type != ZERO_TYPE_F32 && state_type != ZERO_TYPE_MX8) ||
        (state_type == ZERO_TYPE_NONE && param_type != ZERO_TYPE_NONE))
        return ZERO_EINVAL;
    if (!aligned(table, 16)) return ZERO_EALIGN;
    int64_t elems = 0, chunks = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        Span s[kSpansPerTensor];
        int ns = 0;
        const int rc = check_tensor(tensors[i], grad_type, param_type, state_type, s, &ns);
        if (rc != ZERO_OK) return rc;
        if (zdp::add_overflows(elems, tensors[i].n, &elems)) return ZERO_EOVERFLOW;
        chunks += tensors[i].n > 0 ? (tensors[i].n - 1) / kChunk + 1 : 0;
    }
    const int64_t used = static_cast<int64_t>(sizeof(TensorDesc)) * n_tensors +
                         static_cast<int64_t>(sizeof(ChunkRef)) * chunks;
    // the table's memory first serves the sort of the overlap check
    const int64_t spans = static_cast<int64_t>(sizeof(Span)) * kSpansPerTensor * n_tensors;
    std::memset(list, 0, sizeof(*list));
    list->n_tensors = n_tensors;
    list->grad_type = grad_type;
    list->param_type = param_type;
    list->state_type = state_type;
    list->n_elems = elems;
    list->n_chunks = chunks;
    list->table_bytes = (std::max(used, spans) + 15) / 16 * 16;
    if (list->table_bytes > table_cap) return ZERO_ECAPACITY;
    Span* all = static_cast<Span*>(table);
    int64_t na = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        int ns = 0;
        (void)check_tensor(tensors[i], grad_type, param_type, state_type, all + na, &ns);
        na += ns;
    }
    if (write_conflict(all, na)) return ZERO_EALIAS;
    if (list->table_bytes > 0) std::memset(table, 0, static_cast<size_t>(list->table_bytes));
    TensorDesc* desc = static_cast<TensorDesc*>(table);
    ChunkRef* ref = reinterpret_cast<ChunkRef*>(desc + n_tensors);
    for (int32_t i = 0; i < n_tensors; ++i) {
        const zero_tensor& t = tensors[i];
        desc[i] = TensorDesc{t.master,
                             t.grad,
                             static_cast<uint16_t*>(t.param),
                             t.exp_avg,
                             t.exp_avg_sq,
                             t.avg_scale,
                             t.sq_scale,
                             t.n,
                             static_cast<uint64_t>(t.flat_off),
                             0};
        for (int64_t c = 0; c * kChunk < t.n; ++c) *ref++ = ChunkRef{i, static_cast<int32_t>(c)};
    }
    return ZERO_OK;
}

int zero_tensors_grad_norm(const zero_tensor_list* list, const void* table, double loss_scale,
                           const zero_step_ctl* ctl, int32_t* overflow, double* sumsq, void* workspace,
                           void* stream) {
    ListArgs a;
    const int rc = check_list(list, table, &a);
    if (rc != ZERO_OK) return rc;
    if (overflow == nullptr || sumsq == nullptr || workspace == nullptr) return ZERO_EINVAL;
    if (ctl == nullptr && !good_scale(loss_scale)) return ZERO_EINVAL;
    if (!aligned(overflow, 4) || !aligned(sumsq, 8) || !aligned(workspace, 16) || !aligned(ctl, 8))
        return ZERO_EALIGN;
    Span s[5] = {span_of(overflow, 4, true), span_of(sumsq, 8, true), span_of(workspace, zdp::kWsBytes, true),
                 span_of(table, table != nullptr ? list->table_bytes : 0, false),
                 span_of(ctl, ctl != nullptr ? static_cast<int64_t>(sizeof(zero_step_ctl)) : 0, false)};
    if (write_conflict(s, 5)) return ZERO_EALIAS;
    char* w = static_cast<char*>(workspace);
    zdp::Partials p;
    p.ticket = ticket_of(workspace);
    p.sq = reinterpret_cast<double*>(w + zdp::kWsPartSq);
    p.flag = reinterpret_cast<int32_t*>(w + zdp::kWsPartFlag);
    return zdp::launch_tensors_norm(a, ctl == nullptr ? 1.0 / loss_scale : 0.0, ctl, overflow, sumsq, p, stream);
}

int zero_tensors_adam_step(const zero_tensor_list* list, const void* table, const zero_adam_hp* hp,
                           double loss_scale, zero_step_ctl* ctl, const int32_t* overflow, const double* sumsq,
                           int32_t rounding, uint64_t seed, void* workspace, void* stream) {
    ListArgs a;
    const int rc = check_list(list, table, &a);
    if (rc != ZERO_OK) return rc;
    if (hp == nullptr || ctl == nullptr || workspace == nullptr) return ZERO_EINVAL;
    if (a.state_type != ZERO_TYPE_F32 && a.state_type != ZERO_TYPE_MX8) return ZERO_EINVAL;
    if (a.param_type != ZERO_TYPE_NONE && a.param_type != ZERO_TYPE_F16 && a.param_type != ZERO_TYPE_BF16)
        return ZERO_EINVAL;
    if (rounding != ZERO_ROUND_NEAREST && (rounding != ZERO_ROUND_STOCHASTIC || a.state_type != ZERO_TYPE_MX8))
        return ZERO_EINVAL;
    if (!(hp->lr >= 0.0) || !__builtin_isfinite(hp->lr) || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) ||
        !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) || !(hp->eps > 0.0) || !__builtin_isfinite(hp->eps) ||
        !(hp->weight_decay >= 0.0) || !__builtin_isfinite(hp->weight_decay) || !(hp->max_grad_norm >= 0.0) ||
        !__builtin_isfinite(hp->max_grad_norm) || hp->reserved != 0 || hp->scale_interval < 0)
        return ZERO_EINVAL;
    if (hp->max_grad_norm > 0.0 && (sumsq == nullptr || overflow == nullptr)) return ZERO_EINVAL;
    if (hp->scale_interval > 0 &&
        (overflow == nullptr || !(hp->scale_growth > 0.0) || !__builtin_isfinite(hp->scale_growth) ||
         !(hp->scale_backoff > 0.0) || !__builtin_isfinite(hp->scale_backoff)))
        return ZERO_EINVAL;
    if (hp->scale_interval == 0 && !good_scale(loss_scale)) return ZERO_EINVAL;
    if (!aligned(ctl, 8) || !aligned(overflow, 4) || !aligned(sumsq, 8) || !aligned(workspace, 16))
        return ZERO_EALIGN;
    Span s[5] = {span_of(ctl, static_cast<int64_t>(sizeof(zero_step_ctl)), true),
                 span_of(workspace, zdp::kWsBytes, true), span_of(overflow, overflow != nullptr ? 4 : 0, false),
                 span_of(sumsq, sumsq != nullptr ? 8 : 0, false),
                 span_of(table, table != nullptr ? list->table_bytes : 0, false)};
    if (write_conflict(s, 5)) return ZERO_EALIAS;
    zdp::TensorStepArgs t;
    t.lr = hp->lr;
    t.b1 = hp->beta1;
    t.b2 = hp->beta2;
    t.eps = hp->eps;
    t.wd = hp->weight_decay;
    t.inv_scale = hp->scale_interval > 0 ? 0.0 : 1.0 / loss_scale;
    t.max_norm = hp->max_grad_norm;
    t.growth = hp->scale_growth;
    t.backoff = hp->scale_backoff;
    t.interval = hp->scale_interval;
    t.stochastic = rounding == ZERO_ROUND_STOCHASTIC;
    t.seed = seed;
    t.ctl = ctl;
    t.overflow = overflow;
    t.sumsq = sumsq;
    t.ticket = ticket_of(workspace);
    return zdp::launch_tensors_adam(a, t, stream);
}

int zero_mx8_encode(const float* x, int64_t n, int32_t root, uint8_t* codes, uint8_t* scales, int32_t rounding,
                    uint64_t seed, int64_t step, int64_t flat_off, void* stream) {
    if (rounding != ZERO_ROUND_NEAREST && rounding != ZERO_ROUND_STOCHASTIC) return ZERO_EINVAL;
    if (step < 0 || flat_off < 0) return ZERO_EINVAL;
    int64_t end = 0;
    if (n >= 0 && zdp::add_overflows(flat_off, n, &end)) return ZERO_EOVERFLOW;
    const int rc = check_mx8(x, n, root, codes, scales);
    if (rc != ZERO_OK || n == 0) return rc;
    return zdp::launch_mx8_encode(x, n, root != 0, codes, scales, rounding == ZERO_ROUND_STOCHASTIC, seed,
                                  static_cast<uint32_t>(step), static_cast<uint64_t>(flat_off), stream);
}

int zero_mx8_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, int32_t root, float* x, void* stream) {
    const int rc = check_mx8(x, n, root, codes, scales);
    if (rc != ZERO_OK || n == 0) return rc;
    return zdp::launch_mx8_decode(codes, scales, n, root != 0, x, stream);
}

}  // extern "C"
