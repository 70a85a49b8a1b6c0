// Entry points of the 8-bit layer operators: the argument validation of
// every call before its launch, and the workspaces' sizes.  Plain C++ with
// no HIP types, so that this unit can also be built for the host alone (with
// sanitizers).
#include <cstdint>

#include "../../include/zero_dp.h"
#include "zero_dp_block8.h"

namespace {

using zdp::b8_blocks;
using zdp::kB8;
using zdp::kB8MaxCols;
using zdp::kB8MaxRows;

bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(a - 1)) == 0; }

int64_t type_bytes(int32_t type) {
    return type == ZERO_TYPE_F32 ? 4 : type == ZERO_TYPE_F16 || type == ZERO_TYPE_BF16 ? 2 : 0;
}

// The bytes of a matrix: `rows` runs of `width` bytes, `stride` apart.
struct Region {
    uintptr_t lo;
    int64_t rows, width, stride;
};

Region flat(const void* p, int64_t bytes) { return Region{reinterpret_cast<uintptr_t>(p), 1, bytes, bytes}; }

bool empty(const Region& r) { return r.rows == 0 || r.width == 0 || r.lo == 0; }

uintptr_t end_of(const Region& r) {
    return r.lo + static_cast<uintptr_t>((r.rows - 1) * r.stride + r.width);
}

bool overlap(const Region& a, const Region& b) {
    if (empty(a) || empty(b) || end_of(a) <= b.lo || end_of(b) <= a.lo) return false;
    if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
    // rows of one pitch: apart where their columns are
    const uintptr_t pitch = static_cast<uintptr_t>(a.stride);
    const uintptr_t off = a.lo <= b.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
    return off < static_cast<uintptr_t>(a.width) || off + static_cast<uintptr_t>(b.width) > pitch;
}

bool same(const Region& a, const Region& b) {
    return a.lo == b.lo && a.rows == b.rows && a.width == b.width && (a.stride == b.stride || a.rows == 1);
}

// Checks a matrix; with rows and cols given, that it has that size.
int check_matrix(const zero_matrix* m, int64_t rows, int64_t cols, Region* r) {
    if (m == nullptr || m->reserved != 0 || type_bytes(m->type) == 0) return ZERO_EINVAL;
    if (m->rows < 0 || m->cols < 0 || m->stride < m->cols) return ZERO_EINVAL;
    if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) return ZERO_EINVAL;
    if (m->rows > kB8MaxRows || m->cols > kB8MaxCols) return ZERO_EOVERFLOW;
    const int64_t size = type_bytes(m->type);
    int64_t pitch = 0, all = 0;
    if (zdp::mul_overflows(m->stride, size, &pitch) || zdp::mul_overflows(pitch, m->rows, &all)) return ZERO_EOVERFLOW;
    *r = Region{reinterpret_cast<uintptr_t>(m->data), m->rows, m->cols * size, pitch};
    if (m->rows == 0 || m->cols == 0) {
        r->lo = 0;
        return ZERO_OK;
    }
    if (m->data == nullptr) return ZERO_EINVAL;
    return aligned(m->data, size) ? ZERO_OK : ZERO_EALIGN;
}

int check_block8(const zero_block8* m, int64_t rows, int64_t cols, Region* codes, Region* scales) {
    if (m == nullptr || m->reserved != 0 || (m->blocks != ZERO_BLOCK8_ROWS && m->blocks != ZERO_BLOCK8_TILES))
        return ZERO_EINVAL;
    if (m->rows < 0 || m->cols < 0 || m->codes_stride < m->cols || m->scales_stride < 0) return ZERO_EINVAL;
    if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) return ZERO_EINVAL;
    if (m->rows > kB8MaxRows || m->cols > kB8MaxCols || m->codes_stride > kB8MaxCols ||
        m->scales_stride > kB8MaxCols)
        return ZERO_EOVERFLOW;
    if (m->scales_stride < b8_blocks(m->cols)) return ZERO_EINVAL;
    if (m->codes_stride % 16 != 0 || m->scales_stride % 4 != 0) return ZERO_EALIGN;
    const int64_t srows = m->blocks == ZERO_BLOCK8_TILES ? b8_blocks(m->rows) : m->rows;
    int64_t all = 0;
    if (zdp::mul_overflows(m->scales_stride, srows, &all)) return ZERO_EOVERFLOW;
    *codes = Region{reinterpret_cast<uintptr_t>(m->codes), m->rows, m->cols, m->codes_stride};
    *scales = Region{reinterpret_cast<uintptr_t>(m->scales), srows, b8_blocks(m->cols), m->scales_stride};
    if (m->rows == 0 || m->cols == 0) {
        codes->lo = scales->lo = 0;
        return ZERO_OK;
    }
    if (m->codes == nullptr || m->scales == nullptr) return ZERO_EINVAL;
    return aligned(m->codes, 16) && aligned(m->scales, 4) ? ZERO_OK : ZERO_EALIGN;
}

// Whether out overlaps any of the n regions, but for those it may be (`may`:
// a bit for each).
bool conflict(const Region& out, const Region* in, int n, unsigned may = 0) {
    for (int i = 0; i < n; ++i)
        if (overlap(out, in[i]) && !((may >> i & 1u) != 0 && same(out, in[i]))) return true;
    return false;
}

constexpr Region kNone = {0, 0, 0, 0};

}  // namespace

extern "C" {

int zero_block8_encode(const zero_matrix* x, const float* row_mul, const void* col_mul, int32_t col_type,
                       const zero_block8* out, const zero_block8* out_t, void* stream) {
    Region rx, rc = kNone, rs = kNone, tc = kNone, ts = kNone;
    int rc_ = check_matrix(x, -1, -1, &rx);
    if (rc_ != ZERO_OK) return rc_;
    if (out == nullptr && out_t == nullptr) return ZERO_EINVAL;
    if (col_mul != nullptr && type_bytes(col_type) == 0) return ZERO_EINVAL;
    if (out != nullptr && (rc_ = check_block8(out, x->rows, x->cols, &rc, &rs)) != ZERO_OK) return rc_;
    if (out_t != nullptr && x->rows > kB8MaxCols) return ZERO_EOVERFLOW;
    if (out_t != nullptr && (rc_ = check_block8(out_t, x->cols, x->rows, &tc, &ts)) != ZERO_OK) return rc_;
    if (out != nullptr && out_t != nullptr && out->blocks != out_t->blocks) return ZERO_EINVAL;
    if (!aligned(row_mul, 4) || (col_mul != nullptr && !aligned(col_mul, type_bytes(col_type)))) return ZERO_EALIGN;
    if (x->rows == 0 || x->cols == 0) return ZERO_OK;
    const Region in[6] = {rx, flat(row_mul, x->rows * 4), flat(col_mul, x->cols * type_bytes(col_type)), rc, rs, tc};
    if (conflict(rc, in, 3) || conflict(rs, in, 4) || conflict(tc, in, 5) || conflict(ts, in, 6)) return ZERO_EALIAS;
    zdp::EncodeArgs a = {};
    a.x = x->data;
    a.row_mul = row_mul;
    a.col_mul = col_mul;
    if (out != nullptr) {
        a.codes = out->codes;
        a.scales = out->scales;
        a.codes_stride = out->codes_stride;
        a.scales_stride = out->scales_stride;
    }
    if (out_t != nullptr) {
        a.codes_t = out_t->codes;
        a.scales_t = out_t->scales;
        a.codes_t_stride = out_t->codes_stride;
        a.scales_t_stride = out_t->scales_stride;
    }
    a.rows = x->rows;
    a.cols = x->cols;
    a.x_stride = x->stride;
    a.type = x->type;
    a.col_type = col_type;
    a.tiles = (out != nullptr ? out : out_t)->blocks == ZERO_BLOCK8_TILES;
    return zdp::launch_block8_encode(a, stream);
}

int zero_rms_norm8(const zero_matrix* x, const zero_matrix* residual, const void* weight, int32_t weight_type,
                   double eps, const zero_matrix* h, const zero_block8* y, float* rstd, void* stream) {
    Region rx, rr = kNone, rh = kNone, rc, rs;
    int rc_ = check_matrix(x, -1, -1, &rx);
    if (rc_ != ZERO_OK) return rc_;
    if ((residual == nullptr) != (h == nullptr) || type_bytes(weight_type) == 0 || !(eps > 0.0) ||
        !__builtin_isfinite(eps))
        return ZERO_EINVAL;
    if (residual != nullptr) {
        if ((rc_ = check_matrix(residual, x->rows, x->cols, &rr)) != ZERO_OK) return rc_;
        if ((rc_ = check_matrix(h, x->rows, x->cols, &rh)) != ZERO_OK) return rc_;
        if (residual->type != x->type || h->type != x->type) return ZERO_EINVAL;
    }
    if ((rc_ = check_block8(y, x->rows, x->cols, &rc, &rs)) != ZERO_OK) return rc_;
    if (y->blocks != ZERO_BLOCK8_ROWS) return ZERO_EINVAL;
    if (x->rows == 0 || x->cols == 0) return x->rows == 0 ? ZERO_OK : ZERO_EINVAL;
    if (weight == nullptr || rstd == nullptr) return ZERO_EINVAL;
    if (!aligned(weight, type_bytes(weight_type)) || !aligned(rstd, 4)) return ZERO_EALIGN;
    const Region in[7] = {rx, rr, flat(weight, x->cols * type_bytes(weight_type)), rh, rc, rs, kNone};
    if (conflict(rh, in, 3, 3u) || conflict(rc, in, 4) || conflict(rs, in, 5) ||
        conflict(flat(rstd, x->rows * 4), in, 6))
        return ZERO_EALIAS;
    zdp::NormArgs a = {};
    a.x = x->data;
    a.r = residual != nullptr ? residual->data : nullptr;
    a.h = h != nullptr ? h->data : nullptr;
    a.w = weight;
    a.codes = y->codes;
    a.scales = y->scales;
    a.rstd = rstd;
    a.rows = x->rows;
    a.x_stride = x->stride;
    a.r_stride = residual != nullptr ? residual->stride : 0;
    a.h_stride = h != nullptr ? h->stride : 0;
    a.codes_stride = y->codes_stride;
    a.scales_stride = y->scales_stride;
    a.cols = static_cast<int32_t>(x->cols);
    a.type = x->type;
    a.w_type = weight_type;
    a.eps = eps;
    return zdp::launch_norm8(a, stream);
}

int64_t zero_rms_norm8_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kB8MaxRows || cols > kB8MaxCols) return 0;
    return (zdp::norm_back_groups(rows, cols) * cols * 4 + 15) / 16 * 16;
}

int zero_rms_norm8_backward(const zero_matrix* dy, const zero_matrix* h, const void* weight, int32_t weight_type,
                            const float* rstd, const zero_matrix* dh, const zero_matrix* dx, float* dweight,
                            void* workspace, void* stream) {
    Region ry, rh, rd = kNone, rx;
    int rc_ = check_matrix(dy, -1, -1, &ry);
    if (rc_ != ZERO_OK) return rc_;
    if ((rc_ = check_matrix(h, dy->rows, dy->cols, &rh)) != ZERO_OK) return rc_;
    if (dh != nullptr && (rc_ = check_matrix(dh, dy->rows, dy->cols, &rd)) != ZERO_OK) return rc_;
    if ((rc_ = check_matrix(dx, dy->rows, dy->cols, &rx)) != ZERO_OK) return rc_;
    if (h->type != dy->type || dx->type != dy->type || (dh != nullptr && dh->type != dy->type) ||
        type_bytes(weight_type) == 0)
        return ZERO_EINVAL;
    if (dy->cols == 0) return dy->rows == 0 ? ZERO_OK : ZERO_EINVAL;
    const int64_t ws_bytes = zero_rms_norm8_workspace_bytes(dy->rows, dy->cols);
    if (dy->rows > 0 && (weight == nullptr || rstd == nullptr || (dweight != nullptr && workspace == nullptr)))
        return ZERO_EINVAL;
    if (!aligned(weight, type_bytes(weight_type)) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
        !aligned(workspace, 16))
        return ZERO_EALIGN;
    const Region in[7] = {ry, rd, rh, flat(weight, dy->cols * type_bytes(weight_type)), flat(rstd, dy->rows * 4), rx,
                          flat(dweight, dy->cols * 4)};
    if (conflict(rx, in, 5, 3u) || conflict(in[6], in, 6) ||
        (dweight != nullptr && conflict(flat(workspace, ws_bytes), in, 7)))
        return ZERO_EALIAS;
    if (dy->rows == 0 && dweight == nullptr) return ZERO_OK;
    zdp::NormBackArgs a = {};
    a.dy = dy->data;
    a.h = h->data;
    a.dh = dh != nullptr ? dh->data : nullptr;
    a.dx = dx->data;
    a.w = weight;
    a.rstd = rstd;
    a.dw = dweight;
    a.part = static_cast<float*>(workspace);
    a.rows = dy->rows;
    a.dy_stride = dy->stride;
    a.h_stride = h->stride;
    a.dh_stride = dh != nullptr ? dh->stride : 0;
    a.dx_stride = dx->stride;
    a.cols = static_cast<int32_t>(dy->cols);
    a.type = dy->type;
    a.w_type = weight_type;
    return zdp::launch_norm8_backward(a, stream);
}

int64_t zero_block8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || k <= 0 || m > kB8MaxRows || n > kB8MaxRows || k > kB8MaxCols) return 0;
    if (zdp::product_tiles(m, n) > zdp::kProductMaxTiles) return 0;
    const int parts = zdp::product_parts(m, n, k);
    return parts > 1 ? parts * zdp::product_part_rows(m) * zdp::product_part_rows(n) * 4 : 0;
}

int zero_block8_product(const zero_block8* a, const zero_block8* b, const zero_matrix* add, const zero_matrix* out,
                        void* workspace, void* stream) {
    Region in[6] = {kNone, kNone, kNone, kNone, kNone, kNone}, ro;
    int rc_ = check_block8(a, -1, -1, &in[0], &in[1]);
    if (rc_ != ZERO_OK) return rc_;
    if ((rc_ = check_block8(b, -1, a->cols, &in[2], &in[3])) != ZERO_OK) return rc_;
    if ((rc_ = check_matrix(out, a->rows, b->rows, &ro)) != ZERO_OK) return rc_;
    if (add != nullptr) {
        if ((rc_ = check_matrix(add, a->rows, b->rows, &in[4])) != ZERO_OK) return rc_;
        if (add->type != out->type) return ZERO_EINVAL;
    }
    if (a->rows == 0 || b->rows == 0) return ZERO_OK;
    if (zdp::product_tiles(a->rows, b->rows) > zdp::kProductMaxTiles) return ZERO_EOVERFLOW;
    const int64_t ws_bytes = zero_block8_workspace_bytes(a->rows, b->rows, a->cols);
    if (ws_bytes > 0 && workspace == nullptr) return ZERO_EINVAL;
    if (!aligned(workspace, 16)) return ZERO_EALIGN;
    if (conflict(ro, in, 5, 1u << 4)) return ZERO_EALIAS;
    in[5] = ro;
    if (ws_bytes > 0 && conflict(flat(workspace, ws_bytes), in, 6)) return ZERO_EALIAS;
    zdp::ProductArgs p = {};
    const zero_block8* m[2] = {a, b};
    zdp::ProductSide* side[2] = {&p.a, &p.b};
    for (int i = 0; i < 2; ++i)
        *side[i] = zdp::ProductSide{m[i]->codes, m[i]->scales, m[i]->rows, static_cast<uint32_t>(m[i]->codes_stride),
                                    m[i]->scales_stride, m[i]->blocks == ZERO_BLOCK8_TILES ? 7 : 0};
    p.add = add != nullptr ? add->data : nullptr;
    p.out = out->data;
    p.part = static_cast<float*>(workspace);
    p.part_rows = zdp::product_part_rows(a->rows);
    p.part_stride = zdp::product_part_rows(b->rows);
    p.add_stride = add != nullptr ? add->stride : 0;
    p.out_stride = out->stride;
    p.k = static_cast<int32_t>(a->cols);
    p.type = out->type;
    return zdp::launch_block8_product(p, a->cols > 0 ? zdp::product_parts(a->rows, b->rows, a->cols) : 1, stream);
}

}  // extern "C"
