// Internal declarations of the 8-bit layer operators (the encode of a
// matrix, the root-mean-square norm and its gradients, the product of two
// encoded matrices), shared by their host unit (zero_dp_block8.cpp) and their
// device units (zero_dp_block8.hip, zero_dp_product.hip).  Not part of the
// public ABI.
#pragma once

#include <cstdint>

#include "zero_dp_internal.h"

namespace zdp {

constexpr int kB8 = 128;                      // values that share a scale, along a row
constexpr int64_t kB8MaxCols = 1 << 23;       // columns, and bytes between rows of codes
constexpr int64_t kB8MaxRows = INT32_MAX;

inline int64_t b8_blocks(int64_t n) { return (n + kB8 - 1) / kB8; }

// Workgroups of the norm's backward pass, each with a row of partial sums of
// dweight in the workspace: as many as there are rows, up to 1024 (four to a
// CU), fewer for long rows, whose partial sums would fill memory (at most
// 2^26 of them, but 64 rows).
inline int64_t norm_back_groups(int64_t rows, int64_t cols) {
    int64_t g = cols > 0 ? (INT64_C(1) << 26) / cols : 1024;
    g = g > 1024 ? 1024 : g < 64 ? 64 : g;
    return rows < g ? rows : g;
}

// Tiles of 256 x 256 that a product's launch may have (the runtime takes grids
// of less than 2^32 lanes).
constexpr int64_t kProductMaxTiles = 1 << 22;

inline int64_t product_tiles(int64_t m, int64_t n) { return ((m + 255) / 256) * ((n + 255) / 256); }

// Which of the product's kernels takes a size: the one without LDS on the way
// in, with either operand as its stream, or tiles of 128 x 128, 192 x 256 or
// 256 x 256, one workgroup to a CU.
enum ProductShape { kProductFewB, kProductFewA, kProductSmall, kProductMedium, kProductLarge };

constexpr int64_t kProductCus = 256;  // of an MI355X; the choices cost time alone

inline int64_t product_small_tiles(int64_t m, int64_t n) { return ((m + 127) / 128) * ((n + 127) / 128); }

// Parts that the sum over k of a product of small tiles is split into where
// there are few of them (more than one: each part's fp32 sums go to the
// workspace, and a second launch adds them up).
inline int64_t product_split(int64_t tiles, int64_t k) {
    if (tiles > kProductCus) return 1;
    int64_t parts = kProductCus / tiles;
    const int64_t most = k / 1024;
    parts = parts < most ? parts : most;
    if (parts < 2) return 1;
    // parts begin at a multiple of four blocks; none is empty
    const int64_t blocks = b8_blocks(k), per = ((blocks + parts - 1) / parts + 3) / 4 * 4;
    return (blocks + per - 1) / per;
}

// Rows of the other operand that a workgroup of the kernel without LDS takes, in sixteens.
inline int64_t product_few_rows(int64_t other) { return other <= 16 ? 1 : other <= 32 ? 2 : 4; }

inline int64_t product_few_groups(int64_t stream, int64_t other) {
    const int64_t t = product_few_rows(other);
    return ((stream + 15) / 16) * ((other + 16 * t - 1) / (16 * t));
}

// Estimated times in ns, fitted to measurements between 1 x 1600 x 6400 and
// 64 x 8192 x 8192.  Without LDS: 2.7 us and what a CU reads, at 40 bytes a ns
// (70 where the other operand is short), or memory's rate.  Measured, bf16:
// 1 x 6400 x 1600 4.9 us (in tiles 8.5), 267 x 1327 x 826 6.2 (8.9), 1034 x 165
// x 4042 12.2 (14.7), 768 cubed 9.4 (6.5), 64 x 8192 x 8192 46 (22).  Over 60
// random sizes all three choices were timed: the one taken costs 2 % more than
// the fastest on average, 29 % at most (1526 x 462 x 1372: tiles 12.5 us, 9.7).
inline int64_t product_few_ns(int64_t stream, int64_t other, int64_t k) {
    const int64_t t = product_few_rows(other), groups = product_few_groups(stream, other);
    const int64_t share = groups > kProductCus ? groups * 16 / kProductCus : 16;  // of a CU, in sixteenths
    const int64_t work = share * (1 + t) * k / (t <= 2 ? 70 : 40), read = (stream + other) * k / 4500;
    return 2700 + (work > read ? work : read);
}

// In small tiles: 4 us, 0.35 for a block of 128 k, 3 for a split, or memory's rate.
inline int64_t product_small_ns(int64_t m, int64_t n, int64_t k) {
    const int64_t tiles = product_small_tiles(m, n), parts = product_split(tiles, k);
    const int64_t work = 350 * ((b8_blocks(k) + parts - 1) / parts) * ((tiles + kProductCus - 1) / kProductCus);
    const int64_t read = (m + n) * k / 4500;
    return 4000 + (work > read ? work : read) + (parts > 1 ? 3000 : 0);
}

// Whether the kernel without LDS takes a size (its grid has to stay one that
// the estimate was fitted to).
inline bool product_few(int64_t m, int64_t n, int64_t k, ProductShape* shape) {
    const int64_t ns_a = product_few_ns(m, n, k), ns_b = product_few_ns(n, m, k);
    *shape = ns_a < ns_b ? kProductFewA : kProductFewB;
    return (ns_a < ns_b ? product_few_groups(m, n) : product_few_groups(n, m)) <= 4 * kProductCus &&
           (ns_a < ns_b ? ns_a : ns_b) < product_small_ns(m, n, k);
}

// Tiles of 256 x 256 past the last full round that are taken in quarters: up
// to one quarter to a CU.
inline int64_t product_rest(int64_t tiles) {
    const int64_t rest = tiles % kProductCus;
    return tiles > kProductCus && rest <= kProductCus / 4 ? rest : 0;
}

// Among the tiles: by the time that the slowest CU takes, in hundredths of a
// 256 x 256 tile's (K = 4096: small 18.8 us of 55 a round, 192 x 256 43; fp32
// out: 33 of 84, 74).  All three measured over 15 sizes between 2048 x 4800 and
// 16384 x 1600: from K = 768 up the choice is the fastest of them or within 8 %
// of it (5333 x 3500 x 768 bf16 31.2 us large, 28.8 medium); at K = 256, where
// loads and stores weigh more than rounds, within 26 % (4096 x 4800 bf16: 23.2
// large, 18.5 medium).
inline ProductShape product_shape(int64_t m, int64_t n, int64_t k, bool exact) {
    ProductShape few;
    if (product_few(m, n, k, &few)) return few;
    const int64_t small = product_small_tiles(m, n);
    if (small <= kProductCus) return kProductSmall;
    const int64_t medium = ((m + 191) / 192) * ((n + 255) / 256), large = product_tiles(m, n);
    const auto rounds = [](int64_t tiles) { return (tiles + kProductCus - 1) / kProductCus; };
    const int64_t cost_small = rounds(small) * 36;
    const int64_t cost_medium = rounds(medium) * 78;
    const int64_t cost_large =
        product_rest(large) > 0 ? large / kProductCus * 100 + (exact ? 35 : 40) : rounds(large) * 100;
    if (cost_large <= cost_medium && cost_large <= cost_small) return kProductLarge;
    return cost_medium <= cost_small ? kProductMedium : kProductSmall;
}

inline int product_parts(int64_t m, int64_t n, int64_t k) {
    ProductShape few;
    return product_few(m, n, k, &few) ? 1 : static_cast<int>(product_split(product_small_tiles(m, n), k));
}

// The parts' sums lie in whole small tiles.
inline int64_t product_part_rows(int64_t m) { return (m + 127) / 128 * 128; }

struct NormArgs {
    const void* x;
    const void* r;  // residual, or null
    void* h;        // null without a residual
    const void* w;
    uint8_t* codes;
    uint8_t* scales;
    float* rstd;
    int64_t rows, x_stride, r_stride, h_stride, codes_stride, scales_stride;
    int32_t cols, type, w_type;
    double eps;
};

struct NormBackArgs {
    const void* dy;
    const void* h;
    const void* dh;  // or null
    void* dx;
    const void* w;
    const float* rstd;
    float* dw;       // or null
    float* part;     // [norm_back_groups][cols]
    int64_t rows, dy_stride, h_stride, dh_stride, dx_stride;
    int32_t cols, type, w_type;
};

struct EncodeArgs {
    const void* x;
    const float* row_mul;  // or null
    const void* col_mul;   // or null
    uint8_t* codes;        // or null
    uint8_t* scales;
    uint8_t* codes_t;      // or null
    uint8_t* scales_t;
    int64_t rows, cols, x_stride, codes_stride, scales_stride, codes_t_stride, scales_t_stride;
    int32_t type, col_type;
    bool tiles;
};

// One operand of a product: scale row of code row r is r >> shift.
struct ProductSide {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;
    uint32_t codes_stride;
    int64_t scales_stride;
    int32_t shift;
};

struct ProductArgs {
    ProductSide a, b;
    const void* add;  // or null
    void* out;
    float* part;      // [parts][part_rows][part_stride]: whole small tiles
    int64_t add_stride, out_stride, part_rows, part_stride;
    int32_t k, type;
};

// Every argument has been validated by the caller, and no operand is empty
// but k.  Each returns ZERO_OK or ZERO_EHIP.
int launch_norm8(const NormArgs& a, void* stream);
int launch_norm8_backward(const NormBackArgs& a, void* stream);
int launch_block8_encode(const EncodeArgs& a, void* stream);
int launch_block8_product(const ProductArgs& a, int parts, void* stream);

}  // namespace zdp
