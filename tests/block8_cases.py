"""Sizes of products, with the kernel that each is meant for: the GPU tests run
them, and a host test asserts that the library's choice still gives that kernel
(a later rule would otherwise take a kernel's tests away without a word)."""

FEW_B, FEW_A, SMALL, MEDIUM, LARGE = range(5)  # zero_dp_block8.h's ProductShape

# (kernel, quarter tiles of a last round, parts of the sum over k, m, n, k)
PRODUCTS = [
    # 256 x 256: whole tiles, one round exactly; many blocks, the last one short
    (LARGE, False, 1, 4096, 4096, 1300),
    # the last 16 tiles in quarters, whole ones
    (LARGE, True, 1, 4096, 4352, 700),
    # edges cut, in the large tiles and in the quarters; one block, a few, many
    (LARGE, True, 1, 4100, 4100, 128),
    (LARGE, True, 1, 4100, 4100, 700),
    (LARGE, True, 1, 4100, 4100, 1290),
    # a last column of tiles of which a quarter is there
    (LARGE, False, 1, 8192, 1600, 640),
    # 192 x 256: whole; cut, with several words of scales; two blocks, one short
    (MEDIUM, False, 1, 2688, 3328, 1300),
    (MEDIUM, False, 1, 2900, 2900, 1300),
    (MEDIUM, False, 1, 2900, 2900, 1152),
    (MEDIUM, False, 1, 2900, 2900, 140),
    # 128 x 128: whole and in two rounds; cut; a single round; the sum over k split
    (SMALL, False, 1, 2880, 2816, 500),
    (SMALL, False, 1, 2300, 800, 1300),
    (SMALL, False, 1, 2300, 800, 640),
    (SMALL, False, 1, 768, 768, 1300),
    (SMALL, False, 7, 768, 768, 16000),
    (SMALL, False, 6, 300, 200, 9000),
    (SMALL, False, 2, 1400, 1200, 9000),
    # without LDS, 16, 32 and 64 rows of the other operand to a workgroup
    (FEW_B, False, 1, 1, 200, 1600),
    (FEW_B, False, 1, 20, 4000, 300),
    (FEW_B, False, 1, 33, 100, 300),
    (FEW_A, False, 1, 200, 1, 1600),
    (FEW_A, False, 1, 4000, 20, 300),
    (FEW_A, False, 1, 432, 1342, 914),
]

# bytes past a row's end, NaN codes and scales: a last block of which less, or more, than half is there
MASKED = [(SMALL, False, 1, 2300, 800, 140), (SMALL, False, 1, 2300, 800, 200), (MEDIUM, False, 1, 2900, 2900, 140),
          (MEDIUM, False, 1, 2900, 2900, 200), (LARGE, True, 1, 4100, 4100, 140), (LARGE, True, 1, 4100, 4100, 200)]

# no k at all
EMPTY = [(SMALL, False, 1, 2300, 800, 0), (MEDIUM, False, 1, 2900, 2900, 0), (LARGE, True, 1, 4100, 4100, 0)]

# rows 2^23 bytes apart, of one operand taken twice
FAR = [(SMALL, False, 6, 300, 300, 9000), (MEDIUM, False, 1, 2900, 2900, 200), (LARGE, True, 1, 4100, 4100, 200)]
