"""Sizes of the 8-bit product that between them take every way through its dispatch (csrc/matmul_fp8.cu):
test_product_host.py says so of the list, test_gpu_product_paths.py runs it."""

# M, N, K
_TALL = [
    # 32 columns, the blocks of K over 1 to 8 CTAs; the last four: two CTAs an SM
    (150, 20, 130), (6531, 1, 901), (150, 20, 664), (140, 9, 774), (130, 32, 1030), (129, 7, 2050), (200, 30, 11555),
    (300, 24, 9998), (19500, 20, 500), (10119, 5, 1458), (5889, 30, 1056),
    (23600, 5, 6100),
    # 64 columns
    (1000, 50, 300), (6192, 33, 1031), (200, 64, 694), (150, 40, 865), (130, 35, 1107), (140, 34, 2049), (130, 33, 13347),
    (140, 60, 10178),
]
SMALL = _TALL + [(n, m, k) for m, n, k in _TALL] + [
    # 128 columns
    (67, 69, 1), (3090, 136, 1453), (133, 3380, 911), (1813, 133, 1105), (67, 73, 698), (76, 68, 956), (81, 65, 1083),
    (73, 66, 2162), (77, 69, 1302), (66, 80, 11625), (65, 79, 6185), (72, 75, 10015), (67, 102, 8069),
]
# pairs of CTAs: one group of columns of tiles; several, the last one cut
PAIRS = [(1673, 1296, 7), (1300, 4613, 8200), (2600, 2000, 20000)]
# rows of a block of a's and b's scales: a scale for each column of the tile, or one for all
LAYOUTS = [(1, 1), (128, 128)]


def columns_of_a_group(K):
    """Columns of tiles whose rows of b take at most 32 MB (pair_t)."""
    return max(1, (32 << 20) // (-(-K // 128) * 128) // 256)
