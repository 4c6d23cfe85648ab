"""Sizes of the 8-bit product that reach each of its kernels, in each of their
forms, and how to choose among them is checked to do so: (M, N, K, rows of B per
scale, exact sums, A aligned, B aligned) and what the plan has to say of it,
(few rows or tiles, rows, columns, k chunks, more work items than places)."""

ODD, EVEN = False, True


def few(rows, cols, chunks=False, many=False):
    return True, rows, cols, chunks, many


def tile(edge, chunks=False, many=False):
    return False, edge, edge, chunks, many


FAST, EXACT = False, True
CASES = [
    # few rows: every shape, with k chunks and without, aligned, either or both operands not, odd K
    ((1, 8, 272, 128, FAST, EVEN, EVEN), few(16, 16)), ((2, 9, 16608, 1, EXACT, EVEN, EVEN), few(16, 16, True)),
    ((3, 17, 16691, 128, EXACT, EVEN, EVEN), few(16, 16, True)), ((6, 10, 15632, 128, FAST, EVEN, ODD), few(16, 16, True)),
    ((4, 9, 16928, 1, FAST, ODD, EVEN), few(16, 16, True)), ((2, 14, 16816, 128, EXACT, ODD, ODD), few(16, 16, True)),
    ((5, 300, 1000, 1, EXACT, ODD, EVEN), few(16, 16)), ((5, 300, 1001, 128, FAST, EVEN, EVEN), few(16, 16)),
    ((1, 4169, 304, 128, EXACT, EVEN, EVEN), few(16, 32)), ((7, 838, 16080, 1, EXACT, EVEN, EVEN), few(16, 32, True)),
    ((17, 418, 14688, 128, FAST, ODD, EVEN), few(16, 32, True)), ((458, 17, 14482, 1, FAST, EVEN, EVEN), few(16, 32, True)),
    ((6, 1019, 16880, 1, EXACT, ODD, ODD), few(16, 32, True)), ((1, 4319, 262, 1, EXACT, EVEN, EVEN), few(16, 32)),
    ((1, 4385, 288, 1, FAST, EVEN, ODD), few(16, 32)), ((4209, 9, 288, 128, FAST, EVEN, EVEN), few(32, 32)),
    ((1116, 8, 15936, 128, EXACT, EVEN, EVEN), few(32, 32, True)), ((17, 522, 16509, 128, EXACT, EVEN, EVEN), few(32, 32, True)),
    ((17, 538, 16864, 1, FAST, ODD, ODD), few(32, 32, True)), ((19, 674, 12400, 1, EXACT, EVEN, ODD), few(32, 32, True)),
    ((4238, 9, 272, 128, FAST, ODD, EVEN), few(32, 32)), ((4469, 41, 272, 1, FAST, EVEN, EVEN), few(64, 32)),
    ((33, 4292, 320, 128, EXACT, EVEN, EVEN), few(64, 32)), ((1429, 11, 16272, 1, EXACT, EVEN, EVEN), few(64, 32, True)),
    ((33, 597, 14496, 128, EXACT, ODD, EVEN), few(64, 32, True)), ((33, 621, 16720, 1, FAST, ODD, ODD), few(64, 32, True)),
    ((2010, 8, 15602, 1, EXACT, EVEN, EVEN), few(64, 32, True)), ((4539, 33, 268, 1, FAST, EVEN, EVEN), few(64, 32)),
    ((5048, 33, 272, 1, EXACT, ODD, EVEN), few(64, 32)), ((39, 4899, 400, 128, FAST, EVEN, EVEN), few(64, 32)), ((69, 4827, 288, 128, FAST, EVEN, EVEN), few(64, 64)),
    ((250, 2600, 1040, 128, FAST, EVEN, EVEN), few(64, 64)),
    # 128 x 128 tiles, fast
    ((4301, 98, 272, 1, FAST, EVEN, EVEN), tile(128)), ((700, 2930, 2064, 128, FAST, EVEN, EVEN), tile(128)),
    ((1934, 805, 272, 128, FAST, EVEN, ODD), tile(128)), ((4119, 358, 272, 1, FAST, ODD, EVEN), tile(128)),
    ((2235, 689, 257, 128, FAST, EVEN, EVEN), tile(128)), ((5323, 3122, 272, 128, FAST, EVEN, EVEN), tile(128, many=True)),
    ((5496, 2838, 304, 1, FAST, ODD, ODD), tile(128, many=True)), ((18, 2785, 15424, 128, FAST, EVEN, EVEN), tile(128, True)),
    ((300, 500, 16000, 1, FAST, EVEN, EVEN), tile(128, True)), ((73, 1844, 15856, 128, FAST, ODD, EVEN), tile(128, True)),
    ((84, 1372, 16864, 1, FAST, EVEN, ODD), tile(128, True)), ((75, 1641, 16985, 128, FAST, EVEN, EVEN), tile(128, True)),
    # 128 x 128 tiles, exact
    ((227, 4270, 288, 128, EXACT, EVEN, EVEN), tile(128)), ((321, 5883, 272, 128, EXACT, ODD, EVEN), tile(128)),
    ((653, 2980, 272, 128, EXACT, EVEN, ODD), tile(128)), ((532, 3707, 258, 1, EXACT, EVEN, EVEN), tile(128)),
    ((2000, 2030, 1040, 1, EXACT, EVEN, EVEN), tile(128)), ((3973, 2116, 288, 128, EXACT, EVEN, EVEN), tile(128, many=True)),
    ((2315, 3438, 288, 1, EXACT, ODD, EVEN), tile(128, many=True)), ((65, 5965, 3744, 128, EXACT, EVEN, EVEN), tile(128, True)),
    ((401, 707, 16000, 1, EXACT, EVEN, EVEN), tile(128, True)), ((97, 4110, 5460, 128, EXACT, EVEN, EVEN), tile(128, True)),
    # 256 x 256 tiles
    ((2472, 3359, 272, 128, FAST, EVEN, EVEN), tile(256)), ((2437, 3288, 272, 128, FAST, ODD, EVEN), tile(256)),
    ((1834, 4540, 272, 1, FAST, EVEN, ODD), tile(256)), ((3444, 2328, 263, 1, FAST, EVEN, EVEN), tile(256)),
    ((5000, 5200, 1040, 128, FAST, EVEN, EVEN), tile(256, many=True)), ((5300, 5100, 2064, 1, FAST, EVEN, EVEN), tile(256, many=True)),
    ((5951, 4983, 288, 1, FAST, ODD, ODD), tile(256, many=True)), ((4235, 5778, 266, 128, FAST, EVEN, EVEN), tile(256, many=True)),
]
