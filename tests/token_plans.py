"""Shapes of the token-scaled GEMM by the kernel that runs them, as the library's
plan function says it.  test_token_plan_cpu.py checks every line and that every
kernel that is built has one; the GPU tests run them."""
LARGE, SMALL_M = (256, 256), (0, 0)

# (M, N, K, packed) -> tile, split_k, parts: one token to many, K from 16 on, with
# and without a tail
SHAPES = {
    (1, 16, 16, False): (SMALL_M, 1, 1),
    (1, 4608, 7168, False): ((16, 128), 4, 1),
    (7, 130, 272, False): (SMALL_M, 1, 1),
    (32, 300, 144, False): (SMALL_M, 1, 1),
    (33, 1, 16, False): ((16, 128), 1, 1),
    (48, 256, 384, True): ((16, 128), 1, 1),
    (100, 256, 2064, False): ((16, 128), 8, 1),
    (36, 66, 4096, True): ((16, 128), 16, 1),
    (354, 3939, 352, False): ((64, 64), 1, 1),
    (2075, 133, 256, True): ((64, 64), 1, 1),
    (179, 779, 2272, False): ((64, 64), 4, 1),
    (131, 6634, 944, False): ((64, 128), 1, 1),
    (48, 4608, 7168, False): ((64, 64), 2, 1),
    (129, 5521, 1152, True): ((64, 128), 1, 1),
    (1551, 2087, 848, False): ((128, 128), 1, 1),
    (394, 4750, 384, True): ((128, 128), 1, 1),
    (202, 4210, 5376, False): ((64, 128), 1, 1),
    (66, 2051, 10112, True): ((64, 64), 2, 1),
    (2568, 3090, 64, False): ((64, 64), 1, 1),
    (2717, 1417, 112, False): ((64, 64), 1, 1),
    (4000, 4200, 16, False): (LARGE, 1, 4),
    (2568, 3090, 1040, False): (LARGE, 1, 1),
    (2403, 3329, 128, True): ((64, 64), 1, 1),
    (2695, 1423, 384, True): ((64, 64), 1, 1),
    (5000, 3600, 1024, True): (LARGE, 1, 4),
    (772, 4997, 128, False): (LARGE, 1, 2),
    (1100, 4997, 144, False): (LARGE, 1, 2),
    (772, 4997, 128, True): (LARGE, 1, 2),
    (193, 4292, 7296, False): ((128, 128), 2, 1),
    (193, 4292, 7296, True): ((128, 128), 2, 1),
    (4867, 2476, 128, True): (LARGE, 1, 1),
}
