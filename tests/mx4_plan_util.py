"""Sizes at which the microscaled products and experts take each of their kernels: tests/test_mx4_plan_cpu.py asserts on the
host that they do, tests/test_gpu_mx4_plan.py runs them."""

# (4 bits on both sides, M, N, K, with a workspace): rows and columns of a block, pieces of K. Steps
# go round the four stages; most end inside a round, or inside a step.
BLOCKS = {
    (False, 1025, 11008, 608, False): (256, 256, 1),
    (False, 4096, 4096, 1056, True): (256, 256, 1),
    (False, 1300, 3000, 4128, True): (256, 256, 3),
    (False, 700, 11008, 608, False): (256, 192, 1),
    (False, 3000, 4000, 2080, True): (256, 192, 1),
    (False, 257, 11008, 5024, True): (256, 192, 2),
    (False, 769, 8000, 608, True): (128, 256, 1),
    (False, 2048, 4096, 1056, True): (128, 256, 1),
    (False, 333, 4096, 11008, True): (128, 256, 5),
    (False, 4097, 129, 11008, True): (128, 256, 7),
    (False, 129, 11008, 608, True): (128, 128, 1),
    (False, 1500, 129, 5024, True): (128, 128, 8),
    (False, 100, 300, 1056, False): (64, 128, 1),
    (False, 257, 385, 5024, True): (64, 128, 12),
    (True, 4097, 8000, 416, True): (256, 192, 1),
    (True, 3000, 4000, 2080, True): (256, 192, 1),
    (True, 257, 11008, 11008, True): (256, 192, 2),
    (True, 257, 11008, 4128, True): (256, 128, 1),
    (True, 257, 11008, 3936, False): (256, 128, 1),
    (True, 4097, 385, 11008, True): (256, 128, 3),
    (True, 2048, 4096, 1312, True): (128, 128, 1),
    (True, 1300, 129, 11008, True): (128, 128, 8),
    (True, 100, 300, 608, False): (64, 128, 1),
    (True, 600, 129, 11008, True): (64, 128, 11),
}

# (M, E, top_k, D, F): rows of a tile of the experts, 0 without sorting. Several blocks of columns each, D and F no multiples of
# 64 or 128.
WAYS = {
    (1, 8, 5, 416, 352): 0,
    (40, 16, 2, 416, 352): 8,
    (40, 8, 2, 544, 416): 16,
    (100, 3, 2, 544, 416): 64,
    (300, 4, 4, 288, 608): 64,
    (700, 4, 2, 416, 352): 128,
    (1300, 4, 1, 608, 160): 128,
}
