"""Sizes at which the products with 4-bit weights run in tiles, and in which: tests/test_experts_tiles_host.py asks the launch plan."""

SMALL, LARGE = 1, 2       # mhc::experts::Shape

# y = x w^T: T, K, N, shape
PRODUCTS = [(300, 264, 4104, SMALL), (700, 200, 1544, SMALL), (1100, 200, 8200, LARGE), (3000, 520, 8200, LARGE)]
# T, k, E, D, F, shape: the projection back, [T k, F] to D columns
DOWN = [(700, 2, 3, 1000, 200, SMALL), (600, 2, 5, 1032, 264, SMALL), (1200, 2, 3, 8200, 72, SMALL), (1700, 2, 3, 8200, 72, LARGE)]
# the gated projection, [T, D] to T k rows of F columns
GLU = [(700, 2, 3, 200, 1000, SMALL), (600, 2, 5, 264, 1032, SMALL), (1200, 2, 3, 72, 8200, LARGE)]
# either: weights whose last expert lies past 2^32 bytes
FAR = [(200, 2, 17, 32768, 16384, SMALL), (2000, 2, 17, 32768, 16384, LARGE)]
# the projection back: results that wait for their sum past 2^32 bytes
FAR_RESULTS = [(40000, 1, 2, 65536, 64, LARGE)]
