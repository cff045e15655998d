"""Sizes that take every kernel of the W8A8 products into its loop over K, each
with the kernel it is for.

K has more steps than the kernel has stages under way, and some to spare, so
that stages are refilled and the ring wraps; an odd and an even number of them,
with a remainder of K behind the last whole step and without one."""
import ctypes
from collections import namedtuple

import bit_weight_only_pack_amd._lib as _lib

# stream: 1 for the streaming kernels, 0 for tiles; splits: workgroups that share K
Kernel = namedtuple("Kernel", "stream rows channels waves splits")


def choice(rows, N, K, E=0, gathered=0):
    """The kernel that a product of these sizes takes."""
    fn = _lib.lib().lowbit_internal_w8a8_choice
    fn.restype, fn.argtypes = None, [ctypes.c_int] * 5 + [ctypes.c_void_p]
    out = (ctypes.c_int * 5)()
    fn(E, rows, N, K, gathered, ctypes.cast(out, ctypes.c_void_p))
    return Kernel(*out)


DENSE = [   # kernel, (M, N, K)
    (Kernel(1, 8, 16, 8, 1), (1, 300, 7168)), (Kernel(1, 8, 16, 8, 1), (7, 2001, 6936)),
    (Kernel(1, 8, 32, 8, 1), (2, 4505, 5120)), (Kernel(1, 8, 32, 8, 1), (8, 4316, 7208)),
    (Kernel(1, 8, 64, 4, 1), (5, 9283, 4096)), (Kernel(1, 8, 64, 4, 1), (1, 8541, 3880)),
    (Kernel(1, 16, 16, 8, 1), (9, 170, 7168)), (Kernel(1, 16, 16, 8, 1), (16, 1033, 6936)),
    (Kernel(1, 16, 32, 8, 1), (12, 4540, 5120)), (Kernel(1, 16, 32, 8, 1), (10, 4124, 7208)),
    (Kernel(1, 16, 64, 4, 1), (10, 8528, 4096)), (Kernel(1, 16, 64, 4, 1), (16, 8433, 3880)),
    (Kernel(1, 32, 16, 8, 1), (19, 1000, 4096)), (Kernel(1, 32, 16, 8, 1), (31, 2500, 5032)),
    (Kernel(1, 32, 32, 8, 1), (17, 5000, 5120)), (Kernel(1, 32, 32, 8, 1), (32, 4230, 7208)),
    (Kernel(1, 64, 16, 8, 1), (36, 2000, 4096)), (Kernel(1, 64, 16, 8, 1), (64, 3000, 5032)),
    (Kernel(1, 64, 32, 4, 1), (36, 4604, 4096)), (Kernel(1, 64, 32, 4, 1), (63, 4287, 3880)),
    (Kernel(0, 64, 64, 8, 1), (86, 170, 2304)), (Kernel(0, 64, 64, 8, 1), (69, 200, 2648)),
    (Kernel(0, 64, 64, 8, 2), (4179, 16, 7552)), (Kernel(0, 64, 64, 8, 2), (4216, 16, 6432)),
    (Kernel(0, 64, 64, 8, 4), (2071, 17, 6528)), (Kernel(0, 64, 64, 8, 4), (2087, 16, 6184)),
    (Kernel(0, 64, 64, 8, 8), (65, 18, 17408)), (Kernel(0, 64, 64, 8, 8), (70, 66, 17320)),
    (Kernel(0, 64, 64, 4, 1), (77, 9396, 1280)), (Kernel(0, 64, 64, 4, 1), (65, 8892, 1184)),
    (Kernel(0, 64, 64, 4, 2), (20, 17861, 6528)), (Kernel(0, 64, 64, 4, 2), (17, 16876, 6432)),
    (Kernel(0, 64, 64, 4, 4), (18, 17694, 7040)), (Kernel(0, 64, 64, 4, 4), (17, 16631, 5848)),
    (Kernel(0, 64, 64, 4, 8), (21, 17020, 19584)), (Kernel(0, 64, 64, 4, 8), (17, 17012, 17840)),
    (Kernel(0, 128, 128, 4, 1), (325, 9044, 1152)), (Kernel(0, 128, 128, 4, 1), (358, 8234, 1160)),
    (Kernel(0, 128, 128, 4, 2), (4102, 793, 8960)), (Kernel(0, 128, 128, 4, 2), (267, 10773, 7592)),
    (Kernel(0, 128, 128, 4, 4), (4544, 262, 8064)), (Kernel(0, 128, 128, 4, 4), (4114, 263, 8016)),
    (Kernel(0, 128, 256, 8, 1), (582, 6630, 1152)), (Kernel(0, 128, 256, 8, 1), (266, 11113, 1328)),
    (Kernel(0, 128, 256, 8, 2), (74, 17254, 3456)), (Kernel(0, 128, 256, 8, 2), (65, 17652, 3440)),
    (Kernel(0, 128, 256, 8, 4), (85, 9127, 4736)), (Kernel(0, 128, 256, 8, 4), (66, 8426, 3864)),
    (Kernel(0, 128, 256, 8, 8), (66, 5000, 21760)), (Kernel(0, 128, 256, 8, 8), (67, 4420, 18208)),
    (Kernel(0, 256, 256, 4, 1), (1556, 8061, 1152)), (Kernel(0, 256, 256, 4, 1), (1111, 11151, 1192)),
    (Kernel(0, 256, 256, 4, 2), (131, 19091, 15744)), (Kernel(0, 256, 256, 4, 2), (139, 16571, 14320)),
    (Kernel(0, 256, 256, 4, 4), (136, 9240, 18176)), (Kernel(0, 256, 256, 4, 4), (130, 8231, 18072)),
    (Kernel(0, 256, 256, 4, 8), (132, 5642, 38400)), (Kernel(0, 256, 256, 4, 8), (134, 5633, 38496)),
]

# kernel, rows of the experts that have any, (E, N, K): last tiles that are whole, more than half full and less
EXPERTS = [
    (Kernel(1, 16, 32, 2, 1), {0: 9, 1: 8, 5: 33, 7: 17}, (8, 70, 1528)),
    (Kernel(1, 16, 32, 2, 1), {2: 16, 3: 40}, (8, 37, 1152)),
    (Kernel(1, 16, 32, 4, 1), {0: 3, 1: 17, 2: 9}, (3, 70, 7304)),
    (Kernel(1, 16, 32, 4, 1), {0: 36}, (3, 33, 7168)),
    (Kernel(0, 64, 64, 8, 1), {0: 64, 1: 33}, (2, 200, 2432)),
    (Kernel(0, 64, 64, 8, 1), {0: 65, 1: 31, 2: 64}, (3, 130, 2648)),
    (Kernel(0, 64, 64, 4, 1), {e: (64, 1, 0, 17, 33, 9, 2, 5)[e % 8] for e in range(128)}, (128, 67, 1336)),
    (Kernel(0, 64, 64, 4, 1), {e: (0, 40, 7, 16)[e % 4] for e in range(128)}, (128, 65, 1280)),
    (Kernel(0, 128, 128, 4, 1), {0: 128, 1: 64, 2: 65, 3: 129, 4: 192, 5: 193, 7: 75}, (8, 2922, 1152)),
    (Kernel(0, 128, 128, 4, 1), {e: (128, 64, 150, 30, 91)[e % 5] for e in range(100)}, (100, 214, 1352)),
    (Kernel(0, 128, 256, 8, 1), {0: 128, 2: 64, 3: 65, 9: 129, 12: 117}, (40, 1310, 1152)),
    (Kernel(0, 128, 256, 8, 1), {e: (12, 30, 0, 7, 13)[e % 5] for e in range(100)}, (100, 481, 1208)),
    (Kernel(0, 256, 256, 4, 1), {e: (256, 128, 300, 129, 499)[e % 5] for e in range(40)}, (40, 900, 1280)),
    (Kernel(0, 256, 256, 4, 1), {e: (256, 100, 0, 17)[e % 4] for e in range(0, 128)}, (128, 463, 2520)),
]
