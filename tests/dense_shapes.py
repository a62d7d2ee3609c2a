"""Sizes that between them take every way the dense products can run (kernel,
tile, sharing of tiles), for the tests of the choice and of the results."""

# (T, H, I) of the gated block
FFN = [
    (256, 1536, 4096), (700, 1536, 4096), (1024, 2048, 4096), (8189, 1536, 4096),
    (1, 72, 72), (454, 80, 72), (1, 216, 208), (17, 80, 72), (1, 456, 480), (18, 216, 200), (33, 208, 216),
    (1, 4752, 464), (17, 480, 536), (34, 488, 464), (67, 5632, 72), (17, 4640, 488), (5925, 80, 72), (1, 480, 4624),
    (1, 2432, 2376), (2308, 200, 216), (65, 1184, 1352), (17, 512, 4720), (1477, 464, 200), (34, 472, 4824),
    (1, 4816, 200), (17, 2480, 2320), (2434, 144, 936), (344, 1544, 1360), (17, 5056, 200), (1762, 2376, 144),
    (70, 3544, 3616), (1370, 72, 1720), (68, 3112, 4816), (1746, 2224, 72), (65, 3624, 1896), (66, 1808, 7328),
]

# (T, N, K) of the int8 product; on CTA pairs with rows of whole 16 bytes and with others
INT8 = [
    (256, 4096, 4096), (333, 4096, 4096), (203, 1531, 1008), (8189, 8192, 1536),
    (1, 40, 16), (17, 40, 16), (1, 42, 416), (34, 40, 16), (1, 40, 912), (1, 43, 1968), (17, 40, 400), (33, 40, 464),
    (17, 42, 976), (18, 42, 1936), (34, 40, 1936), (5190, 40, 16), (5210, 42, 16), (1, 9424, 400), (1, 4744, 928),
    (1, 2344, 2032), (18, 9812, 432), (17, 4788, 992), (4726, 43, 416), (17, 2553, 2000), (2329, 48, 1024),
    (33, 2588, 2048), (6372, 43, 1104), (1541, 15939, 16), (4856, 48, 1840), (5324, 47, 1840), (3156, 41, 5776),
    (3703, 48, 4272), (137, 4583, 2448), (4329, 144, 2480), (67, 3760, 6464), (68, 6932, 3520), (76, 3838, 6496),
]


def ways_ffn(T, H, I):
    from group_limited_routed_moe_b200 import moe
    return {(p, *moe.dense_plan(p, T, I, H)) for p in moe.PRODUCTS if p != "int8"}


def ways_int8(T, N, K):
    """With whether rows of the output are whole 16 bytes, which CTA pairs store
    in another way."""
    from group_limited_routed_moe_b200 import moe
    plan = moe.dense_plan("int8", T, N, K)
    return {("int8", *plan, N % 8 == 0 if plan[0] == "pairs" else None)}


def uncovered(sizes=40_000, seed=1):
    """Ways that sizes spread over the range take and none of the lists does."""
    import math
    import random
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    covered = set().union(*(ways_ffn(*s) for s in FFN), *(ways_int8(*s) for s in INT8))
    found = set()
    for _ in range(sizes):
        T = log(1, 9000)
        found |= ways_ffn(T, 8 * log(9, 1024), 8 * log(9, 1024))
        found |= ways_int8(T, log(40, 16384), 16 * log(1, 512))
    return found - covered
