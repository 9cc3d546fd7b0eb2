"""Which kernels a block-scaled FP8 call takes: the library's rules on sizes
(launch_gemm, launch_skinny, fp8_linear_in_one, launch_fp8_moe) written down a
second time, so that a test on the CPU can tell whether the GPU tests' shapes
reach every one of them."""

CUS = 256


def up(n, d):
    return -(-n // d)


def linear_in_one(M, K, N):
    groups, rounds = M * up(K, 128), up(N, 32 * CUS)
    return M <= 16 and (groups <= 64 or groups * rounds <= 256)


def _skinny(M, K, N, out, fused):
    tiles = up(N, 16)
    if tiles <= CUS:
        columns, waves = 16, 16
    elif 2 * CUS < tiles <= 4 * CUS:
        columns, waves = 64, 8
    else:
        columns, waves = 32, 16 if fused and up(K, 128) > 8 else 8
    turned = K % 4096 == 0 and up(N, columns) > 1
    return ("few", columns, waves, "one launch" if fused else "codes", "turned" if turned else "straight")


def product(M, K, N, out):
    """The kernel of svdq_fp8_gemm."""
    tiles = lambda n, m: up(N, n) * up(M, m)  # noqa: E731
    wide = out == "f32"
    if M <= (16 if wide else 8) or (M <= 16 and (linear_in_one(M, K, N) or tiles(64, 32) > CUS)):
        return _skinny(M, K, N, out, False)
    for n, m in ((32, 32), (64, 32), (64, 64), (64, 128), (128, 128)):
        if tiles(n, m) <= CUS:
            return ("tile", n, m)
    if wide:
        size = 64 if tiles(64, 64) <= 6 * CUS else 128
        return ("tile, more than one each", size, size)
    big = tiles(256, 256)
    if big < CUS // 2:
        return ("tile, more than one each", 128, 128)
    rest = big % CUS
    if not 0 < rest <= CUS // 2:
        return ("256", "one round" if big <= CUS else "rounds", "whole")
    # the halves of the last tiles, four token tiles at a time across the columns
    tiles_n, tiles_m = up(N, 256), up(M, 256)
    past = False
    for i in range(big - rest, big):
        group = i // (4 * tiles_n)
        gm = min(4, tiles_m - group * 4)
        m0 = (group * 4 + (i - group * 4 * tiles_n) % gm) * 256 + 128
        past |= m0 >= M
    return ("256", "one round" if big <= CUS else "rounds", "divided, a half past M" if past else "divided")


def linear(M, K, N, out):
    """The kernel of svdq_fp8_linear's product."""
    return _skinny(M, K, N, out, True) if linear_in_one(M, K, N) else product(M, K, N, out)


def experts(T, H, I, E, top_k):  # noqa: E741
    """(up kernel, down kernel) of svdq_fp8_moe_layer."""
    pairs = T * top_k
    most = min(E, pairs)
    in_up = T * E <= 256
    slots = (1 if T <= 4 else 0) if in_up else 1 if T <= 4 else 2 if pairs <= 4 * E else 0
    up_kernel = ("choice in it" if in_up else "choice before", slots, "turned" if H % 4096 == 0 else "straight")
    G = up(I, 128)
    cols = 8 if H // 16 <= CUS // 2 and G > 4 and pairs <= 8 * E else 16
    steps, shift = (G * cols + 15) // 16, 0
    while most << shift < 16 and 2 << shift <= steps and (2 << shift) * pairs * cols * 4 <= 32 << 10:
        shift += 1
    slots = 4 if pairs * cols * 4 << shift <= 24 << 10 else 2
    # steps of a unit of the first share of I: more than 4 are more than one batch
    unit = up(up(G, 1 << shift), 16 // cols)
    return up_kernel, (slots, cols, "one batch" if unit <= 4 else "batches")
