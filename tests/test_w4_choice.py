"""Which kernel a 4-bit product takes (CPU: the choice is the host's)."""
import itertools

import pytest

from w4_choice import block_rows, choose

TYPES = list(itertools.product(("bf16", "f32"), ("bf16", "f32"), (False, True), ("bf16", "f32")))


@pytest.mark.parametrize("x,scale,zero,y", TYPES)
def test_blocks_are_no_higher_than_their_form(x, scale, zero, y):
    """What is estimated is what runs: a height that the form does not have is not chosen."""
    seen = set()
    for n, E, (M, K), G, swiglu in itertools.product(
            (1, 7, 64, 300, 1024, 2100, 4096, 8192, 65536, 1000000, 8388608), (1, 8, 64, 256),
            ((8, 128), (1024, 2048), (4096, 4096), (2048, 512), (65536, 4096), (16384, 16384)), (32, 128), (False, True)):
        if swiglu and M % 16:
            continue
        c = choose(n, E, M, K, G, E > 1, x, scale, zero, y, swiglu)
        if c[0] == "block":
            assert c[1] % 64 == 0 and 64 <= c[1] <= block_rows(x, scale, zero), (n, E, M, K, G, swiglu, c)
            seen.add(c[1])
        else:
            assert c[1] in ((4, 8) if x == "f32" else (4, 8, 16)) and not (c[2] and K <= 256)
    assert seen == set(range(64, block_rows(x, scale, zero) + 1, 64))


# Blocks where a height counts, bf16 rows and results, even routing: (rows of all experts, experts, channels,
# columns, group, SwiGLU, zero points) and measured times in us for blocks of 64, 128, 192 and 256 rows.
MEASURED = [
    ((2500 * 8, 256, 1024, 2048, 64, True, False), {128: 219, 192: 216, 256: 217}),
    ((3500 * 8, 256, 1024, 2048, 64, True, False), {128: 272, 192: 237, 256: 234}),
    ((4500 * 8, 256, 1024, 2048, 64, True, False), {128: 414, 192: 279, 256: 281}),
    ((5500 * 8, 256, 1024, 2048, 64, True, False), {128: 425, 192: 348, 256: 307}),
    ((6500 * 8, 256, 1024, 2048, 64, True, False), {128: 432, 192: 460, 256: 334}),
    ((7500 * 8, 256, 1024, 2048, 64, True, False), {128: 484, 192: 469, 256: 416}),
    ((8192 * 8, 256, 1024, 2048, 64, True, False), {128: 534, 192: 531, 256: 478}),
    ((300 * 8, 16, 2048, 512, 64, False, False), {64: 33, 128: 26, 192: 32, 256: 32}),
    ((600 * 8, 16, 2048, 512, 64, False, False), {64: 47, 128: 47, 192: 35, 256: 34}),
    ((1200 * 8, 16, 2048, 512, 64, False, False), {64: 74, 128: 67, 192: 61, 256: 73}),
    ((2048 * 8, 256, 2048, 512, 64, False, False), {64: 169, 128: 155, 192: 155, 256: 155}),
    ((6000 * 8, 256, 2048, 512, 64, False, False), {64: 370, 128: 337, 192: 288, 256: 266}),
    ((8192 * 8, 256, 2048, 512, 64, False, False), {64: 489, 128: 415, 192: 406, 256: 380}),
    ((1200 * 8, 64, 1024, 2048, 64, True, True), {64: 151, 128: 121, 192: 84}),
    ((2500 * 8, 64, 1024, 2048, 64, True, True), {64: 291, 128: 189, 192: 163}),
    ((2048, 0, 4096, 4096, 128, False, False), {64: 156, 128: 104, 192: 125, 256: 150}),
    ((4096, 0, 4096, 4096, 128, False, False), {64: 300, 128: 200, 192: 244, 256: 154}),
    ((8192, 0, 4096, 4096, 128, False, False), {64: 594, 128: 391, 192: 364, 256: 299}),
    ((4096, 0, 4096, 4096, 128, False, True), {64: 369, 128: 221, 192: 280}),
    ((8192, 0, 4096, 4096, 128, False, True), {64: 733, 128: 438, 192: 419}),
]


@pytest.mark.parametrize("sizes,times", MEASURED, ids=lambda v: "-".join(map(str, v)) if isinstance(v, tuple) else "")
def test_height_is_the_fastest_measured(sizes, times):
    """Or within 5 % of it."""
    n, E, M, K, G, swiglu, zero = sizes
    kind, rows = choose(n, max(E, 1), M, K, G, E > 0, zero=zero, swiglu=swiglu)
    assert kind == "block" and times[rows] <= 1.05 * min(times.values()), rows


def test_large_counts_are_quickly_estimated():
    """A tenth of a millisecond a call at most, the best of several tries."""
    import time
    choose(8, 8, 64, 64, 64)
    best = 1.0
    for _ in range(7):
        t = time.perf_counter()
        for n in (100000, 1000000, 8388608):
            for E in (1, 2, 8, 256):
                choose(n, E, 4096, 4096, 64)
        best = min(best, time.perf_counter() - t)
    assert best < 12 * 100e-6


def test_block_cases_reach_every_block_instance():
    """The GPU tests' cases go to blocks, and between them run every form, scale grouping, epilogue and number of
    row subtiles per wave."""
    from w4_block_cases import CASES, LARGE, tiles
    seen = set()
    for name, (counts, M, K, G, x, scale, zero, y, swiglu) in CASES.items():
        kind, rows = choose(sum(counts), len(counts), M, K, G, len(counts) > 1, x, scale, zero, y, swiglu)[:2]
        assert kind == "block", name
        for n in tiles(counts, rows):
            seen.add((x, zero or scale == "f32", G == 32, swiglu, -(-n // 64)))
    want = {(x, general, g32, swiglu, n)
            for x in ("bf16", "f32") for general in (False, True) for g32 in (False, True) for swiglu in (False, True)
            for n in range(1, block_rows(x, "bf16", general) // 64 + 1)}
    assert seen == want, sorted(want - seen)
    for name, (n, E, M, K, G, grouped, kw) in LARGE.items():
        assert choose(n, E, M, K, G, grouped, **kw)[0] == "block", name
