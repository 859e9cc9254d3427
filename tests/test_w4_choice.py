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
