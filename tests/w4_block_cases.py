"""Cases of the 4-bit products that the choice gives to the block kernel, for its GPU tests; a CPU test asks the choice
and counts which of its instances they run."""

# rows of 16 experts: none, one, around the edges of 16-row subtiles and of every block's height, a hot one
COUNTS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 130, 191, 193, 255, 256, 257, 2001]
FEWER = COUNTS[:-1] + [701]  # for blocks of 192 rows
DENSE = [3801]
# 12 experts of 97 to 130 rows
EVEN = [97, 128, 130, 112, 0, 127, 113, 129, 100, 128, 1, 120]

# name: (rows of each expert, channels, columns, group, rows' type, scales' type, zero points, result's type, SwiGLU)
CASES = {
    "bf16": (COUNTS, 2056, 320, 64, "bf16", "bf16", False, "bf16", False),
    "bf16 G32": (COUNTS, 2056, 352, 32, "bf16", "bf16", False, "f32", False),
    "bf16 SwiGLU": (COUNTS, 2064, 640, 128, "bf16", "bf16", False, "bf16", True),
    "bf16 SwiGLU G32": (COUNTS, 2064, 160, 32, "bf16", "bf16", False, "f32", True),
    "bf16 dense": (DENSE, 4104, 384, 128, "bf16", "bf16", False, "bf16", False),
    "bf16 dense SwiGLU": (DENSE, 4112, 192, 64, "bf16", "bf16", False, "bf16", True),
    "zero points": (FEWER, 2056, 192, 64, "bf16", "bf16", True, "bf16", False),
    "zero points G32": (FEWER, 2056, 96, 32, "bf16", "f32", True, "bf16", False),
    "fp32 scales SwiGLU": (FEWER, 2064, 320, 64, "bf16", "f32", False, "f32", True),
    "zero points SwiGLU G32": (FEWER, 2064, 352, 32, "bf16", "bf16", True, "bf16", True),
    "zero points dense": (DENSE, 4104, 1152, 128, "bf16", "f32", True, "f32", False),
    "zero points even": (EVEN, 8200, 256, 128, "bf16", "bf16", True, "bf16", False),
    "fp32 rows": (COUNTS, 2056, 320, 64, "f32", "bf16", False, "f32", False),
    "fp32 rows G32": (COUNTS, 2056, 352, 32, "f32", "bf16", False, "bf16", False),
    "fp32 rows SwiGLU": (COUNTS, 2064, 192, 64, "f32", "bf16", False, "f32", True),
    "fp32 rows SwiGLU G32": (COUNTS, 2064, 96, 32, "f32", "bf16", False, "f32", True),
    "fp32 rows, zero points": (COUNTS, 2056, 384, 128, "f32", "f32", True, "f32", False),
    "fp32 rows, zero points, G32": (EVEN, 4104, 160, 32, "f32", "bf16", True, "f32", False),
    "fp32 rows, zero points, SwiGLU": (COUNTS, 2064, 320, 64, "f32", "f32", True, "bf16", True),
    "fp32 rows, zero points, SwiGLU G32": (COUNTS, 2064, 352, 32, "f32", "bf16", True, "f32", True),
    "fp32 rows dense": (DENSE, 4104, 256, 64, "f32", "f32", True, "f32", False),
}

# single calls of the tests beside them: (rows, experts, channels, columns, group, grouped, keywords of the choice)
LARGE = {
    "codes past 4 GiB": (10240, 256, 2064, 16384, 128, True, {}),
    "rows past 4 GiB": (140000, 1, 520, 16384, 128, False, {}),
    "results past 4 GiB": (40000, 1, 65536, 32, 32, False, {}),
    "gates": (241 * 9, 1, 4112, 32, 32, False, dict(x="f32", scale="f32", y="f32", swiglu=True)),
    "all of fp32": (2000, 1, 4104, 64, 32, False, dict(x="f32", scale="f32", y="f32")),
    "every code and zero": (2048, 1, 4096, 32, 32, False, dict(scale="f32", zero=True, y="f32")),
    "offsets": (2400, 4, 2056, 64, 32, True, dict(x="f32", y="f32")),
}


def tiles(counts, per):
    """Rows of the row tiles that the experts' rows are cut into."""
    out = []
    for rows in counts:
        nt = -(-rows // per)
        if nt == 0:
            continue
        part = -(-(-(-rows // nt)) // 16) * 16 if len(counts) > 1 else per
        out += [min(part, rows - i * part) for i in range(nt)]
    return out
