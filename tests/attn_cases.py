"""Shapes of linear attention that get a plan of several segments, and the plans they get:
the tests on the CPU hold the plans, those on the GPU the results."""

# batch, steps, heads, key and value heads, key and value size, type, backward; whole (batch, head)
# pairs, steps of a segment, segments.  Every width and number of columns of a
# workgroup, with pairs walked whole beside pairs in segments, and all in segments.
PLANS = [
    (2, 520, 388, 194, 64, 64, "bf16", False, (768, 64, 9)),
    (2, 520, 260, 260, 40, 128, "bf16", False, (512, 64, 9)),
    (2, 700, 260, 130, 128, 64, "bf16", False, (512, 64, 11)),
    (2, 1500, 132, 132, 128, 128, "bf16", False, (256, 128, 12)),
    (2, 700, 132, 66, 120, 99, "bf16", False, (256, 64, 11)),
    (2, 520, 68, 34, 128, 200, "bf16", False, (128, 64, 9)),
    (2, 340, 132, 66, 256, 64, "bf16", False, (256, 64, 6)),
    (2, 340, 68, 68, 256, 256, "bf16", False, (128, 64, 6)),
    (2, 520, 132, 132, 64, 64, "bf16", True, (256, 64, 9)),
    (2, 340, 43, 43, 64, 128, "bf16", True, (85, 64, 6)),
    (2, 340, 43, 43, 128, 33, "bf16", True, (85, 64, 6)),
    (2, 1500, 43, 43, 128, 128, "bf16", True, (85, 64, 24)),
    (2, 340, 22, 11, 128, 256, "bf16", True, (42, 64, 6)),
    (2, 340, 22, 11, 255, 64, "bf16", True, (42, 64, 6)),
    (2, 340, 22, 22, 256, 256, "bf16", True, (42, 64, 6)),
    (2, 340, 260, 130, 64, 64, "f32", False, (512, 64, 6)),
    (2, 1000, 132, 132, 64, 128, "f32", False, (256, 64, 16)),
    (2, 700, 132, 66, 99, 60, "f32", False, (256, 64, 11)),
    (2, 700, 132, 132, 128, 128, "f32", False, (256, 64, 11)),
    (2, 520, 68, 68, 256, 256, "f32", False, (128, 64, 9)),
    (2, 340, 88, 44, 64, 64, "f32", True, (170, 64, 6)),
    (2, 520, 43, 43, 128, 70, "f32", True, (85, 64, 9)),
    (2, 340, 22, 22, 64, 256, "f32", True, (42, 64, 6)),
    (2, 340, 22, 11, 256, 130, "f32", True, (42, 64, 6)),
    (2, 700, 6, 3, 128, 128, "bf16", True, (0, 128, 6)),
    (1, 2782, 3, 3, 64, 64, "bf16", False, (0, 128, 22)),
    (2, 700, 6, 3, 256, 64, "f32", False, (0, 64, 11)),
    (1, 2000, 3, 1, 64, 128, "f32", True, (0, 128, 16)),
]
