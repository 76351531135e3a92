"""Shapes of linear attention that get a plan of several segments, and the plans they get:
the tests on the CPU hold the plans, those on the GPU the results."""

# batch, steps, heads, key and value heads, key and value size, type, backward; whole (batch, head)
# pairs, steps of a segment, segments.  Every width and number of columns of a
# workgroup, with pairs walked whole beside pairs in segments, and all in segments.
PLANS = [
    (2, 700, 388, 194, 64, 64, "bf16", False, (768, 192, 4)),
    (2, 700, 260, 260, 40, 128, "bf16", False, (512, 192, 4)),
    (2, 700, 260, 130, 128, 64, "bf16", False, (512, 192, 4)),
    (2, 700, 132, 132, 128, 128, "bf16", False, (256, 192, 4)),
    (2, 700, 132, 66, 120, 99, "bf16", False, (256, 192, 4)),
    (2, 700, 68, 34, 128, 200, "bf16", False, (128, 192, 4)),
    (2, 520, 132, 66, 256, 64, "bf16", False, (256, 192, 3)),
    (2, 520, 68, 68, 256, 256, "bf16", False, (128, 192, 3)),
    (2, 700, 132, 132, 64, 64, "bf16", True, (256, 192, 4)),
    (2, 700, 43, 43, 64, 128, "bf16", True, (85, 192, 4)),
    (2, 700, 43, 43, 128, 33, "bf16", True, (85, 192, 4)),
    (2, 700, 43, 43, 128, 128, "bf16", True, (85, 192, 4)),
    (2, 520, 22, 11, 128, 256, "bf16", True, (42, 192, 3)),
    (2, 520, 22, 11, 255, 64, "bf16", True, (42, 192, 3)),
    (2, 520, 22, 22, 256, 256, "bf16", True, (42, 192, 3)),
    (2, 520, 388, 194, 64, 64, "f32", False, (768, 192, 3)),
    (2, 520, 68, 68, 256, 256, "f32", False, (128, 192, 3)),
    (2, 520, 132, 66, 64, 64, "f32", True, (256, 192, 3)),
    (2, 520, 88, 88, 128, 70, "f32", True, (170, 192, 3)),
    (2, 520, 22, 22, 64, 256, "f32", True, (42, 192, 3)),
    (2, 520, 22, 11, 256, 130, "f32", True, (42, 192, 3)),
]
