"""Shapes of the operators around the chunked scan by the launch plan they get
(tests/plan_probe.cpp; held to it by test_layer_plans.py), so that every instance a
large shape runs is also run by a small one."""

# Bz, L, D, N, G, (channels of a workgroup, steps of a segment, segments, whole workgroups)
SCAN_FWD = [
    # one segment, 64 channels wide: two, four, eight and sixteen states in a lane
    (100, 43, 70, 5, 1, (64, 43, 1, 0)),
    (32, 43, 770, 12, 1, (64, 43, 1, 0)),
    (100, 43, 400, 24, 1, (64, 43, 1, 0)),
    (32, 43, 770, 40, 1, (64, 43, 1, 0)),
    # the last tiles halved
    (40, 43, 400, 5, 1, (64, 43, 1, 256)),
    (520, 50, 40, 5, 1, (64, 50, 1, 512)),
    (257, 43, 130, 12, 1, (64, 43, 1, 768)),
    (64, 43, 770, 24, 1, (64, 43, 1, 768)),
    (64, 61, 770, 40, 1, (64, 61, 1, 768)),
    # segments, 64 channels wide
    (40, 300, 200, 5, 1, (64, 40, 8, 0)),
    (40, 300, 200, 12, 1, (64, 40, 8, 0)),
    (24, 300, 240, 12, 2, (64, 40, 8, 0)),
    (1, 500, 770, 16, 1, (64, 16, 32, 0)),
    (32, 700, 200, 24, 1, (64, 88, 8, 0)),
    (64, 300, 40, 64, 1, (64, 40, 8, 0)),
    # long segments, 32 channels wide
    (64, 300, 70, 5, 1, (32, 40, 8, 0)),
    (32, 300, 130, 12, 1, (32, 40, 8, 0)),
    (32, 300, 130, 24, 1, (32, 40, 8, 0)),
    (32, 300, 70, 40, 1, (32, 40, 8, 0)),
]

# Bz, L, D, N, G, (channels of a workgroup, steps of a segment, segments)
SCAN_BWD = [
    # one segment of more than two batches
    (770, 45, 20, 5, 1, (64, 48, 1)),
    (512, 61, 30, 12, 2, (64, 64, 1)),
    (400, 45, 40, 24, 1, (32, 48, 1)),
    (770, 45, 20, 40, 1, (32, 48, 1)),
    # segments of more than two batches, joined by the workgroups themselves
    (64, 200, 20, 5, 1, (64, 24, 9)),
    (100, 400, 20, 12, 1, (64, 40, 10)),
    (100, 200, 40, 24, 1, (32, 40, 5)),
    (100, 200, 40, 40, 1, (32, 40, 5)),
    # and joined by the kernel of its own
    (16, 1000, 20, 5, 1, (64, 24, 42)),
    (6, 700, 130, 12, 1, (64, 24, 30)),
    (6, 700, 70, 24, 1, (32, 24, 30)),
    (6, 700, 70, 40, 1, (32, 24, 30)),
    # the most segments that the workgroups join, and one more
    (2, 384, 20, 12, 1, (64, 16, 24)),
    (2, 388, 20, 12, 1, (64, 16, 25)),
    (2, 384, 20, 24, 1, (32, 16, 24)),
    (2, 388, 20, 24, 1, (32, 16, 25)),
]

# Bz, L, pieces, W, silu, (channels of a thread, steps of a walk forward, backward)
CONV = [
    (200, 45, (20,), 4, True, (4, 8, 4)),
    (150, 41, (260,), 4, False, (4, 8, 8)),       # one step past five walks
    (250, 33, (17, 3), 3, True, (1, 8, 4)),       # one past a forward workgroup's four walks
    (400, 65, (20,), 4, True, (4, 16, 16)),       # one past a workgroup's, forward and backward
    (400, 65, (17, 3), 2, True, (1, 16, 16)),
    (600, 97, (20,), 3, False, (4, 16, 32)),      # one past three walks of the backward
    (600, 97, (9, 5, 2), 4, True, (1, 16, 32)),
    (400, 257, (20,), 4, True, (4, 16, 64)),      # one past a backward workgroup's
    (400, 257, (5, 3), 4, False, (1, 16, 64)),
]


def lengths(Bz, L):
    """Unequal lengths: none, one, inside a walk or a batch of steps, and the whole."""
    return [(0, L, 1, L - 1)[b] if b < 4 else (37 * b + 5) % (L + 1) for b in range(Bz)]
