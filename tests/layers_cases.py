"""Shapes and inputs of the layer norm and linear layer tests."""
import numpy as np
import torch

# (P, C, N).  Token rows: one element, one token, widths that are no multiple
# of a vector, the widths at which the vectors per thread change, the widest.
LN_ROWS = [(1, 1, 1), (1, 8, 1), (3, 7, 1), (1, 1024, 1), (5, 1023, 1), (2, 2048, 1), (3, 2056, 1), (2, 4099, 1),
           (300, 64, 1), (700, 136, 1), (2, 16384, 1), (1, 16383, 1), (1300, 264, 1),
           # either side of each change of threads or of values a thread
           (5, 255, 1), (5, 256, 1), (5, 257, 1), (3, 2047, 1), (700, 2049, 1), (4, 3001, 1), (2, 4095, 1), (3, 4096, 1),
           (2, 4097, 1), (2, 4104, 1), (2, 8191, 1), (2, 8192, 1), (2, 8193, 1), (2, 8200, 1)]
# Batch columns: one channel, odd batches, whole and ragged tiles of 64 batch
# items, more channels than the widest tile takes, a large batch.
LN_TILES = [(1, 1, 2), (3, 5, 3), (7, 64, 16), (4, 128, 64), (2, 512, 64), (2, 2048, 8), (1, 4096, 4), (1, 16384, 4),
            (1, 5000, 3), (5, 33, 84), (2, 16, 200), (3, 20, 12), (6, 64, 20), (2, 256, 20), (1, 3, 10240),
            (600, 16, 4), (800, 24, 32)]

# (P, Cin, Cout, N)
LIN_TOKENS = [(1, 1, 1, 1), (1, 64, 64, 1), (1, 1000, 1003, 1), (2, 2048, 96, 1), (3, 5, 7, 1), (8, 1000, 1003, 1),
              (9, 128, 64, 1), (17, 8, 8, 1), (64, 256, 512, 1), (130, 72, 136, 1), (129, 257, 255, 1),
              (513, 96, 200, 1), (300, 1024, 264, 1), (1, 4096, 512, 1), (1025, 128, 640, 1), (33, 520, 1024, 1)]
LIN_PIXELS = [(1, 3, 5, 2), (7, 16, 8, 4), (49, 64, 64, 16), (5, 33, 40, 12), (4, 128, 256, 64), (3, 64, 100, 84),
              (10, 24, 24, 8), (3, 40, 48, 32), (2, 16, 16, 200), (6, 65, 63, 16), (1, 128, 128, 96), (30, 64, 128, 24),
              (1, 200, 72, 7), (100, 16, 24, 16), (2, 136, 320, 128), (9, 48, 72, 20), (5, 64, 64, 40),
              (1, 72, 64, 256)]
# enough tiles for tiles of 128 x 128 in one pass or another
LIN_WIDE = [(2500, 40, 1992, 1), (2300, 72, 2047, 1), (1300, 64, 1608, 1), (65, 1992, 2500, 1), (600, 264, 280, 16),
            (300, 264, 520, 32), (150, 260, 264, 64), (150, 264, 296, 80)]
# contractions longer than one accumulator's run, K not split to shorter ones
LIN_LONG = [(1280, 1100, 1000, 1), (1270, 1100, 1003, 1), (90, 1000, 1100, 8)]
# two-CTA tiles of 256 x 256 in one pass at least: output rows that end on, just
# past and just short of 128 and 256, with and without whole vectors to a row,
# sums in one run and in several, K split and whole, copied operands
LIN_PAIR = [(245, 520, 1248, 4), (285, 1049, 803, 4), (238, 656, 760, 8), (300, 585, 739, 8),
            (41, 1936, 1736, 4), (513, 3778, 546, 1), (541, 3728, 552, 1), (596, 531, 3752, 1),
            (181, 1993, 267, 4), (311, 193, 1843, 4), (174, 400, 1952, 4), (332, 152, 2040, 8),
            (134, 2456, 3168, 1), (557, 544, 3736, 1), (144, 3096, 2552, 1), (138, 2553, 3256, 1),
            (2125, 1028, 544, 1), (2308, 136, 3943, 1), (1153, 584, 1884, 1), (572, 582, 3876, 1),
            (18, 2033, 1267, 7), (19, 1160, 1968, 8), (26, 1768, 1376, 7), (1082, 129, 515, 8),
            (264, 583, 3812, 1), (39, 1873, 1211, 7), (257, 960, 2523, 1), (257, 2048, 1184, 1),
            (36, 1184, 1936, 8), (257, 2243, 1152, 1), (1152, 2376, 263, 1), (5, 1505, 1715, 64),
            (478, 1648, 152, 8), (61, 1209, 1923, 8), (2449, 136, 3520, 1), (513, 2352, 1004, 1),
            (2848, 133, 3248, 1), (2570, 3076, 161, 1)]
# up to four tokens: whole and odd rows, more channels than one warp's loads take
LIN_FEW = [(1, 5, 7, 1), (1, 2056, 40, 1), (1, 4099, 33, 1), (2, 7, 5, 1), (2, 1001, 1003, 1), (2, 4104, 24, 1),
           (3, 24, 41, 1), (3, 2048, 96, 1), (3, 4099, 33, 1), (4, 5, 7, 1), (4, 136, 72, 1), (4, 1003, 1001, 1),
           (4, 4096, 520, 1)]
# one channel on a side, one column
LIN_THIN = [(5000, 64, 1, 1), (3000, 1, 65, 1), (2500, 1, 1, 1), (700, 1, 1, 16), (1, 4096, 1, 64), (2, 1, 5, 1000),
            (1, 1, 4099, 4), (40, 300, 1, 3), (1, 3, 2, 2049)]
# either side of the change to 1024 threads a tile
LN_WIDE_TILES = [(2, 1024, 16), (2, 1025, 16), (4, 1500, 16), (4, 2048, 16), (3, 2000, 12), (5, 1100, 12), (2, 1400, 12),
                 (300, 1032, 16)]


def shape_id(s):
    return "x".join(map(str, s))


def bf16(a):
    """a rounded to bfloat16, as fp64."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).double().numpy()


def stored(a, kind):
    """a as the type `kind` holds it, fp64."""
    return bf16(a) if kind == "bf16" else np.ascontiguousarray(a, np.float32).astype(np.float64)


def activations(rng, shape):
    """Unit noise over channel offsets, a few channels much larger than the others."""
    x = rng.standard_normal(shape) * np.where(rng.random((shape[1], 1)) < 0.05, 20.0, 1.0)
    return x + rng.standard_normal((shape[1], 1)) * 3.0
