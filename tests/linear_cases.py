"""Products (rows, in, out) of tests/test_gpu_linear_tiles.py that together reach every
tile side, split along the depth or not, and every remainder of the rings of panels."""

# by form: x W' of (rows, in, out), dz W and dz' x of the same three
PANELS = ([("bf16", (70, 64 * p, 75)) for p in range(1, 9)] + [("f32", (70, 32 * p, 75)) for p in (1, 2, 3, 4, 7)]
          + [("f16", (2048, 64 * p, 2048)) for p in range(4, 11)] + [("bf16", (4096, 64 * p, 4096)) for p in range(1, 8)]
          + [("bf16", (4096, 64 * 5 + 8, 4096)), ("f16", (2048, 64 * 7 - 8, 2040)), ("f32", (2048, 32 * 9 + 4, 2048))])
# (kind, out-of-x W' shape): deep ones that are split, on each tile side
SPLIT = [("bf16", (40, 8192, 48)), ("bf16", (456, 82448, 72)), ("f16", (136, 164112, 1000)), ("f32", (8, 4096, 8)),
         ("f32", (72, 11360, 8184))]
LARGE = [("bf16", (2500, 130, 4200)), ("bf16", (1140, 1272, 2904)), ("f32", (8160, 488, 464))]


def forms(shape):
    """(P, Q, depth) of the three products of (rows, in, out)."""
    rows, inner, outer = shape
    return [(outer, rows, inner), (inner, rows, outer), (inner, outer, rows)]

# x W' with odd rows and edges, by the tile side that it runs on
EDGES = [(64, "f32", (130, 192, 75)), (64, "bf16", (130, 192, 75)), (128, "f16", (2041, 448, 2043)), (128, "f32", (8155, 484, 467)),
         (256, "bf16", (4091, 320, 4093))]
