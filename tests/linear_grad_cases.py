"""Products (rows, in, out) of tests/test_gpu_linear_grad_tiles.py: for either gradient,
dz W (form 1, depth out) and dz' x (form 2, depth rows), every tile side, split along the
depth or not, every remainder of the rings of panels, and odd edges."""
# by type: (P, Q) of a gradient's product whose unsplit tiles have this side, and the
# panels of 128 bytes along its depth
PRODUCTS = {("bf16", 64): ((200, 136), (1, 2, 3, 4, 5)), ("f16", 64): ((136, 200), (1, 2, 3, 4, 5)), ("f32", 64): ((72, 136), (1, 2, 3, 4, 5)),
            ("bf16", 128): ((2048, 2048), (4, 5, 6, 7, 9)), ("f16", 128): ((2048, 2048), (4, 5, 6, 7, 9)),
            ("f32", 128): ((464, 8160), (18, 19, 20)),
            ("bf16", 256): ((4096, 4096), (1, 2, 3, 4, 5, 6, 7, 8)), ("f16", 256): ((4096, 4096), (1, 2, 3, 4, 5, 6, 7, 8))}
# odd sides, a depth that ends inside a panel or a chunk
EDGES = {("bf16", 64): (203, 133, 147), ("f16", 64): (131, 203, 197), ("f32", 64): (75, 130, 77), ("bf16", 128): (2043, 2041, 445),
         ("f16", 128): (2046, 2047, 325), ("f32", 128): (467, 8155, 623), ("bf16", 256): (4093, 4091, 325), ("f16", 256): (4090, 4095, 203)}
# deep ones, in pieces
SPLIT = {("bf16", 64): (48, 40, 8192), ("f16", 64): (72, 136, 9001), ("f32", 64): (8, 40, 4100), ("bf16", 128): (1000, 1000, 11365),
         ("f16", 128): (1000, 997, 11360), ("f32", 128): (1000, 1000, 16203), ("bf16", 256): (4090, 2043, 11360), ("f16", 256): (4088, 2043, 11365)}


def shape_of(form, p, q, depth):
    """(rows, in, out) whose gradient of this form is a product of P x Q elements."""
    return (q, p, depth) if form == 1 else (depth, p, q)


def cases():
    """(form, kind, side, split, (P, Q, depth))"""
    for form in (1, 2):
        for (kind, side), ((p, q), panels) in PRODUCTS.items():
            for n in panels:
                yield form, kind, side, False, (p, q, n * (32 if kind == "f32" else 64))
        for (kind, side), s in EDGES.items():
            yield form, kind, side, False, s
        for (kind, side), s in SPLIT.items():
            yield form, kind, side, True, s
