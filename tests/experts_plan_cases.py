"""Sizes that reach each tiling of the experts' products: (product, tiling, (R, n, H, I)).

A tiling is "edge r half-stages of its LDS ring".  Products over the experts' rows:
  gateup  x [Wg; Wu]^T      down  h Wd^T       dh  dy Wd       dx  dx alone
and grads, dx and the weight gradients of one call: in one launch, or the weight
gradients streamed on 256 CUs ("stream").  Rows, columns and k end inside a tile and a
stage.  That the library plans what is written here is checked without a GPU, so a
change of the plans that leaves a tiling untested shows."""

EXPERTS = [
    ("gateup", "64r10", (1, 1, 8, 8)), ("gateup", "64r5", (40, 40, 8, 400)),
    ("gateup", "256r5", (1600, 8, 152, 3120)), ("gateup", "128r10", (32362, 51, 8, 40)),
    ("gateup", "128r5", (1053, 22, 8, 1392)), ("gateup", "256r5", (93, 69, 1680, 368)),
    ("down", "64r10", (7, 2, 24, 40)), ("down", "64r5", (31, 31, 1224, 8)), ("down", "256r5", (4609, 23, 2248, 136)),
    ("down", "128r10", (3028, 24, 1160, 8)), ("down", "128r5", (32881, 53, 72, 8)),
    ("down", "256r5", (19, 19, 2768, 1896)), ("dh", "64r10", (7, 2, 24, 40)), ("dh", "64r5", (49, 46, 8, 720)),
    ("dh", "256r5", (3609, 18, 136, 2840)), ("dh", "128r10", (31682, 64, 24, 80)),
    ("dh", "128r5", (2892, 62, 8, 968)), ("dh", "256r5", (49, 41, 1784, 1240)), ("dx", "64r10", (7, 2, 24, 40)),
    ("dx", "64r5", (31, 31, 1224, 8)), ("dx", "256r5", (10524, 54, 872, 72)), ("dx", "128r10", (3028, 24, 1160, 8)),
    ("dx", "128r5", (32881, 53, 72, 8)), ("dx", "256r5", (69, 42, 1224, 1088)), ("grads", "64r10", (7, 2, 24, 40)),
    ("grads", "64r5", (49, 46, 8, 208)), ("grads", "128r10", (534, 1, 2048, 400)),
    ("grads", "128r5", (266, 4, 2544, 328)), ("grads", "256r5", (1464, 3, 2712, 200)),
    ("grads", "stream", (68, 58, 8, 296)),
]


def spread(R, n):
    """Rows of each expert: uneven, with an expert without any where there are two and more."""
    if n == 1:
        return [R]
    rows = [0] * n
    for i in range(R):                       # a walk that comes back to some experts more often
        rows[(i * i // 3 + i) % (n - 1)] += 1
    return rows
