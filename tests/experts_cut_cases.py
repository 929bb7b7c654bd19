"""Sizes whose last round of 256-row tiles is cut into halves, with rows in both: (product, (R, n, H, I)), rows as
experts_plan_cases.spread has them, on 256 CUs.  There are whole tiles and a full round before the cut, k ends inside a
stage, and the halves have an even number of stages and an odd one."""

CUTS = [("gateup", (2741, 8, 200, 2320)), ("gateup", (7426, 18, 136, 808)),
        ("down", (7491, 18, 1640, 224)), ("down", (8032, 18, 1632, 136)),
        ("dh", (5386, 8, 200, 2328)), ("dh", (8137, 18, 144, 1592)),
        ("dx", (8007, 18, 1584, 72)), ("dx", (10524, 54, 872, 72))]
