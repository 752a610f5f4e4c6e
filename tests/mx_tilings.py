"""Sizes that reach each tiling of the MXFP4 products, at their edges: ragged rows, columns and inner dimensions, odd
row strides, experts without rows first, last and side by side, and more tiles than the persistent grid has
workgroups. Not a test module; tests/test_mx_tilings.py checks that the sizes do reach what they are listed under."""

from __future__ import annotations

# name -> place in kTilings, and tile rows, columns and LDS stages
TILINGS = {"stream": (0, 32, 32, 0), "64x64": (1, 64, 64, 3), "64x128": (2, 64, 128, 3), "128x128 deep": (3, 128, 128, 3),
           "128x128": (3, 128, 128, 2), "128x256": (4, 128, 256, 2), "256x256": (5, 256, 256, 2)}

# (tiling, several tiles to a workgroup, m, n, k)
DENSE = [
    ("stream", False, 70, 333, 600),
    ("64x64", False, 33, 4107, 1057), ("64x64", True, 8515, 387, 300),
    ("64x128", False, 200, 5001, 1057), ("64x128", True, 919, 8279, 300),
    ("128x128 deep", False, 1301, 2701, 600),
    ("128x128", False, 8210, 769, 300), ("128x128", True, 4099, 2301, 1400),
    ("128x256", False, 513, 7365, 300), ("128x256", True, 6007, 4001, 520),
    ("256x256", False, 2501, 5001, 300), ("256x256", True, 5001, 8201, 600),
]

# (tiling, several, rows the buffers hold, n, k, rows of each expert)
ROWS = [
    ("stream", False, 90, 301, 600, [0, 40, 0, 0, 3, 33, 0, 0]),
    ("64x64", False, 8, 1025, 600, [0, 1, 0, 0, 1, 1, 0, 0]), ("64x64", True, 689, 2673, 600, [0, 8, 611, 0, 65, 0]),
    ("64x128", False, 285, 4949, 600, [0, 70, 60, 0, 2, 0]), ("64x128", True, 285, 4949, 300, [0, 134, 144, 0, 2, 0]),
    ("128x128 deep", False, 773, 2913, 600, [0, 145, 44, 0, 3, 0]),
    ("128x128 deep", True, 815, 3599, 300, [0, 1, 259, 0, 550, 0]),
    ("128x128", False, 3193, 4241, 300, [0, 8, 0, 0, 802, 784, 0, 0]),
    ("128x128", True, 4309, 2617, 300, [0, 7, 0, 0, 12, 4285, 0, 0]),
    ("128x256", False, 1053, 4277, 600, [0, 61, 0, 0, 461, 2, 0, 0]),
    ("128x256", True, 1482, 4917, 300, [0, 48, 0, 0, 1188, 241, 0, 0]),
    ("256x256", False, 4885, 4107, 300, [0, 64, 936, 0, 220, 0]),
    ("256x256", True, 4618, 4573, 300, [0, 3516, 1, 0, 1096, 0]),
]

# (tiling, several, m, n, rows of each expert; its padded rows are the inner dimension, with 256 more behind the last)
WGRAD = [
    ("stream", False, 70, 65, [0, 280, 0, 0, 2, 700, 0, 0]),
    ("64x64", False, 161, 323, [0, 7, 0, 0, 1, 336, 0, 0]), ("64x64", True, 34, 4121, [0, 346, 0, 0, 71, 32, 0, 0]),
    ("64x128", False, 292, 385, [0, 59, 0, 0, 8, 333, 0, 0]), ("64x128", True, 129, 2049, [0, 13, 0, 0, 4, 700, 0, 0]),
    ("128x128 deep", False, 258, 771, [0, 26, 0, 0, 188, 293, 0, 0]),
    ("128x128", False, 2062, 259, [0, 280, 0, 0, 2, 39, 0, 0]), ("128x128", True, 3462, 261, [0, 700, 0, 0, 359, 53, 0, 0]),
    ("128x256", False, 3165, 129, [0, 22, 0, 0, 276, 1, 0, 0]), ("128x256", True, 2563, 541, [0, 436, 0, 0, 107, 600, 0, 0]),
    ("256x256", False, 3088, 389, [0, 1, 0, 0, 290, 31, 0, 0]), ("256x256", True, 4783, 641, [0, 406, 0, 0, 211, 700, 0, 0]),
]

# (tiling, m, n) of gradients of four experts over 1024 rows, of which some or all have none
WGRAD_FEW = [("stream", 161, 323), ("64x64", 200, 800), ("64x128", 300, 1500), ("128x128 deep", 580, 771),
             ("128x128", 2300, 780), ("128x256", 3088, 389), ("256x256", 4100, 700)]


def padded(counts, pad):
    """Offsets of experts whose rows are padded to a multiple of pad."""
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // pad) * pad)
    return off


def workgroups(mode, name):
    """The persistent grid: as many workgroups as fit 256 CUs by LDS (mode: 0 dense, 1 rows, 2 weight gradients)."""
    _, bm, bn, stages = TILINGS[name]
    stage = (bm + bn) * 128 + (max(bm, 128) + max(bn, 128)) * 8
    return 256 * (160 * 1024 // (stage * stages + (4096 if mode else 0)))


def tiles(name, rows, n, groups=1):
    _, bm, bn, _ = TILINGS[name]
    return groups * sum(-(-r // bm) for r in rows) * -(-n // bn)
