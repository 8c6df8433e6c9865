"""Calls of the 4-bit product with its epilogue that take each of its forms, with the form that the
plans choose for them as tests/host_forms prints it:
  "vec <nt> <r> <rs> <splits> <slots>"     few tokens: tiles of 16 tokens and weight rows
  "tiles <wide> <splits> <least> <most>"   more: blocks of 32 rows of X to a tile; wide: the
                                           weights in eight bits first
"""

# (tokens, d_out, d_in, group, gated, form): each tile and sharing of waves, with and without splits
FEW = [
    (3, 18, 128, 32, 0, "vec 1 1 1 1 8"),
    (3, 18, 28672, 32, 0, "vec 1 1 1 7 8"),
    (3, 8190, 128, 32, 0, "vec 1 2 1 1 8"),
    (3, 1002, 28672, 32, 0, "vec 1 2 1 7 8"),
    (3, 11010, 128, 32, 0, "vec 1 3 1 1 8"),
    (3, 2050, 28672, 32, 0, "vec 1 4 1 7 8"),
    (19, 18, 128, 32, 0, "vec 2 1 1 1 8"),
    (19, 18, 11008, 32, 0, "vec 2 1 1 3 8"),
    (19, 8190, 128, 32, 0, "vec 2 2 1 1 8"),
    (19, 2050, 11008, -1, 0, "vec 2 2 1 3 8"),
    (19, 11010, 128, 32, 0, "vec 2 3 1 1 8"),
    (19, 16390, 128, 32, 0, "vec 2 4 1 1 8"),
    (37, 18, 128, 32, 0, "vec 3 1 1 1 8"),
    (37, 18, 8192, 32, 0, "vec 3 1 1 4 8"),
    (37, 8190, 128, 32, 0, "vec 3 2 1 1 8"),
    (37, 1002, 11008, 32, 0, "vec 3 2 1 5 8"),
    (37, 22014, 128, 128, 0, "vec 3 2 4 1 8"),
    (37, 11010, 128, 32, 0, "vec 3 3 1 1 8"),
    (37, 2050, 8192, 32, 0, "vec 3 3 1 4 8"),
    (37, 16390, 128, 32, 0, "vec 3 4 1 1 8"),
    (37, 2050, 11008, 32, 0, "vec 3 4 1 6 8"),
    (50, 18, 128, 32, 0, "vec 4 1 1 1 8"),
    (50, 18, 4096, 32, 0, "vec 4 1 1 2 8"),
    (50, 8190, 128, 32, 0, "vec 4 2 1 1 8"),
    (50, 1002, 11008, 32, 0, "vec 4 2 1 6 8"),
    (50, 22014, 128, 64, 0, "vec 4 2 4 1 8"),
    (50, 11010, 128, 32, 0, "vec 4 3 1 1 8"),
    (50, 2050, 8192, 64, 0, "vec 4 3 1 4 8"),
    (50, 16390, 128, 32, 0, "vec 4 4 1 1 8"),
    (50, 2050, 8192, 32, 0, "vec 4 4 1 6 8"),
    (3, 18, 128, 32, 1, "vec 1 2 1 1 8"),
    (3, 18, 11008, 32, 1, "vec 1 2 1 3 8"),
    (3, 11010, 4096, 32, 1, "vec 1 4 1 1 8"),
    (3, 2050, 28672, 32, 1, "vec 1 4 1 7 8"),
    (19, 18, 128, 32, 1, "vec 2 2 1 1 8"),
    (19, 18, 8192, 32, 1, "vec 2 2 1 3 8"),
    (19, 16390, 128, 32, 1, "vec 2 4 1 1 8"),
    (19, 2050, 11008, 32, 1, "vec 2 4 1 5 8"),
    (37, 18, 128, 32, 1, "vec 3 2 1 1 8"),
    (37, 18, 8192, 32, 1, "vec 3 2 1 4 8"),
    (37, 22014, 128, 128, 1, "vec 3 2 4 1 8"),
    (37, 16390, 128, 32, 1, "vec 3 4 1 1 8"),
    (37, 2050, 8192, 32, 1, "vec 3 4 1 4 8"),
    (50, 18, 128, 32, 1, "vec 4 2 1 1 8"),
    (50, 18, 4096, 32, 1, "vec 4 2 1 2 8"),
    (50, 22014, 128, 64, 1, "vec 4 2 4 1 8"),
    (50, 16390, 128, 32, 1, "vec 4 4 1 1 8"),
    (50, 2050, 8192, 32, 1, "vec 4 4 1 6 8"),
]
# past 12288 weight rows up to 16 tokens take two tiles of rows and four slots
FEW += [(m, 12290, 352 if g in (32, -1) else 384, g, gated, "vec 1 2 1 1 4")
        for m in (2, 16) for g in (32, 64, 128, -1) for gated in (0, 1)]

# tiles of three to eight blocks, for every group size (k not whole chunks where that can be)
TILES = [(m, n, {32: 160, 64: 192, 128: 256, -1: 160}[g], g, gated, form)
         for g in (32, 64, 128, -1) for gated in (0, 1)
         for m, n, form in ((65, 22014, "tiles 0 1 3 3"), (210, 16382, "tiles 0 1 3 4"), (577, 8190, "tiles 0 1 4 5"),
                            (326, 16382, "tiles 0 1 5 6"), (413, 16382, "tiles 0 1 6 7"),
                            (483, 22014, "tiles 0 1 8 8") if g == 32 else (962, 8190, "tiles 0 1 7 8"))]
TILES += [(100, 130, 4128 if g in (32, -1) else 4096, g, gated, "tiles 0 8 1 1")
          for g in (32, 64, 128, -1) for gated in (0, 1)]
# the weights in eight bits first, for every group size
WIDE = [(1355, 11006, {32: 672, 64: 704, 128: 640, -1: 672}[g], g, gated, "tiles 1 1 3 4")
        for g in (32, 64, 128, -1) for gated in (0, 1)]
WIDE += [(471, 4098, 2048, 32, 0, "tiles 1 1 1 1"), (645, 22014, 544, 32, 1, "tiles 1 1 1 2"),
         (647, 253, 28672, 32, 0, "tiles 1 8 1 1"), (647, 254, 28672, 32, 1, "tiles 1 8 1 1")]
