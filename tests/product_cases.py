"""Products by expert in every kernel that they can take: the tile's shape, the
depth in parts or not, and how each operand's lines reach LDS.

SHAPES names, for each product and type, sizes that take each shape: groups of
rows that end inside a tile, several tiles each way, a depth of 8 steps and more
(of parts, too) that ends inside a step.  LINES says where the operands lie:
elements from an aligned address, elements between one row and the next.
"""

# (product, bytes of an element, rows, experts, hidden, out): the tile, whether in parts
SHAPES = {
    ("out", 2, 4099, 3, 520, 2056): ("256x256", False),
    ("out", 2, 2111, 3, 8200, 1032): ("256x256", True),
    ("out", 2, 1505, 3, 520, 648): ("128x128", False),
    ("out", 2, 1505, 3, 2056, 648): ("128x128", True),
    ("out", 2, 301, 3, 1032, 200): ("32x64", False),
    ("out", 2, 301, 3, 2056, 200): ("32x64", True),
    ("out", 4, 4099, 3, 264, 520): ("128x128", False),
    ("out", 4, 1505, 3, 776, 648): ("128x128", True),
    ("out", 4, 301, 3, 520, 200): ("32x64", False),
    ("out", 4, 301, 3, 1032, 200): ("32x64", True),
    ("drows", 2, 4099, 3, 2056, 520): ("256x256", False),
    ("drows", 2, 2111, 3, 1032, 8200): ("256x256", True),
    ("drows", 2, 4099, 3, 392, 520): ("128x128", False),
    ("drows", 2, 1505, 3, 392, 4104): ("128x128", True),
    ("drows", 2, 301, 3, 392, 520): ("32x128", False),
    ("drows", 2, 301, 3, 392, 1544): ("32x128", True),
    ("drows", 2, 301, 3, 264, 1288): ("32x64", False),
    ("drows", 2, 301, 3, 264, 2056): ("32x64", True),
    ("drows", 4, 4099, 3, 520, 264): ("128x128", False),
    ("drows", 4, 1505, 3, 648, 1288): ("128x128", True),
    ("drows", 4, 903, 7, 1032, 264): ("32x128", False),
    ("drows", 4, 301, 3, 200, 520): ("32x64", False),
    ("drows", 4, 301, 3, 200, 1032): ("32x64", True),
    ("dweights", 2, 4099, 7, 776, 1288): ("256x256", False),
    ("dweights", 2, 16411, 3, 776, 776): ("256x256", True),
    ("dweights", 2, 4099, 7, 392, 392): ("128x128", False),
    ("dweights", 2, 12301, 3, 392, 392): ("128x128", True),
    ("dweights", 2, 4099, 3, 200, 136): ("32x64", False),
    ("dweights", 2, 8203, 3, 200, 136): ("32x64", True),
    ("dweights", 4, 2111, 7, 392, 648): ("128x128", False),
    ("dweights", 4, 4099, 5, 392, 520): ("128x128", True),
    ("dweights", 4, 2111, 3, 200, 136): ("32x64", False),
    ("dweights", 4, 4099, 3, 200, 136): ("32x64", True),
}

# (shift, extra of a row) of the first operand and of the second; whether each goes straight
# into LDS in bf16, for which lines have to lie at 4-byte addresses.  The weights are dense, so
# they have no extra.
LINES = {
    (0, 6, 0, 2): "tt", (1, 0, 2, 0): "ft", (2, 0, 1, 6): "tf", (0, 3, 1, 0): "ff",
}


def cases():
    """(sizes, lines) of every case."""
    return [(s, l) for s in SHAPES for l in LINES if s[1] == 2 or l == (0, 6, 0, 2)]


def kernel(sizes, lines):
    """What a case takes: (product, bytes, lines, tile, parts).  Large tiles have the
    straight form alone."""
    tile, parts = SHAPES[sizes]
    how = LINES[lines]
    return (sizes[0], sizes[1], how, "128x128" if how != "tt" and tile == "256x256" else tile, parts)


def widths(kind, hidden, out):
    """Elements in a row of the first operand, and of the second where it is not the
    weights."""
    return (hidden if kind == "out" else out), (hidden if kind == "dweights" else None)


def groups(rows, experts):
    """Uneven rows for `experts` experts that leave 3 rows behind: about half for the
    first, one row and none among the others'."""
    first = rows // 2 + 5
    some = [first, 1, *([0] if experts > 3 else [])]
    left, more = rows - 3 - sum(some), experts - len(some)
    rest = [left // more + (7 if i % 2 else -7) for i in range(more)]
    rest[-1] += left - sum(rest)
    return some + rest
