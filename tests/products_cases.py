"""Cases of the products of E4M3 and bf16 rows, each made for a kernel: sizes, alignment and the name of the kernel
that the library's rule takes for them.  A CPU test holds the names to the rule and the cases to the kernels that
there are; GPU tests run them.

A case is a dict: `out`, `N`, `K`, `pad` elements behind each row of x and w, `shift` elements in front of the
first; dense ones have `T`, grouped ones `xd`, `sizes` (rows of each expert) and `gather`.  Distances (ldx, ldw, lds,
ldo, w_stride) that are not given are the closest ones."""
from tests import products_rule as rule


def name_of(k):
    """'tiles f8 copied 64x128', 'groups bf16 registers', 'stream f8x 8x16/8 cached': rows x channels of a block,
    a stream's waves."""
    if k.way == "stream":
        return "stream %s %dx%d/%d %s" % (k.unit, k.rows, k.channels, k.last, "past" if k.flag else "cached")
    way = "copied" if k.flag else "registers"
    return "groups %s %s" % (k.unit, way) if k.way == "groups" else "tiles %s %s %dx%d" % (k.unit, way, k.rows, k.channels)


def rows_of_x(c):
    if "T" in c:
        return c["T"]
    M = sum(c["sizes"])
    return max(1, M // 3) if c["gather"] else M


def ld(c, name):
    """A distance in elements."""
    K, N, close = c["K"], c["N"], c["K"] + c.get("pad", 0)
    default = {"ldx": close, "ldw": close, "lds": -(-K // 128), "ldws": -(-K // 128), "ldo": N}
    if name in default:
        return c.get(name, default[name])
    if name == "w_stride":
        return c.get(name, N * ld(c, "ldw"))
    return c.get(name, -(-N // 128) * ld(c, "ldws"))


def kernel(c):
    """The kernel that the rule takes for a case."""
    size = 2 if c.get("xd") == "bf16" else 1
    grouped = "sizes" in c
    copied = rule.copies(ld(c, "ldx") * size, ld(c, "ldw") * size, c.get("shift", 0) * size,
                         ld(c, "w_stride") * size if grouped else 0, rows_of_x(c) if grouped and c["gather"] else 0)
    if grouped:
        return rule.grouped(c["xd"], c["out"], sum(c["sizes"]), c["N"], c["K"], len(c["sizes"]), copied)
    return rule.dense(c["out"], c["T"], c["N"], c["K"], copied)


def _dense(name, out, T, N, K, pad=0, shift=0, **more):
    return dict(more, name=name, out=out, T=T, N=N, K=K, pad=pad, shift=shift)


def _grouped(name, xd, out, sizes, N, K, pad=0, shift=0, gather=True, **more):
    return dict(more, name=name, xd=xd, out=out, sizes=sizes, N=N, K=K, pad=pad, shift=shift, gather=gather)


# Every kernel of the dense product, with K of more than the 64 stages that a wave of a stream or a run of a tile's
# weights' scales takes at once, where it is a tile: stage quads of the rows' scales come again and again.
DENSE = [
    _dense("stream f8x 8x16/16 cached", "bf16", 7, 4000, 9001, 3, 1),
    _dense("stream f8x 8x16/8 cached", "bf16", 5, 5003, 9001, 3),
    _dense("stream f8x 8x16/8 cached", "f32", 8, 4112, 1000),
    _dense("stream f8x 16x16/8 cached", "bf16", 13, 1500, 70000),
    _dense("stream f8x 16x32/8 cached", "bf16", 13, 5003, 9001, 1, 1),
    _dense("stream f8x 16x32/8 cached", "f32", 16, 4100, 70000),
    _dense("stream f8x 32x16/8 cached", "f32", 40, 1500, 9001),
    _dense("stream f8x 32x32/8 cached", "bf16", 25, 5003, 2056, 8),
    _dense("stream f8x 32x32/8 cached", "f32", 48, 3003, 70000),
    _dense("stream f8x 32x32/4 cached", "bf16", 25, 9003, 9001, 3),
    _dense("stream f8x 32x32/4 cached", "f32", 32, 8200, 1111),
    _dense("stream f8x 32x64/4 cached", "f32", 64, 8190, 40000),
    _dense("stream f8 32x16/8 cached", "bf16", 40, 1500, 9001),
    _dense("stream f8 32x32/8 cached", "bf16", 48, 3003, 70000),
    _dense("stream f8 32x64/4 cached", "bf16", 64, 5003, 40000),
    _dense("tiles f8 copied 64x64", "bf16", 333, 1500, 9002, 2),
    _dense("tiles f8 copied 64x128", "bf16", 320, 5003, 9000),
    _dense("tiles f8 copied 64x128", "bf16", 320, 5003, 12288),
    _dense("tiles f8 copied 64x128", "bf16", 320, 5003, 1 << 17),
    _dense("tiles f8 copied 128x128", "bf16", 200, 9003, 9000, 4, 4),
    _dense("tiles f8 copied 128x256", "bf16", 600, 7003, 9001, 3),
    _dense("tiles f8 copied 256x256", "bf16", 1100, 9003, 8321, 15),
    _dense("tiles f8 registers 64x64", "bf16", 333, 5003, 2048, 3, 1),
    _dense("tiles f8 registers 64x64", "bf16", 320, 5003, 12288, 3, 1),
    _dense("tiles f8 registers 64x128", "bf16", 200, 9003, 9000, 3, 1),
    _dense("tiles f8 registers 128x256", "bf16", 600, 7003, 9001, 2),
    _dense("tiles f8x copied 64x64", "f32", 320, 5003, 9000),
    _dense("tiles f8x copied 64x64", "f32", 320, 5003, 1 << 17),
    _dense("tiles f8x copied 64x128", "f32", 1100, 9003, 9002, 2),
    _dense("tiles f8x copied 128x128", "f32", 200, 9003, 12288),
    _dense("tiles f8x copied 128x256", "f32", 600, 7003, 9001, 3, 4),
    _dense("tiles f8x registers 64x64", "f32", 320, 5003, 9000, 3, 1),
    _dense("tiles f8x registers 64x64", "f32", 320, 5003, 12288, 3, 1),
    _dense("tiles f8x registers 128x256", "f32", 1500, 3503, 9001, 2, 3),
]

FEW = [1, 0, 3, 2, 0, 0, 9, 1]
SOME = [9, 0, 17, 5, 8, 0, 20, 1]
MANY = [64, 0, 128, 129, 192, 193, 256, 300, 1]

# Every kernel of the grouped product.
GROUPED = [
    _grouped("stream %s 8x16/8 cached" % unit, xd, out, [3, 0, 12, 1], 250, 1300, 4, 4)
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream %s 16x16/8 cached" % unit, xd, out, [10, 9, 0, 31, 10, 10, 7, 0], 200, 9001, 3)
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream %s 32x32/8 cached" % unit, xd, out, [10, 9, 0, 31, 10, 10, 7, 3] * 2, 300, 1111)
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream %s 16x32/4 cached" % unit, xd, out, FEW * 5, 260, 1300, 1)
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream %s 32x64/4 cached" % unit, xd, out, SOME * 5, 260, 1300, 1, 1, False)
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream %s %s/4 past" % (unit, block), xd, out, sizes * 4, 4003, 4200 if xd == "fp8" else 2100)
    for block, sizes in (("16x32", FEW), ("32x64", SOME))
    for unit, xd, out in (("f8x", "fp8", "bf16"), ("f8x", "fp8", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"))
] + [
    _grouped("stream f8 8x16/8 cached", "fp8", "bf16", [29], 250, 1300),
    _grouped("stream f8 16x16/8 cached", "fp8", "bf16", [60, 0], 1000, 9001, 3),
    _grouped("stream f8 32x32/8 cached", "fp8", "bf16", [90, 0, 1, 40], 700, 1111),
    _grouped("tiles f8 copied 64x128", "fp8", "bf16", [20, 0, 33, 1, 64, 16, 5, 8] * 4, 2603, 9002, 2),
    _grouped("tiles f8 registers 64x128", "fp8", "bf16", MANY, 2603, 9000, 3, 1),
    _grouped("tiles f8 registers 128x256", "fp8", "bf16", [400, 0, 257, 900], 2603, 9001, 2),
    _grouped("groups f8 copied", "fp8", "bf16", MANY, 7303, 9000),
    _grouped("groups f8 copied", "fp8", "bf16", MANY * 4, 2603, 515, 1, 0, False),
    _grouped("tiles f8x copied 64x128", "fp8", "f32", [30, 0, 64, 65, 100], 7303, 9000),
    _grouped("tiles f8x copied 128x256", "fp8", "f32", MANY, 7303, 9000, 4, 4, False),
    _grouped("tiles f8x registers 128x256", "fp8", "f32", MANY, 2603, 9001, 2, 1),
]
for _out in ("bf16", "f32"):
    GROUPED += [
        _grouped("tiles bf16 copied 64x128", "bf16", _out, [30, 0, 64, 65, 10], 7303, 4501, 1),
        _grouped("groups bf16 copied", "bf16", _out, MANY, 7303, 4500),
        _grouped("groups bf16 registers", "bf16", _out, MANY, 7303, 1301, 2, 1, False),
    ]

# Rows far apart in tiles: as far as the load unit's copies reach (2^23 bytes, gathered ones R*ldx up to 2^31; rows'
# scales 2^21, gathered R*lds up to 2^29), and just further, where rows pass through registers; offsets of out that
# pass 2^32 elements.
FAR = [
    _dense("tiles f8 copied 256x256", "bf16", 1024, 9003, 300, ldx=1 << 23, lds=1 << 21, ldo=(1 << 23) + 2),
    _dense("tiles f8x copied 128x256", "f32", 600, 7003, 300, ldx=1 << 23, lds=1 << 21, ldo=(1 << 23) + 1),
    _dense("tiles f8 copied 64x128", "bf16", 320, 5003, 301, ldx=(1 << 23) - 4, ldw=1 << 23, lds=1 << 20, ldo=1 << 24),
    _dense("tiles f8 registers 64x64", "bf16", 320, 5003, 1500, ldx=(1 << 23) + 4, lds=1 << 21, ldo=1 << 24),
    _dense("tiles f8 registers 128x256", "bf16", 600, 7003, 300, 3, 1, ldx=(1 << 25) + 1, lds=1 << 21, ldo=(1 << 23) + 1),
    _grouped("groups f8 copied", "fp8", "bf16", MANY, 7303, 300, ldx=((1 << 31) // 421) & ~3, lds=(1 << 29) // 421,
             ldo=(1 << 22) + 2, w_stride=(1 << 32) + 4, ws_stride=(1 << 30) + 1),
    _grouped("tiles f8x copied 128x256", "fp8", "f32", MANY, 7303, 300, ldx=((1 << 31) // 421) & ~3, lds=(1 << 29) // 421,
             ldo=(1 << 22) + 2, w_stride=(1 << 32) + 4, ws_stride=(1 << 30) + 1),
    _grouped("groups f8 copied", "fp8", "bf16", MANY, 7303, 300, gather=False, ldx=1 << 23, lds=1 << 21, ldo=(1 << 22) + 2),
    _grouped("tiles f8 registers 64x128", "fp8", "bf16", MANY, 2603, 300, ldx=(((1 << 31) // 421) & ~3) + 4, lds=(1 << 29) // 421,
             ldo=(1 << 22) + 1, w_stride=(1 << 32) + 4, ws_stride=(1 << 30) + 1),
]

# Tiles and groups' tiles for the tests of lists that are none, of NaN, of captures and of other streams.
TILES = {
    "dense f8": _dense("tiles f8 copied 64x128", "bf16", 320, 5003, 700),
    "dense f8, registers": _dense("tiles f8 registers 64x64", "bf16", 333, 5003, 2001, 3, 1),
    "dense f8x": _dense("tiles f8x copied 64x64", "f32", 333, 5003, 700),
    "dense f8 stream": _dense("stream f8 32x16/8 cached", "bf16", 80, 1003, 700),
    "tiles f8": _grouped("tiles f8 copied 64x128", "fp8", "bf16", [20, 0, 33, 1, 64, 16, 5, 8] * 4, 2603, 515, 1),
    "tiles f8, registers": _grouped("tiles f8 registers 64x128", "fp8", "bf16", MANY, 2603, 700, 3, 1),
    "tiles f8x": _grouped("tiles f8x copied 128x256", "fp8", "f32", MANY * 4, 2603, 515, 1),
    "groups f8": _grouped("groups f8 copied", "fp8", "bf16", MANY * 4, 2603, 515, 1),
    "tiles bf16": _grouped("tiles bf16 copied 64x128", "bf16", "f32", [20, 0, 33, 1, 64, 66, 45, 8] * 4, 2603, 514),
    "groups bf16": _grouped("groups bf16 copied", "bf16", "bf16", MANY * 4, 2603, 514),
    "stream f8x": _grouped("stream f8x 32x64/4 cached", "fp8", "bf16", SOME * 5, 260, 515, 1),
}


def label(c):
    size = "%dx%dx%d" % (c["T"] if "T" in c else sum(c["sizes"]), c["N"], c["K"])
    return "%s-%s-%s-%d-%d" % (c["name"].replace(" ", "_"), c["out"], size, c.get("pad", 0), c.get("shift", 0))
