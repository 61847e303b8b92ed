"""Which kernel and shape a call takes: the launchers' rules over again, with their tables read from the sources, so that a
test can say whether every one of them is reached by some size."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_03_amd", "csrc")
CUS = 256


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _table(text, name):
    """[[number, ...], ...] of a constexpr array of structures."""
    body = re.search(name + r"\[\] = (\{.*?\});", text, re.S).group(1)
    return [[float(v) for v in row.split(",")] for row in re.findall(r"\{([^{}]+)\}", body)]


def _number(text, name):
    return eval(re.search(r"constexpr \w+ " + name + r" = ([\d <*+]+);", text).group(1))


_INT8 = _source("dense_int8.hip")
_ROWS = _source("rows.hip")
ROWS_SHAPES = _table(_INT8, "kRowsShapes")
TILE_COSTS = _table(_INT8, "kTileCosts")
UNIT_SHAPES = _table(_source("dense.hpp"), "kUnitShapes")
VERY_FEW_ROWS = _number(_INT8, "kVeryFewRows")
FEW_WAVES = _number(_ROWS, "kFewWaves")
L2_BYTES = _number(_ROWS, "kL2Bytes")


def up(a, b):
    return -(-a // b)


def _stream_shape(M, pairs, Kp):
    """(row tiles, column halves) of dense_stream_kernel, rows on 16 bytes."""
    best = None
    for mt, ct in UNIT_SHAPES:
        rows = int(mt) * 16
        if rows > 16 and M <= rows / 2:
            continue
        groups = pairs * (4 // int(ct)) * up(M, rows)
        ns = up(groups, CUS) * (min(rows, M) + int(ct) * 16) * Kp * 2 / 37.0 + 2000.0
        if best is None or ns < best[0]:
            best = (ns, (int(mt), int(ct)))
    return best[1]


def int8_product(M, N, K, gated=False, vec=True, rows16=True):
    """The kernel of an int8 product whose rows lie within a buffer's reach, with what tells its variants apart: rows of C and
    R that move by four (vec), whether K ends inside 16 bytes, whether there is an up weight.  And the expected time, ns."""
    pairs, Kp = up(N, 32 if gated else 64), up(K, 128) * 64
    part = K % 16 != 0
    rows = None
    for i, (mt, ct, ends, rate, rate_any, least) in enumerate(ROWS_SHAPES):
        n, ct = int(mt) * 16, int(ct)
        if (not rows16 and rate_any == 0) or up(M, n) > 65535:
            continue
        each = up(pairs * (4 // ct) * up(M, n), CUS)
        size = (min(n, M) + ct * 16) * 2.0 * Kp
        ns = 2300.0 + ends + size / (80 if rows16 else 65) + (each - 1) * max(size / (rate if rows16 else rate_any) + ends / 8, least)
        if rows is None or ns < rows[0]:
            rows = (ns, (int(mt), ct))
    if not rows16:
        return ("rows", rows[1], "any", vec, gated), rows[0]
    if M <= VERY_FEW_ROWS and not part:
        return ("stream", (1, 1) if _stream_shape(M, pairs, Kp) == (1, 1) else (1, 2), gated), 0.0
    tile = None
    for i, (ends, whole) in enumerate(TILE_COSTS):
        tiles = up(M, (i + 1) * 32) * up(pairs, 4)
        each = up(tiles, CUS)
        if tiles >= 1 << 24:
            continue
        ns = 5000.0 + each * (ends + (whole - ends) * Kp / 2048) * (1.15 if each == 1 else 1.0)
        if tile is None or ns < tile[0]:
            tile = (ns, i + 1)
    if tile is not None and tile[0] < rows[0]:
        return ("tile", tile[1], "part" if part else "whole", vec, gated), tile[0]
    return ("rows", rows[1], "part" if part else "whole", vec, gated), rows[0]


def int8_product_kernels():
    """All of them (those of rows far apart are reached by strides, not by sizes)."""
    return ({("stream", s, g) for s in ((1, 1), (1, 2)) for g in (False, True)}
            | {("rows", (int(s[0]), int(s[1])), k, v, g) for s in ROWS_SHAPES for k in ("whole", "part", "any")
               if k != "any" or s[4] > 0 for v in (False, True) for g in (False, True)}
            | {("tile", n + 1, k, v, g) for n in range(len(TILE_COSTS)) for k in ("whole", "part") for v in (False, True)
               for g in (False, True)})


BYTES = {None: 0, "f32": 4, "bf16": 2, "f16": 2}


def rows_kernel(rows, H, x, residual=None, y=None, codes=True, norm=True, want_sum=True):
    """(norm, bytes of x, of the residual, past the caches, threads of a row, groups in registers) of rows_kernel."""
    out = rows * H * ((BYTES[residual] if want_sum else 0) + BYTES[y] + int(codes))
    groups = up(H, 8)
    one, two = up(groups, 64) * 64, up(up(groups, 2), 64) * 64
    if groups <= 64:
        shape = (16 if groups <= 16 else 32 if groups <= 32 else 64, 1)
    elif groups <= 1024 and (rows * (one // 64) <= FEW_WAVES or (not norm and one < 2 * two)):
        shape = (1024, 1)
    elif groups <= 128:
        shape = (64, 2)
    else:
        shape = (1024, 2 if groups <= 2048 else 0)
    return (norm, BYTES[x], BYTES[residual], out > L2_BYTES) + shape


def rows_kernels():
    """All of them.  A norm's rows that the chip holds at once are not so many that their outputs go past the caches."""
    shapes = [(16, 1), (32, 1), (64, 1), (64, 2), (1024, 1), (1024, 2), (1024, 0)]
    return {(norm, x, r, past) + s for norm in (False, True) for x in (2, 4) for r in ((0, 2, 4) if norm else (0,))
            for past in (False, True) for s in shapes if not (norm and past and s == (1024, 1))}
