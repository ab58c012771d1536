"""The library's choice of tiles and of parts of the sum for an 8-bit product, written down once more: tests of a
kernel variant assert with it that their sizes reach that variant, whatever the rates become."""
from __future__ import annotations

# side of a tile: tiles of it that a CU holds, microseconds of a stage alone and shared
RATES = {"linear": {256: (1, 1.6, 1.6), 128: (2, 0.6, 0.55), 64: (4, 0.3, 0.22)},
         "grad": {256: (1, 1.45, 1.45), 128: (2, 0.7, 0.5), 64: (4, 0.41, 0.23)}}
JOIN, PART_BYTES = 2.5, 6e6


def mnk(kind, t, c, r):
    """Sides and depth of the product of a layer with t tokens, c columns (inputs) and r rows (outputs)."""
    return {"linear": (t, r, c), "dgrad": (t, c, r), "wgrad": (r, c, t)}[kind]


def stages(kind, k):
    return -(-k // (128 if kind == "linear" else 64))


def cut(kind, b, t, c, r):
    """(side of the tiles, parts) as the sizes alone decide them."""
    m, n, k = mnk(kind, t, c, r)
    steps, best = stages(kind, k), None
    for tile, (fit, alone, shared) in RATES["linear" if kind == "linear" else "grad"].items():
        tiles = b * -(-m // tile) * -(-n // tile)
        for parts in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64):
            if parts > 1 and steps < 2 * parts:
                break
            rounds, rest = divmod((tiles * parts + 255) // 256, fit)
            us = rounds * max(alone, shared * fit) + (max(alone, shared * rest) if rest else 0)
            us *= (steps + parts - 1) // parts + 1
            if parts > 1:
                us += JOIN + 8 * parts * float(b * m * n) / PART_BYTES
            if best is None or us < best[0]:
                best = (us, tile, parts)
    return best[1:]


def plan(kind, b, t, c, r, aligned=True):
    """(side of the tiles, parts, tiles in all) of a call whose operands go straight into LDS, or do not."""
    tile, parts = cut(kind, b, t, c, r)
    m, n, k = mnk(kind, t, c, r)
    direct = aligned and (k % 16 == 0 if kind == "linear" else k % 8 == 0 if kind == "dgrad" else True)
    if tile == 256 and not (direct and (kind != "linear" or stages(kind, k) >= 4 * parts)):
        tile = 128
    return tile, parts, b * -(-m // tile) * -(-n // tile)
