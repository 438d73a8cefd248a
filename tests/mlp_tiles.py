"""How the gated block's products are cut into tiles and parts of K, as the
library does it (csrc/gated_mlp.hip: cut_tiles, cut, Sizes, the workspaces), and
the sizes that the GPU tests take so that every kernel runs on every kind of
cut.  test_mlp_tiles_cpu.py holds this against the library's workspaces, and the
sizes against the kinds."""

CUS, STAGE_K, MIN_STAGES, COLUMN_GROUPS = 256, 64, 6, 128
MAX_TILES = (1 << 23) - 1


def _up(n, d):
    return -(-n // d)


def _stage_us(tile, units):
    if tile == 256:
        return 1.5
    if tile == 128:
        return 0.6 if units <= CUS else 1.07
    return 0.25 if units <= CUS else 0.42 if units <= 2 * CUS else 0.58


def _ends_us(tile, wide):
    return {256: (11.0, 20.0), 128: (4.0, 6.0), 64: (3.0, 4.0)}[tile][wide]


def _cut_tiles(tile, tiles, stages, splittable, wide):
    """((tile, tiles that are whole, those in parts, parts), cost)."""
    slots = CUS * {256: 1, 128: 2, 64: 3}[tile]
    full = tiles // slots * slots
    tail = tiles - full
    ends = _ends_us(tile, wide)
    units, rest = (tiles, 0, 1), stages * _stage_us(tile, tail) + ends if tail else 0.0
    if splittable and tail:
        for splits in range(2, min(stages // MIN_STAGES, slots // tail) + 1):
            parts = _up(stages, splits) * _stage_us(tile, tail * splits) + ends + (19.0 if tile == 256 else 6.0)
            if parts < rest:
                units, rest = (full, tail, splits), parts
    return (tile, *units), full // slots * (stages * _stage_us(tile, slots) + ends) + rest


def _cut(extents, stages, splittable, wide, gate=False):
    best = None
    for tile in (256, 128, 64):
        tiles = sum(_up(m, tile) * _up(n, tile // 2 if gate else tile) for m, n in extents)
        if tile < 256 and tiles > MAX_TILES:
            break
        c, cost = _cut_tiles(tile, tiles, stages, splittable, wide)
        if best is None or cost < best[1]:
            best = c, cost
    return best[0]


def cuts(rows, d, h, gate=True, up=True, down=True):
    """(tile, whole tiles, tiles in parts, parts) of each launch of the forward
    and the backward pass; gate, up, down: which of the weights' gradients."""
    hp, per = _up(h, 64) * 64, lambda n: _up(n, STAGE_K)
    r = {}
    if not (rows <= 16 or (rows <= 32 and hp <= 8 * CUS)):
        r["gate"] = _cut([(rows, hp)], per(d), False, False, True)
        r["gate saved"] = _cut([(rows, hp)], per(d), False, True, True)
        r["down"] = _cut([(rows, d)], per(h), True, False)
    r["dhidden"] = _cut([(rows, h)], per(d), False, True)
    r["dx"] = _cut([(rows, d)], 2 * per(h), True, False)
    r["dweights"] = _cut([(h, d)] * (gate + up) + [(d, h)] * down, per(rows), True, False)
    return r


def kind(cut):
    _, whole, parts, splits = cut
    return "whole" if splits == 1 else "mixed" if whole else "parts"


def workspaces(rows, d, h):
    """Bytes of the forward's and the backward's workspace."""
    align = lambda n: (n + 255) & ~255
    dp, hp = _up(d, 64) * 64, _up(h, 64) * 64
    c = cuts(rows, d, h)
    values = lambda cut: cut[2] * cut[3] * cut[0] ** 2 if cut[3] > 1 else 0
    few = "down" not in c
    pad_d, pad_h = d % 8 != 0, h % 8 != 0
    copies = lambda x: align(x * rows * dp * 2), align(h * dp * 2), align(h * dp * 2)
    forward = align(rows * hp * 2)
    if not few:
        forward += (align(rows * dp * 2) + 2 * align(h * dp * 2)) * pad_d + align(d * hp * 2) * pad_h + align(values(c["down"]) * 4)
    part = values(c["dx"])
    if rows >= 2 * MIN_STAGES * STAGE_K - STAGE_K:
        part = max([part] + [values(cuts(rows, d, h, m & 1, m >> 1 & 1, m >> 2)["dweights"]) for m in range(1, 8)])
    backward = (2 * align(rows * hp * 2) + (2 * align(rows * dp * 2) + 2 * align(h * dp * 2)) * pad_d + align(d * hp * 2) * pad_h
                + align(part * 4) + align(2 * _up(rows, c["dhidden"][0]) * 2 * hp * 4) + align(COLUMN_GROUPS * d * 4))
    return forward, backward


# Sizes whose launches hold what no other test's do: whole tiles and tiles in
# parts next to each other (of one product, of three), and of the weights'
# gradients whole tiles of 256 x 256 and parts of 64 x 64.
SIZES = [(1106, 1300, 1943), (1589, 2705, 2524), (2379, 293, 3595), (17725, 436, 1090), (11778, 1706, 1479), (17183, 133, 2088),
         (17393, 146, 963), (262, 2986, 1311), (2165, 9, 8)]
