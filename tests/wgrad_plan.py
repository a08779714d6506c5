"""The weight-gradient kernel's plan, written again from its description: the
tile's width in 64-column waves and the segments of the rows.  It picks test
shapes; the library's own plan is held to it through the workspace sizes."""


def _one(rows, M, N, gated, wn):
    tile_m, tile_n = (64 if gated else 128), 64 * wn
    tiles = -(-M // tile_m) * (-(-N // tile_n) if N > 0 else 1)
    steps = -(-rows // 32)
    most = max(1, min(128, steps // 4))

    def load(s):
        items, per = tiles * s, -(-steps // s)
        slab = 2.0 if wn == 4 else 1.25 if items <= 256 else 1.0
        return -(-items // 256) * per * slab + 0.25 * s

    best = min(load(s) for s in range(1, most + 1))
    segs = next(s for s in range(1, most + 1) if s == most or load(s) <= 1.05 * best)
    seg_steps = max(1, -(-steps // segs))
    return load(segs), wn, max(1, -(-steps // seg_steps))


def plan(rows, M, N, gated=False):
    """(waves along N, segments) for rows x M (gated: 2 M) and rows x N."""
    narrow = _one(rows, M, N, gated, 2)
    if N <= 128:
        return narrow[1:]
    wide = _one(rows, M, N, gated, 4)
    return (wide if wide[0] <= narrow[0] else narrow)[1:]


def workspace(rows, M, N, gated=False):
    segs, out = plan(rows, M, N, gated)[1], 2 * M if gated else M
    return segs * (out * (-(-N // 4) * 4) + -(-out // 4) * 4) * 4 if segs > 1 else 0
