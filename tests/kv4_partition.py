"""How the attention kernels cut a batch into runs, restated: the list of items' tiles
(with the units that stand for an item's fixed cost), equal parts for the CTAs, and in
the decode kernel for their warps.  Tests use it to assert that their sizes reach what
they are for."""
PREFILL_ROWS, PREFILL_TILE, PREFILL_PAD, PREFILL_MIN = 256, 128, 4, 2
DECODE_TILE, DECODE_PAD, DECODE_MIN = 64, 1, 4
FEW_ROWS = 48


def _cut(items, parts, least):
    """Items are (pad, tiles, tag); the list's units in `parts` equal runs of at least
    `least`: per run the (tiles, tag) of the items with tiles in it."""
    total = sum(p + n for p, n, _ in items)
    per = max(least, -(-total // parts))
    runs = [[] for _ in range(parts)]
    at = 0
    for pad, n, tag in items:
        lo, hi = at + pad, at + pad + n
        at = hi
        while lo < hi:
            c = lo // per
            end = min(hi, (c + 1) * per)
            runs[c].append((end - lo, tag))
            lo = end
    return runs, per


def prefill_runs(kv, ql, hkv, group, window=0, sms=152, above=0):
    """Per CTA the runs (tiles, rows of the item), in order; requests of more than
    `above` rows."""
    items = []
    for n, m in zip(kv, ql):
        rows = m * group
        if m == 0 or rows <= above:
            continue
        for r0 in range(0, rows, PREFILL_ROWS):
            r1 = min(rows, r0 + PREFILL_ROWS)
            hi = max(0, min(n, n - m + (r1 - 1) // group + 1))
            lo = max(0, n - m + r0 // group - window + 1) if window else 0
            lo //= PREFILL_TILE
            tiles = max(1, -(-hi // PREFILL_TILE) - lo)
            items += [(PREFILL_PAD, tiles, r1 - r0)] * hkv
    return _cut(items, sms, PREFILL_MIN)[0]


def decode_segments(kv, ql, hkv, group, row_tiles, window=0, sms=152, upto=None):
    """Per warp of every CTA the tile counts of its segments; row_tiles: 1 or 2 tiles of
    eight rows an item.  Requests of up to `upto` rows (None: all)."""
    rows_item, warps = 8 * row_tiles, 12 if row_tiles == 1 else 8
    units = []  # one entry a unit: the item, or None for a pad
    k = 0
    for n, m in zip(kv, ql):
        rows = m * group
        if m == 0 or (upto is not None and rows > upto):
            continue
        start = max(0, n - m - window + 1) if window else 0
        tiles = max(1, -(-n // DECODE_TILE) - start // DECODE_TILE)
        for _ in range(-(-rows // rows_item) * hkv):
            units += [None] * DECODE_PAD + [k] * tiles
            k += 1
    per = max(DECODE_MIN, -(-len(units) // sms))
    out = []
    for c0 in range(0, len(units), per):
        mine = units[c0:c0 + per]
        for w in range(warps):
            if len(mine) < warps:
                lo, hi = min(w, len(mine)), min(w + 1, len(mine))
            else:
                lo, hi = len(mine) * w // warps, len(mine) * (w + 1) // warps
            counts = {}
            for x in mine[lo:hi]:
                if x is not None:
                    counts[x] = counts.get(x, 0) + 1
            out.append(list(counts.values()))
    return out
