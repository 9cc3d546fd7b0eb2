"""Which kernel an 8-bit cache's attention call takes and how it is cut: the library's
rules on sizes (attn_plan, launch_kv8_attention) written down a second time, so that a
test can tell what its case reaches."""

from collections import namedtuple

from numpy import float32 as f

CUS, MOST, WAVES = 256, 64, 4

# rows: queries of a block, up to 64 in the kernel for few; splits: parts of a
# sequence's pages; sorted: tiles in the order of all sequences' pages
Plan = namedtuple("Plan", "rows splits sorted")


def up(n, d):
    return -(-n // d)


def _cut(rows, queries, B, pages, Hk):
    few = rows <= 64
    tiles = B if few else (queries + (rows - 1) * B) // rows
    fill = min(MOST, CUS // (tiles * Hk))
    splits = 1
    if few:
        if pages > 16:
            deep = min(up(pages, 64) if pages > 128 else 1, 16 * CUS // (B * Hk))
            splits = min(max(fill, deep, 1), up(pages, WAVES), MOST)
    else:
        best = f(1.3) * f(pages)
        for s in range(2, min(fill, pages) + 1):
            time = f(1.3) * f(up(pages, s)) + f(6.0) + f(0.00026) * f(queries) * f(Hk) * f(s)
            if time < best:
                best, splits = time, s
    return tiles * Hk * splits, Plan(rows, splits, not few and 1 < B <= 64 and tiles * Hk > CUS)


def _plan(T, B, pages, Hk, group):
    queries, rows = T * group, 16
    while rows < 256 and queries > rows * B:
        rows *= 2
    blocks, plan = _cut(rows, queries, B, pages, Hk)
    return _cut(128, queries, B, pages, Hk)[1] if rows == 256 and blocks <= CUS * 3 // 4 else plan


def attention(T, B, max_pages, Hq, Hk, window=0):
    plan = _plan(T, B, max_pages, Hk, Hq // Hk)
    pages = (window + T + 62) // 64 + 1
    if window and pages < max_pages:
        shown = _plan(T, B, pages, Hk, Hq // Hk)
        plan = shown._replace(splits=min(shown.splits, plan.splits))
    return plan


def of(lengths, new, Hq, Hk, window=0, width=None):
    """The plan of a batch whose table is as wide as its longest sequence, or `width`."""
    return attention(sum(new), len(new), width or max(1, max(up(n, 64) for n in lengths)), Hq, Hk, window)


def workspace(T, B, max_pages, Hq, Hk, D):
    if T == 0 or B == 0:
        return 0
    splits = _plan(T, B, max_pages, Hk, Hq // Hk).splits
    return 0 if splits == 1 else T * Hq * splits * (D + 2) * 4
