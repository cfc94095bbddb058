"""The order in which the prompt attention hands its items out, replayed on the host: which CTAs
(or pairs of them) get which 256 query rows, in which turn."""

ROWS, KEYS = 256, 128  # query rows of an item, keys of a tile


def blocks(lens):
    return [(n + ROWS - 1) // ROWS for n in lens]


def in_order(lens, heads):
    """(sequence, block, head) of every item: last blocks first, of those all sequences that have one."""
    b = blocks(lens)
    return [(s, q, h) for q in range(max(b, default=0) - 1, -1, -1) for s in range(len(lens)) if b[s] > q for h in range(heads)]


def use_pairs(lens, heads, sms):
    n = sum(lens)
    items = (n // ROWS + min(len(lens), n)) * heads
    each = n // len(lens)
    pairs = (2 * items <= sms and each >= 1024) or (items <= sms and each >= 4096)
    return pairs, min(items, sms // 2 if pairs else sms)


def turns(lens, heads, sms):
    """pairs?, and per CTA (or pair) its items in the order of its turns."""
    pairs, workers = use_pairs(lens, heads, sms)
    items = in_order(lens, heads)
    out = []
    for w in range(workers):
        mine, want, k = [], w, 0
        while want < len(items):
            mine.append(items[want])
            k += 1
            want = k * workers + (w if k % 2 == 0 else workers - 1 - w)
        out.append(mine)
    return pairs, out


def key_tiles(lens, item, tile, rank):
    """Key tiles that CTA `rank` of a pair takes for query tile 0 or 1 of an item."""
    s, q, _ = item
    all_ = 2 * q + 1 + tile
    if tile and all_ > -(-lens[s] // KEYS):
        all_ = 0
    return (all_ - rank + 1) // 2 if all_ > rank else 0


def loads(lens, item, rank):
    """Key tiles that CTA `rank` of a pair loads for an item."""
    return max(key_tiles(lens, item, t, rank) for t in (0, 1))


def empty_turns(lens, heads, sms, first=1):
    """Turns from `first` on in which the second CTA of a pair has no key tile, over all pairs."""
    pairs, t = turns(lens, heads, sms)
    return sum(1 for mine in t for k, it in enumerate(mine) if k >= first and not loads(lens, it, 1)) if pairs else 0
