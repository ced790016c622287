"""A model of the tree kernel's rings of E4M3 tiles: which warp may go on when, and whether a key tile's scales can be
overwritten while a softmax still reads them.  The counts come from the kernel's source; no GPU is needed.

A call's key tiles go through these steps, each a counter here:
  load     tile t: its scales into entry t % ring, then its key codes, then the value codes LEAD - 1 tiles before;
           item x of the stream of copies waits until item x - NC has been converted (stages of codes)
  convert  item x, once it is copied and item x - NS has been used by the products (stages of halves)
  scores   of tile t by a group, once its keys are converted and the group's output product before it is complete
  softmax  of tile t by a group, once its scores are there; it reads the scales all the while
  output   of tile t, once the group's softmax is done and its values are converted
The products are issued in one order, by one thread."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "query_aware_sparse_append_gb300",
                      "csrc", "tree.cu")


def _counts():
    """(d, wide) -> (stages of halves, stages of codes, key tiles ahead), and entries of the ring of scales."""
    text = open(SOURCE).read()
    s = re.search(r"constexpr int kStages = D == 64 \? (\d+) : FP8 \? (\d+) : \d+;", text)
    c = re.search(r"constexpr int kCodeStages = !FP8 \? 0 : D == 64 \? (\d+) : WIDE \? (\d+) : (\d+);", text)
    lead = re.search(r"LEAD = WIDE \? (\d+) : (\d+);", text)
    ring = re.search(r"constexpr int kScaleRing = (\d+);", text)
    assert s and c and lead and ring, "the kernel states its stages another way: bring this model in line"
    ahead = [int(x) for x in lead.groups()]
    forms = {(d, wide): (int(s[1 if d == 64 else 2]), int(c[1 if d == 64 else 2 if wide else 3]), ahead[0 if wide else 1])
             for d in (64, 128) for wide in (False, True)}
    return forms, int(ring[1])


def _overwritten(ns, nc, lead, ring, wide, segments, slow):
    """The tile whose scales come over those of tile `slow` while a softmax reads them, or None.  Everything else runs
    as far as its waits allow while that softmax stands still, which is the worst that can happen to it."""
    # copies in their order and the products in theirs, over all segments
    load, items, products, base = [], 0, [], 0
    key_item, value_item = {}, {}
    for n in segments:
        for t in range(n + lead - 1):
            if t < n:
                load.append(("scales", base + t))
                load.append(("copy", items))
                key_item[base + t] = items
                items += 1
            if t >= lead - 1:
                load.append(("copy", items))
                value_item[base + t - lead + 1] = items
                items += 1
        groups = (lambda j: (0, 1)) if wide else (lambda j: (j & 1,))
        for j in range(min(lead, n)):
            products += [("scores", base + j, g) for g in groups(j)]
        for j in range(n):
            for g in groups(j):
                products.append(("output", base + j, g))
                if j + lead < n:
                    products.append(("scores", base + j + lead, g))
        base += n
    last_use = {}                                    # the item's stage is free after this product
    for at, (kind, tile, _) in enumerate(products):
        last_use[key_item[tile] if kind == "scores" else value_item[tile]] = at
    at_load = converted = issued = copied = 0
    softmax_done = set()
    moved = True
    while moved:
        moved = False
        while at_load < len(load):
            kind, x = load[at_load]
            if kind == "scales":
                if x != slow and x % ring == slow % ring and x > slow:
                    reading = any(p[0] == "scores" and p[1] == slow for p in products[:issued])
                    if reading:
                        return x
            else:
                if x >= nc and converted <= x - nc:
                    break
                copied = x + 1
            at_load += 1
            moved = True
        while converted < copied and (converted < ns or last_use[converted - ns] < issued):
            converted += 1
            moved = True
        while issued < len(products):
            kind, tile, group = products[issued]
            if kind == "scores":
                if key_item[tile] >= converted:
                    break
                if tile != slow:                     # the softmax that stands still is the only one that takes time
                    softmax_done.add((tile, group))
            elif value_item[tile] >= converted or (tile, group) not in softmax_done:
                break
            issued += 1
            moved = True
    return None


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("segments", [[40], [9], [3, 5, 11, 30], [1] * 30, [2] * 20, [7, 1, 1, 20, 8]])
def test_scales_stay_until_their_softmax_is_done(d, wide, segments):
    forms, ring = _counts()
    ns, nc, lead = forms[d, wide]
    for slow in range(sum(segments)):
        over = _overwritten(ns, nc, lead, ring, wide, segments, slow)
        assert over is None, "scales of tile %d come over those of tile %d, whose softmax runs" % (over, slow)


def test_the_model_sees_a_ring_that_is_too_short():
    assert _overwritten(8, 6, 2, 8, False, [40], 0) == 8
    assert all(_overwritten(8, 6, 2, 9, False, [40], slow) is None for slow in range(40))
    assert _overwritten(8, 6, 1, 7, True, [40], 3) == 10
    assert all(_overwritten(8, 6, 1, 8, True, [40], slow) is None for slow in range(40))


@pytest.mark.parametrize("lead,wide", [(2, False), (1, True)])
def test_the_length_that_the_kernel_asserts_is_enough(lead, wide):
    assert "(NS + NC + 1) / 2 + LEAD <= kScaleRing" in open(SOURCE).read()
    for ns in range(2 + lead, 10):
        for nc in range(1, 8):
            ring = (ns + nc + 1) // 2 + lead
            for segments in ([30], [3, 5, 9], [1] * 20, [2] * 12):
                for slow in range(sum(segments)):
                    assert _overwritten(ns, nc, lead, ring, wide, segments, slow) is None, (ns, nc)
