"""The ring of scales of the 8-bit attention kernel for few rows (k_attn_decode_8bit.cu), as a model
of its warps without a GPU: whatever the order in which they get on, a warpgroup finds the batch of
scales that it waits for.

Two warpgroups take the segments in turn, so each waits for the batches of every second segment
only.  A wait by one bit of the phase returns at once when the barrier is two phases behind, so it
is sound only if the batch before, in the same place of the ring, has been filled: what holds a
warpgroup back until then is the segment's header, which follows the last key tile of the segment
before, which follows (kStages tiles earlier) a product."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lora_serving_device_gb300", "csrc")
RING, KEYS, WGS = 4, 128, 2   # segments ahead, keys of a tile, warpgroups


def shape(d):
    """Key tiles in flight and batches of the ring, as the source has them for d values a head."""
    with open(os.path.join(CSRC, "k_attn_decode_8bit.cu")) as f:
        text = f.read()
    assert re.search(r"kRing = 4;", text) and re.search(r"kTile = kKeys \* D;", text)
    stages = int(re.search(r"kStages = (\d+)u / kStage;", text).group(1)) // (2 * KEYS * d)
    ring = re.search(r"ScaleRing<([^>]+)> scales;", text).group(1)
    if ring.isdigit():
        return stages, int(ring)
    wide, narrow = re.search(r"%s = D == 128 \? (\d+) : (\d+);" % ring.split("::")[-1], text).groups()
    return stages, int(wide if d == 128 else narrow)


def stale(segments, stages, batches, a_batch, first):
    """Runs the warps over segments of these many tiles; of those that can get on, the first that
    `first` names takes a step.  True if a warpgroup took scales that are not its batch's."""
    tiles = [(s, i) for s, n in enumerate(segments) for i in range(n)]
    start = [sum(segments[:s]) for s in range(len(segments) + 1)]
    batch0 = [0]
    for n in segments:
        batch0.append(batch0[-1] + -(-n // a_batch))
    headers = keys = values = filled = products = 0      # done so far, each in order
    freed = [0] * batches                                # batches of each place that were read
    at = [[w, 0, False] for w in range(WGS)]             # segment, tile in it, scales at hand
    weights = set()                                      # tiles whose weights are there
    place = [-1] * batches                               # the batch that lies there
    phases = [0] * batches                               # completed, of its barrier

    def loader():
        nonlocal headers, keys
        if headers < len(segments) and keys == start[headers]:
            s = headers - RING
            if s >= 0 and (products < start[s + 1] or values < start[s + 1] or filled < batch0[s + 1] or
                           (at[s % WGS][0] <= s)):
                return False
            headers += 1
            return True
        if keys < start[headers] and (keys < stages or products > keys - stages):
            keys += 1
            return True
        return False

    def value_loader():
        nonlocal values
        if values < start[headers] and (values < stages or products > values - stages):
            values += 1
            return True
        return False

    def finder():
        nonlocal filled
        if filled >= batch0[headers] or filled // batches > freed[filled % batches]:
            return False
        place[filled % batches] = filled
        phases[filled % batches] += 1
        filled += 1
        return True

    def product():
        nonlocal products
        if products < len(tiles) and products in weights and products < values:
            products += 1
            return True
        return False

    wrong = []

    def warpgroup(w):
        s, i, ready = at[w]
        if s >= headers:
            return False
        n = batch0[s] + i // a_batch
        if not ready:
            if phases[n % batches] & 1 == (n // batches) & 1:
                return False
            if place[n % batches] != n:
                wrong.append(n)
            at[w][2] = True
            return True
        if start[s] + i >= keys:
            return False
        last = i == segments[s] - 1
        if last or (i + 1) % a_batch == 0:
            freed[n % batches] += 1
            at[w][2] = False
        weights.add(start[s] + i)
        at[w][1] += 1
        if last:
            at[w][:] = [s + WGS, 0, False]
        return True

    warps = {"loader": loader, "values": value_loader, "finder": finder, "product": product,
             "wg0": lambda: warpgroup(0), "wg1": lambda: warpgroup(1)}
    while products < len(tiles) and not wrong:
        assert any(warps[x]() for x in first()), "the warps wait for one another"
    return bool(wrong)


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_a_warpgroup_finds_its_scales(d, page):
    stages, batches = shape(d)
    a_batch = 2 if page == 8 else 4
    rng = random.Random(d + page)
    names = ["loader", "values", "finder", "product", "wg0", "wg1"]
    late = [x for x in names if x != "finder"] + ["finder"]   # the scales come when nothing else can get on
    for _ in range(150):
        most = rng.choice([1, 3, 9, 20])
        segments = [rng.randint(1, most) for _ in range(rng.randint(2, 12))]
        assert not stale(segments, stages, batches, a_batch, lambda: late), segments
        assert not stale(segments, stages, batches, a_batch, lambda: rng.sample(names, len(names))), segments


def test_the_model_knows_a_ring_that_is_too_small():
    late = ["loader", "values", "product", "wg0", "wg1", "finder"]
    assert stale([16, 16], 12, 4, 2, lambda: late)
    assert not stale([16, 16], 12, 8, 2, lambda: late)
