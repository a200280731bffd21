"""The divided attention's line of key tiles over several sequences, cut into
runs: every tile of every item once, in bounds, whatever the offsets hold."""

import pytest

from test_block_args import ITEM, locate, place_items, run_edge, tiles

BLOCKS = 148
# (lengths, query heads, causal): divided on a device of 148 SMs.
DIVIDED = [([6000, 3001], 1, False), ([6000, 3001], 1, True), ([3001, 6000], 2, True), ([0, 9000, 1, 8999], 1, False),
           ([0, 9000, 1, 6999], 1, True), ([1, 10200, 300], 1, False), ([11200, 0, 300, 7], 1, True),
           ([4000, 4000], 2, True), ([257, 8743], 1, True), ([8743, 257], 1, False), ([2900] * 4, 1, True)]
# What falling or far offsets come to, and the other lengths of the GPU tests.
OTHERS = [([4000, 5001], 1), ([3001, 0], 1), ([0, 8000], 1), ([9000, 0], 1), ([0, 0], 1), ([1, 1], 1),
          ([5500, 3, 6000], 1), ([0, 8980], 1), ([1, 4499], 1)]


def runs(lens, Hq, causal):
    total = place_items(lens, Hq, causal)[1]
    run = max(6, (total + BLOCKS - 1) // BLOCKS)
    for b in range(BLOCKS):
        at, end = (run_edge(lens, Hq, causal, min(w * run, total), total, run) for w in (b, b + 1))
        yield at, end


@pytest.mark.parametrize("lens,Hq,causal", DIVIDED + [(n, h, c) for n, h in OTHERS for c in (False, True)])
def test_runs_cover_every_key_tile_once(lens, Hq, causal):
    line, total = place_items(lens, Hq, causal)
    T, seen, front = sum(lens), set(), 0
    for at, end in runs(lens, Hq, causal):
        assert at == front and at <= end          # one run behind another
        front = end
        first = True
        while at < end:
            (begin, n, q0, head), r = locate(lens, Hq, causal, at)
            k = max(tiles(n, q0, 0, causal), tiles(n, q0, 1, causal))
            ka, kb = max(0, r - 1), min(k, end - at + r - 1)
            assert 0 <= ka < kb <= k and 0 <= q0 < n and 0 <= begin and begin + n <= T and head < Hq
            assert ka == 0 or first               # a block leaves one part of each kind at most
            assert kb == k or at + 1 + kb - r >= end
            # both slots of an item attend the first key tile of a run that goes on with it
            if ka > 0:
                assert all(tiles(n, q0, s, causal) > ka for s in range(2) if q0 + s * ITEM // 2 < n)
            for j in range(ka, kb):
                assert (begin, q0, head, j) not in seen
                seen.add((begin, q0, head, j))
            at += 1 + kb - r
            first = False
    assert front == total and len(seen) == sum(k for *_, k in line)


@pytest.mark.parametrize("causal", [False, True])
def test_no_run_begins_at_an_items_last_key_tile(causal):
    """Runs of any length, from any place: an edge moves to the item's end
    where one key tile would be left (so both slots of an item have work in
    every part of it)."""
    lens, Hq = [5000, 129, 2600, 1, 640], 1
    total = place_items(lens, Hq, causal)[1]
    for run in (6, 7, 16, 33, 100):
        for w in range(total):
            at = run_edge(lens, Hq, causal, w, total, run)
            if at == total:
                continue
            (_, n, q0, _), r = locate(lens, Hq, causal, at)
            k = max(tiles(n, q0, 0, causal), tiles(n, q0, 1, causal))
            assert r == 0 or 3 <= r <= k - 1
