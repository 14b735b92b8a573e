"""The barrier phases that the tile kernel's loading warp waits for before its block ends, on a
model of an mbarrier: for every way its loop can end, each wait is for the last copy's phase."""
import itertools
import os


class Bar:
    """Phases of a barrier that one arrival completes."""

    def __init__(self):
        self.phase = 0

    def complete(self):
        self.phase += 1

    def done(self, parity):  # try_wait.parity
        return (self.phase & 1) != parity


def ending(tiles, stop):
    """Bars after the loading loop over `tiles` tiles that ended at `stop`: None (the end's mark), or
    (tile, 'k' / 'v' / 'next') for the wait that gave up; copies asked for; the loop's counter behind
    it; whether all waits went well."""
    full = [Bar(), Bar()]
    asked = [0, 0]
    k, ok = 0, True
    while ok:
        if stop == (k, "k"):
            ok = False
            break
        if k == tiles:
            full[0].complete()  # the end's mark
            break
        asked[0] += 1
        full[0].complete()
        if stop == (k, "v"):
            ok = False
            break
        asked[1] += 1
        full[1].complete()
        ok = stop != (k, "next")
        k += 1
    return full, asked, k, ok


def test_every_ending_waits_for_the_last_copies():
    for tiles in range(0, 6):
        for stop in [None, (tiles, "k")] + list(itertools.product(range(tiles), ("k", "v", "next"))):
            full, asked, k, ok = ending(tiles, stop)
            if stop is not None and stop[1] == "v":  # at the loop's own exit
                waits = [(0, k & 1)] + ([(1, (k & 1) ^ 1)] if k > 0 else [])
            else:
                waits = [(i, (k & 1) ^ 1) for i in range(2) if k > 0 and (i == 1 or not ok)]
            # K's last copy has been converted where the loop came to the end's mark
            assert {i for i, _ in waits} == {i for i in range(2) if asked[i] and (i == 1 or not ok)}, (tiles, stop)
            for i, parity in waits:
                assert full[i].done(parity), (tiles, stop, i)  # all landed: returns at once
                full[i].phase -= 1  # the last copy in flight: it is this one that is waited for
                assert not full[i].done(parity), (tiles, stop, i)
                full[i].phase += 1


def test_the_loading_warp_waits_however_its_loop_ends():
    """The waits stand behind the loop (one way out of it, a wait for the next segment that gave up,
    had none)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "quantized_kv_cache_kv4_b200", "csrc", "kv4_block8_tile.cu")) as f:
        src = f.read()
    load = src[src.index("- load -"):src.index("- schedule -")]
    behind = load[load.rindex("nxt = ask_page();"):]
    assert "wait(&bars.raw_full[0], (k & 1) ^ 1)" in behind
    assert "wait(&bars.raw_full[1], (k & 1) ^ 1)" in behind
