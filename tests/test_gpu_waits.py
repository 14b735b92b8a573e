"""A wait that gives up in the block-scaled cache's attention or in the attention weights: the
testing hook withholds one worker's first copy (nothing is issued, so nothing is in flight) and bounds each wait. The call returns with KV4_DEVERR_TIMEOUT alone, that worker's part
counts as empty, everything else is as usual, and so is the next call."""
import numpy as np
import pytest
import torch

from test_gpu_long_batches import Batch8, SMS, bf, ints, paging, rows

pytestmark = pytest.mark.gpu

TIMEOUT = 32
WARPS = 4  # of a block


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_kv_cache_kv4_b200 import build
    build.build()


def withhold(worker, attempts=64):
    from quantized_kv_cache_kv4_b200 import kv4
    kv4._lib.kv4_test_withhold_copy(worker, attempts)


def pages_of(L):
    return max(1, -(-L // 16))


def share(total, workers, least, w):
    """[begin, end) of worker w, as the kernels deal `total` items."""
    k = max(1, min(workers, total // least))
    per, more = divmod(total, k)
    at = lambda i: min(i * per + min(i, more), total)  # noqa: E731
    return at(w), at(w + 1)


def empty_masks(lens, n, H, G):
    return {b: torch.zeros((H, m * G, L), dtype=torch.bool) for b, (L, m) in enumerate(zip(lens, n))}


def lost_of_warp(lens, n, H, G, unit_rows, worker):
    """The positions that worker's share of (sequence, kv head, unit, page) covers, by row."""
    lost = empty_masks(lens, n, H, G)
    units = [-(-m * G // unit_rows) for m in n]
    total = sum(u * pages_of(L) * H for u, L in zip(units, lens))
    bound = (-(-sum(n) * G // unit_rows) + len(lens)) * H * pages_of(max(lens))
    warps = max(1, min(SMS * 3 * WARPS, bound // 4))
    grid = min(-(-warps // WARPS), SMS * (3 if unit_rows == 8 else 2))
    t0, t1 = share(total, grid * WARPS, 4, worker)
    at, seen = 0, []
    for b, L in enumerate(lens):
        for h in range(H):
            for u in range(units[b]):
                lo, hi = max(t0, at), min(t1, at + pages_of(L))
                if lo < hi:
                    r = slice(u * unit_rows, (u + 1) * unit_rows)
                    lost[b][h, r, 16 * (lo - at):16 * (hi - at)] = True
                    seen.append((b, h, u, hi - lo, pages_of(L)))
                at += pages_of(L)
    return lost, seen


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 7], ids=["8-rows", "16-rows", "two-units"])
@pytest.mark.parametrize("worker", [0, 5, 611])
def test_equal_shares(fmt, n, worker):
    """Shares that end inside units and hold whole ones; the same warp's next units are empty too."""
    H, G = 4, 4
    lens = np.random.default_rng(31).integers(1, 260, 150).tolist()
    lens[0] = 900
    assert len(lens) * H > 296
    counts = [min(n, L) for L in lens]
    m = Batch8(fmt, lens, H, G, *(bf(x) for x in rows(sum(lens), H, 32)), seed=5)
    unit_rows = 8 if n * G <= 8 else 16
    lost, seen = lost_of_warp(lens, counts, H, G, unit_rows, worker)
    assert seen
    withhold(worker)
    m.check(counts, 33, lost=lost, flag=TIMEOUT)
    m.check(counts, 33)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 4])
def test_clusters(fmt, n):
    """A unit dealt to the warps of a cluster: one warp's run of its pages is left out."""
    lens, H, G = [2000, 777], 2, 4
    m = Batch8(fmt, lens, H, G, *(bf(x) for x in rows(sum(lens), H, 34)), seed=6)
    units, pages, ctas = 2 * H, pages_of(max(lens)), 1
    while ctas < 8 and units * ctas * 2 <= 296 and pages >= 2 * WARPS * ctas * 2:
        ctas *= 2
    parts = ctas * WARPS
    assert pages <= 32 * WARPS * ctas and parts == 32
    for unit, part in ((0, 0), (1, 31), (3, 7)):  # (sequence 0, head 0), (0, 1), (1, 1)
        b, h = divmod(unit, H)
        p = pages_of(lens[b])
        lost = empty_masks(lens, [n, n], H, G)
        lost[b][h, :, 16 * (p * part // parts):16 * (p * (part + 1) // parts)] = True
        withhold(unit * parts + part)
        m.check([n, n], 35, lost=lost, flag=TIMEOUT)
    m.check([n, n], 35)


def lost_of_block(lens, n, H, G, worker):
    """The positions of block `worker`'s share of (sequence, kv head, unit of 256 rows, key tile)."""
    lost, units = empty_masks(lens, n, H, G), []
    for b, (L, m) in enumerate(zip(lens, n)):
        for h in range(H):
            for u in range(-(-m * G // 256)):
                last = min(m - 1, ((u + 1) * 256 - 1) // G)
                units.append((b, h, u, max(0, L - m + last) // 128 + 1))
    bound = (-(-sum(n) * G // 256) + len(lens)) * H * (max(lens) // 128 + 1)
    t0, t1 = share(sum(x[3] for x in units), min(SMS, bound), 1, worker)
    at, whole, cut = 0, 0, 0
    for b, h, u, nt in units:
        lo, hi = max(t0, at), min(t1, at + nt)
        if lo < hi:
            lost[b][h, 256 * u:256 * u + 256, 128 * (lo - at):128 * (hi - at)] = True
            whole, cut = whole + (hi - lo == nt), cut + (hi - lo < nt)
        at += nt
    return lost, whole, cut


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name,lens,H,G,n", [
    ("long-units", [1500, 1417, 40], 8, 4, [700, 333, 1]),
    ("many-units", np.random.default_rng(36).integers(20, 300, 130).tolist(), 8, 4, None),
    ("one-tile", [300, 65, 128], 2, 1, [65, 65, 2]),
], ids=["long-units", "many-units", "one-tile"])
def test_tiles(fmt, name, lens, H, G, n):
    """Every role of a block gives up, whole units and parts of units are empty."""
    n = n or [-(-2 * L // 3) for L in lens]
    m = Batch8(fmt, lens, H, G, *(bf(x) for x in rows(sum(lens), H, 37)), seed=7)
    wholes = cuts = 0
    for worker in (0, 5, 97):
        lost, whole, cut = lost_of_block(lens, n, H, G, worker)
        wholes, cuts = wholes + whole, cuts + cut
        withhold(worker, 1 << 14)  # (a block's roles wait for one another through whole segments)
        m.check(n, 38, lost=lost, flag=TIMEOUT if whole + cut else 0)
    assert wholes + cuts and (name == "one-tile" or wholes and cuts)
    m.check(n, 38)


@pytest.mark.parametrize("Hq,H", [(8, 4), (16, 2)], ids=["two-heads-per-warp", "one-head-per-warp"])
@pytest.mark.parametrize("worker", [0, 3, 70])
def test_weights(Hq, H, worker):
    """The totals of the warp's share stay as they were, all others are the usual ones."""
    from quantized_kv_cache_kv4_b200 import kv4
    S, R, G = 4, 40, Hq // H
    lens = [700, 33, 2, 410, 160, 1300]
    B, hpw = len(lens), 2 if G <= 4 else 1
    cfg = kv4.make_config(Hq, H, S, R)
    table, pages = paging(lens, 8)
    cache = kv4.allocate_cache(cfg, pages, B, B)
    batch = kv4.BatchTensors(ints(table), ints(lens), ints(range(B)), ints(range(B)), max(lens))
    err = ints([0])
    k, v = (bf(x) for x in rows(sum(lens), H, 39))
    kv4.quantize_append(cache, batch, k, v, ints(np.concatenate([[0], np.cumsum(lens)])), err)
    q = bf(rows(B, Hq, 40)[0])
    out, lse = torch.empty_like(q), torch.empty((B, Hq), device="cuda")
    ws = torch.empty(kv4.workspace_size(cfg, B, max(lens)), dtype=torch.uint8, device="cuda")
    kv4.decode_attention(cache, batch, q, out, ws, None, lse, err)
    old = torch.rand((B, H, max(lens)), device="cuda")
    usual, cut = (torch.full_like(old, -3.0) for _ in range(2))
    kv4.attention_weights(cache, batch, q, lse, usual, acc_in=old, err=err)
    withhold(worker)
    kv4.attention_weights(cache, batch, q, lse, cut, acc_in=old, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == TIMEOUT
    # a sequence's tiles per pair of heads: INT4 pages that hold [S, L - R), sink tiles, ring tiles
    tiles = []
    for L in lens:
        t = [range(max(S, 16 * p), min(L - R, 16 * p + 16)) for p in range(S // 16, (L - R - 1) // 16 + 1)] if L - R > S else []
        t += [range(0, min(S, L))]
        if max(S, L - R) < L:
            slots = [[p for p in range(max(S, L - R), L) if p % R // 16 == i] for i in range(-(-R // 16))]
            t += slots
        tiles.append(t)
    slots = -(-H // hpw)
    total = sum(len(t) for t in tiles) * slots
    bound = B * slots * (max(lens) // 16 + 2 + 1 + -(-R // 16))
    grid = min((bound // 4 + WARPS) // WARPS, SMS * 3)
    t0, t1 = share(total, grid * WARPS, 4, worker)
    want, at, left = usual.clone(), 0, 0
    for b, t in enumerate(tiles):
        for h in range(slots):
            for x in t:
                if t0 <= at < t1:
                    want[b, h * hpw:h * hpw + hpw, list(x)] = -3.0
                    left += 1
                at += 1
    assert left == t1 - t0 > 0
    assert torch.equal(cut, want)
    err.zero_()
    kv4.attention_weights(cache, batch, q, lse, cut, acc_in=old, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(cut, usual)
