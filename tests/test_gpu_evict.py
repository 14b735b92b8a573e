"""Eviction by accumulated attention weight on the GPU: weights against the float64 oracle
within counted roundings, selection and moves exactly, and a run of decode steps over a cache
that is evicted on the way."""
import numpy as np
import pytest
import torch

from oracle import evict_oracle as E
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_kv_cache_kv4_b200 import build
    build.build()


def _mods():
    from quantized_kv_cache_kv4_b200 import kv4, session, workload
    return kv4, session, workload


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, Hq=8, Hkv=2, S=4, R=32, **kw):
    kv4, session, workload = _mods()
    wl = workload.custom_workload(lens, num_q_heads=Hq, num_kv_heads=Hkv, num_sinks=S, num_recent=R,
                                  seed=kw.pop("seed", 17), **kw)
    s = session.DecodeSession(wl, keep_streams=range(len(lens)))
    s.append_step(0)
    torch.cuda.synchronize()
    return s


def magnitude(q, k, S, R):
    """Per position and query head: the sum of the magnitudes that a logit is summed from
    (INT4: |q| (15 scale + |min|); INT8: |q| 127 scale), / sqrt(128)."""
    c4, s4, m4 = O.quantize_int4(k)
    big = np.repeat(15 * s4.astype(np.float64) + np.abs(m4.astype(np.float64)), 32, -1)
    _, s8 = O.quantize_int8(k)
    prot = O.protected_mask(len(k), S, R)
    big[prot] = 127 * s8.astype(np.float64)[prot][..., None]
    G = q.shape[0] // k.shape[1]
    return np.stack([big[:, j // G] @ np.abs(q[j].astype(np.float64)) for j in range(len(q))]) / np.sqrt(128)


WEIGHTS = [
    ("short", [1, 2, 4, 5, 15, 16, 17, 36, 37, 38, 100], 8, 2, 4, 32),
    ("gqa1", [40, 333], 4, 4, 4, 32),
    ("gqa8", [40, 333], 16, 2, 16, 128),
    ("gqa3", [70, 201], 9, 3, 1, 17),
    ("no-sinks", [60, 9, 300], 8, 2, 0, 100),
    ("no-recent", [60, 9, 300], 8, 2, 20, 0),
    ("no-protection", [60, 1, 300], 8, 2, 0, 0),
    ("long", [3001, 144, 145, 160], 8, 2, 16, 128),
]


@pytest.mark.parametrize("name,lens,Hq,Hkv,S,R", WEIGHTS, ids=[w[0] for w in WEIGHTS])
def test_weights(name, lens, Hq, Hkv, S, R):
    kv4, _, _ = _mods()
    s = make(lens, Hq, Hkv, S, R, outlier_channels=3, outlier_scale=10.0)
    B = len(lens)
    lse = torch.empty((B, Hq), device="cuda")
    s.attention_step(0, lse=lse)
    stride = max(lens) + 5
    old = torch.rand((B, Hkv, stride), device="cuda")
    out = torch.full_like(old, -3.0)
    batch = s.batch(s.step_lens[0])
    kv4.attention_weights(s.cache, batch, s.q[0], lse, out, acc_in=old, err=s.err)
    fresh = torch.full_like(old, -3.0)
    kv4.attention_weights(s.cache, batch, s.q[0], lse, fresh, err=s.err)
    place = old.clone()
    kv4.attention_weights(s.cache, batch, s.q[0], lse, place, acc_in=place, err=s.err)
    torch.cuda.synchronize()
    s.check_err()
    G = Hq // Hkv
    for b, L in enumerate(lens):
        k, _ = s.streams[b]
        K, _ = O.effective_kv(k[:L], k[:L], S, R)
        q = s.q[0, b].float().cpu().numpy()
        l = lse[b].cpu().numpy()
        want = E.weights(q, K, l, G)
        # each of a logit's roundings is at most 2^-24 of its summed magnitudes (128 products, 8
        # parameter terms, the scales' products); 2^x and the sums a few 2^-22
        per = np.exp(np.einsum("lhd,hgd->hgl", K, q.reshape(Hkv, G, 128).astype(np.float64)) / np.sqrt(128)
                     - l.reshape(Hkv, G, 1).astype(np.float64))
        mag = magnitude(q, k[:L], S, R).reshape(Hkv, G, L) + np.abs(l.reshape(Hkv, G, 1))
        tol = (per * (150 * 2.0 ** -24 * mag + 2.0 ** -20)).sum(1)
        got = fresh[b, :, :L].cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), (b, (np.abs(got - want) / tol).max())
        # a weight sums to about 1 over the positions for each query head
        assert np.all(np.abs(got.sum(-1) - G) < 0.02 * G), b
        total = old[b, :, :L].cpu().numpy()
        assert np.all(np.abs(out[b, :, :L].cpu().numpy() - total - want) <= tol + 2.0 ** -24 * (total + want) + 1e-12)
        assert torch.equal(out[b, :, :L], place[b, :, :L])
        assert torch.all(out[b, :, L:] == -3.0) and torch.equal(place[b, :, L:], old[b, :, L:])


def test_weights_flags_what_it_cannot_read():
    kv4, _, _ = _mods()
    s = make([300, 300, 300], 8, 2, 4, 32)
    lse = torch.empty((3, 8), device="cuda")
    s.attention_step(0, lse=lse)
    s.page_table[1, 5] = -7
    s.ring_idx[2] = 99
    out = torch.full((3, 2, 304), -3.0, device="cuda")
    kv4.attention_weights(s.cache, s.batch(s.step_lens[0]), s.q[0], lse, out, err=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 1 | 4
    assert torch.all(out[1, :, 80:96] == -3.0) and torch.all(out[1, :, :80] >= 0)
    assert torch.all(out[2, :, 268:300] == -3.0) and torch.all(out[2, :, :268] >= 0)
    s.err.zero_()
    small = torch.full((3, 2, 299), -3.0, device="cuda")  # shorter than the sequences
    kv4.attention_weights(s.cache, s.batch(s.step_lens[0]), s.q[0], lse, small, err=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 2 and torch.all(small == -3.0)


def batch_of(lens, pages=1):
    kv4, _, _ = _mods()
    return kv4.BatchTensors(torch.zeros((len(lens), pages), dtype=torch.int32, device="cuda"), ints(lens),
                            ints([0] * len(lens)), None, max(1, max(lens)))


SELECT = [
    ([0, 1, 5, 40, 41, 300, 1000], 2, 4, 36, 40),
    ([300, 1000, 4097, 33], 2, 4, 28, 32),       # no candidate stays
    ([300, 1000, 2500], 3, 0, 0, 1),
    ([17, 300], 1, 0, 0, 299),
    ([5000, 1025, 1024, 1023], 2, 16, 128, 1024),
    ([20000], 2, 16, 128, 9999),
    ([40000, 70000], 1, 1, 0, 2),
]


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("lens,H,S,R,budget", SELECT)
def test_select(lens, H, S, R, budget, kind):
    kv4, _, _ = _mods()
    cfg = kv4.make_config(H, H, S, R)
    B, stride = len(lens), max(lens) + 3
    rng = np.random.default_rng(len(lens) * 1000 + budget)
    acc = rng.standard_normal((B, H, stride)).astype(np.float32)
    if kind == "ties":
        acc = np.round(np.abs(acc), 1)
    elif kind == "equal":
        acc[:] = 0.25
    elif kind == "special":
        pick = rng.integers(0, 8, acc.shape)
        for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45)):
            acc[pick == i] = x
        acc[0, 0] = np.nan
    keep = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    err = ints([0])
    kv4.evict_select(cfg, batch_of(lens), torch.from_numpy(acc).cuda(), keep, new, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    keep = keep.cpu().numpy()
    assert new.tolist() == [min(L, budget) for L in lens]
    for b, L in enumerate(lens):
        for h in range(H):
            want = E.select(acc[b, h, :L], S, R, budget)
            assert keep[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)


def test_select_flags_a_length_past_the_totals():
    kv4, _, _ = _mods()
    cfg = kv4.make_config(2, 2, 1, 2)
    keep, new, err = ints(np.zeros((3, 2, 8))), ints([7, 7, 7]), ints([0])
    kv4.evict_select(cfg, batch_of([30, 31, -1]), torch.rand((3, 2, 30), device="cuda"), keep, new, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and new.tolist() == [8, 0, 0]
    assert torch.all(keep[1:] == -1) and torch.all(keep[0] >= 0)


def rows_of(cache, table, b, positions):
    """Bytes of the rows at `positions` ([H, n]) of sequence b: codes and parameters, [H, n, 160]."""
    out = []
    for h in range(positions.shape[0]):
        pg = torch.as_tensor(table[b][positions[h] // 16], device="cuda").long()
        sl = torch.as_tensor(positions[h] % 16, device="cuda").long()
        parts = [t[pg, h, :, sl].reshape(len(pg), -1) for t in (cache.k_codes, cache.v_codes)]
        parts += [t[pg, h, sl].reshape(len(pg), -1).view(torch.uint8) for t in (cache.k_params, cache.v_params)]
        out.append(torch.cat(parts, 1))
    return torch.stack(out)


def ring_rows(cache, ring, slots):
    t = torch.as_tensor(slots, device="cuda").long()
    parts = []
    for c, s in ((cache.ring_k, cache.ring_ks), (cache.ring_v, cache.ring_vs)):
        parts += [c[ring][:, t // 16, :, t % 16].reshape(len(t), c.shape[1], 128).view(torch.uint8),
                  s[ring][:, t].t().contiguous().view(torch.uint8).reshape(len(t), c.shape[1], 2)]
    return torch.cat(parts, 2)


COMPACT = [
    ([37, 150, 300, 511], 2, 2, 4, 32, 100),
    ([1000, 777, 20, 0, 401], 8, 2, 16, 128, 400),
    ([300, 33, 34, 36], 9, 3, 1, 31, 33),
    ([700, 520], 4, 4, 0, 100, 257),
    ([90, 2000], 8, 1, 20, 0, 64),
    ([90, 1500], 2, 1, 0, 0, 1),
]


@pytest.mark.parametrize("where", ["own", "own-totals", "other", "other-ring"])
@pytest.mark.parametrize("lens,Hq,Hkv,S,R,budget", COMPACT)
def test_select_and_compact(lens, Hq, Hkv, S, R, budget, where):
    kv4, _, _ = _mods()
    lens = [max(1, L) for L in lens]
    s = make(lens, Hq, Hkv, S, R)
    B, c = len(lens), s.cache
    batch = s.batch(s.step_lens[0])
    rng = np.random.default_rng(3)
    acc = torch.from_numpy(rng.random((B, Hkv, max(lens))).astype(np.float32)).cuda()
    keep = torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda")
    new = torch.empty(B, dtype=torch.int32, device="cuda")
    kv4.evict_select(s.cfg, batch, acc, keep, new, s.err)
    n = new.cpu().numpy()
    k = keep.cpu().numpy()
    table = s.page_table.cpu().numpy()
    before = [rows_of(c, table, b, k[b, :, :n[b]]) for b in range(B)]
    wins = [np.arange(max(S, n[b] - R), n[b]) for b in range(B)]
    rings = s.ring_idx.cpu().numpy()
    ring_before = [ring_rows(c, int(rings[b]), (wins[b] + lens[b] - n[b]) % max(R, 1)) for b in range(B)] if R else []
    want_acc = [torch.stack([acc[b, h][torch.as_tensor(k[b, h, :n[b]], device="cuda").long()] for h in range(Hkv)])
                for b in range(B)]
    acc_out, to, dst = torch.full((B, Hkv, budget + 1), -3.0, device="cuda"), None, table
    to_ring = None
    if where == "own-totals":
        acc_out = acc
    if where.startswith("other"):
        # other pages of the same pool: a pool twice as large
        need = [-(-int(x) // 16) for x in n]
        extra = rng.permutation(sum(need)) + c.num_pages
        for name in ("k_codes", "v_codes", "k_params", "v_params"):
            t = getattr(c, name)
            setattr(c, name, torch.cat([t, torch.zeros((len(extra),) + t.shape[1:], dtype=t.dtype, device="cuda")]))
        dst, at = np.full((B, max(need) + 1), -1, np.int32), 0
        for b in range(B):
            dst[b, :need[b]] = extra[at:at + need[b]]
            at += need[b]
        to = ints(dst)
        if where == "other-ring" and R:
            for name in ("ring_k", "ring_v", "ring_ks", "ring_vs"):
                t = getattr(c, name)
                setattr(c, name, torch.cat([t, torch.zeros_like(t)]))
            to_ring = ints(rings + B)
            rings = rings + B
    kv4.evict_compact(c, batch, keep, new, to, to_ring, acc, acc_out, s.err)
    torch.cuda.synchronize()
    s.check_err()
    for b in range(B):
        at = np.tile(np.arange(n[b]), (Hkv, 1))
        assert torch.equal(rows_of(c, dst, b, at), before[b]), b
        assert torch.equal(acc_out[b, :, :n[b]], want_acc[b]), b
        if where not in ("own-totals",):
            assert torch.all(acc_out[b, :, n[b]:] == -3.0)
        if R:
            assert torch.equal(ring_rows(c, int(rings[b]), wins[b] % R), ring_before[b]), b
    # and attention over what is left: kept INT4 rows, the sinks' and the window's INT8 copies
    out_batch = kv4.BatchTensors(to if to is not None else s.page_table, new, s.sink_idx,
                                 to_ring if to_ring is not None else s.ring_idx, budget)
    o32 = torch.empty((B, Hq, 128), device="cuda")
    ws = torch.empty(kv4.workspace_size(s.cfg, B, budget), dtype=torch.uint8, device="cuda")
    kv4.decode_attention(c, out_batch, s.q[0], s.out, ws, o32, None, s.err)
    torch.cuda.synchronize()
    s.check_err()
    for b, L in enumerate(lens):
        kk, vv = s.streams[b]
        K, V = O.effective_kv(kk[:L], vv[:L], S, R)
        q = s.q[0, b].float().cpu().numpy()
        G = Hq // Hkv
        for h in range(Hkv):
            sel = k[b, h, :n[b]]
            ref, _ = O.attention(q[h * G:h * G + G], K[sel, h:h + 1], V[sel, h:h + 1])
            got = o32[b, h * G:h * G + G].cpu().numpy()
            assert np.abs(got - ref).max() <= 2e-3 * max(1.0, np.abs(ref).max()), (b, h)


def test_compact_flags_bad_positions():
    """Positions out of range or order are skipped, a window that is not whole keeps its ring,
    wrong counts move nothing."""
    kv4, _, _ = _mods()
    s = make([200, 200, 200, 200], 8, 2, 4, 32)
    batch = s.batch(s.step_lens[0])
    acc = torch.rand((4, 2, 200), device="cuda")
    keep, new = torch.empty((4, 2, 64), dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    kv4.evict_select(s.cfg, batch, acc, keep, new, s.err)
    keep[0, 0, 40] = 3      # below its place
    keep[1, 1, 63] = 200    # past the length (and the window's last)
    new[2] = 65             # more than there are
    before = {n: getattr(s.cache, n).clone() for n in ("k_codes", "k_params", "ring_k")}
    kv4.evict_compact(s.cache, batch, keep, new, err=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 2 | 64
    pages = s.page_table[2, :13].long()
    assert torch.equal(s.cache.k_codes[pages], before["k_codes"][pages])
    r = int(s.ring_idx[1])
    assert torch.equal(s.cache.ring_k[r, 1], before["ring_k"][r, 1])
    assert torch.equal(s.cache.ring_k[int(s.ring_idx[2])], before["ring_k"][int(s.ring_idx[2])])
    p = int(s.page_table[0, 2])
    assert torch.equal(s.cache.k_codes[p, 0, :, 8], before["k_codes"][p, 0, :, 8])
    # other pages that are none
    s.err.zero_()
    kv4.evict_select(s.cfg, batch, acc, keep, new, s.err)
    to = torch.full((4, 4), -1, dtype=torch.int32, device="cuda")
    kv4.evict_compact(s.cache, batch, keep, new, to, err=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) & 1


def test_captured_eviction():
    """Weights, selection and moves captured into one graph give what eager calls give."""
    kv4, _, _ = _mods()
    res = []
    for captured in (False, True):
        s = make([150, 400, 64], 8, 2, 4, 32)
        batch = s.batch(s.step_lens[0])
        lse = torch.empty((3, 8), device="cuda")
        s.attention_step(0, lse=lse)
        acc = torch.zeros((3, 2, 400), device="cuda")
        keep = torch.zeros((3, 2, 50), dtype=torch.int32, device="cuda")
        new = torch.zeros(3, dtype=torch.int32, device="cuda")

        def calls():
            kv4.attention_weights(s.cache, batch, s.q[0], lse, acc, acc_in=acc, err=s.err)
            kv4.evict_select(s.cfg, batch, acc, keep, new, s.err)
            kv4.evict_compact(s.cache, batch, keep, new, acc_in=acc, acc_out=acc, err=s.err)

        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls()
            graph.replay()
        else:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                calls()
        torch.cuda.synchronize()
        s.check_err()
        n = new.cpu().numpy()
        table = s.page_table.cpu().numpy()
        res.append([keep, new] + [rows_of(s.cache, table, b, np.tile(np.arange(n[b]), (2, 1))) for b in range(3)]
                   + [acc[b, :, :n[b]] for b in range(3)])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_pages_behind_four_gigabytes():
    """Weights and moves of rows whose pages lie past 2^32 bytes are those of a small pool."""
    kv4, _, _ = _mods()
    lens, H, G, S, R, budget = [700, 150], 8, 4, 4, 32, 100
    cfg = kv4.make_config(H * G, H, S, R)
    pages = [-(-L // 16) for L in lens]
    g = torch.Generator(device="cuda").manual_seed(191)
    k, v = (torch.randn((sum(lens), H, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, H * G, 128), generator=g, device="cuda").to(torch.bfloat16)
    got = []
    for pool in (sum(pages), 2 ** 32 // (1024 * H) + 100):
        cache = kv4.allocate_cache(cfg, pool, 2, 2)
        table = np.zeros((2, max(pages)), np.int32)
        table[0, :pages[0]] = pool - 1 - np.arange(pages[0])
        table[1, :pages[1]] = pool - 1 - pages[0] - np.arange(pages[1])
        batch = kv4.BatchTensors(ints(table), ints(lens), ints([0, 1]), ints([0, 1]), 700)
        err = ints([0])
        kv4.quantize_append(cache, batch, k, v, ints([0, lens[0], sum(lens)]), err)
        out, lse = torch.empty_like(q), torch.empty((2, H * G), device="cuda")
        ws = torch.empty(kv4.workspace_size(cfg, 2, 700), dtype=torch.uint8, device="cuda")
        kv4.decode_attention(cache, batch, q, out, ws, None, lse, err)
        acc = torch.zeros((2, H, 700), device="cuda")
        kv4.attention_weights(cache, batch, q, lse, acc, err=err)
        keep = torch.empty((2, H, budget), dtype=torch.int32, device="cuda")
        new = ints([0, 0])
        kv4.evict_select(cfg, batch, acc, keep, new, err)
        kv4.evict_compact(cache, batch, keep, new, err=err)
        after = kv4.BatchTensors(batch.page_table, new, batch.sink_idx, batch.ring_idx, budget)
        out2 = torch.empty_like(q)
        kv4.decode_attention(cache, after, q, out2, ws, None, None, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and new.tolist() == [budget, budget]
        assert out2.float().abs().max() > 0.01
        got.append([out, lse, acc, keep, out2, cache.k_codes[-sum(pages):].clone(), cache.v_params[-sum(pages):].clone(),
                    cache.ring_k.clone()])
        del cache
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("other", [False, True], ids=["own-pages", "other-pages"])
def test_compact_flags_a_sink_that_was_not_kept(other):
    """A kept set without a sink: its INT8 copy stays where it is, so another row in its place would
    be read as the sink. The place is flagged and left as it was; the rest moves."""
    kv4, _, _ = _mods()
    s = make([200, 200], 8, 2, 4, 32)
    c, batch = s.cache, s.batch(s.step_lens[0])
    acc = torch.rand((2, 2, 200), device="cuda")
    keep, new = ints(np.zeros((2, 2, 64))), ints([0, 0])
    kv4.evict_select(s.cfg, batch, acc, keep, new, s.err)
    k = keep.cpu().numpy()
    k[1, 0, 2] = next(p for p in range(4, 168) if p not in k[1, 0])  # one more of the others instead
    keep.copy_(torch.from_numpy(np.sort(k, -1)))
    k = keep.cpu().numpy()
    assert k[1, 0, 2] == 3 and np.all(np.diff(k[1, 0]) > 0)
    table, places = s.page_table.cpu().numpy(), np.tile(np.arange(64), (2, 1))
    dst = table
    if other:
        extra = np.arange(8, dtype=np.int32).reshape(2, 4) + c.num_pages
        for name in ("k_codes", "v_codes", "k_params", "v_params"):
            t = getattr(c, name)
            setattr(c, name, torch.cat([t, torch.full((8,) + t.shape[1:], 7, dtype=t.dtype, device="cuda")]))
        dst = extra
    want = [rows_of(c, table, b, k[b]) for b in range(2)]
    before = rows_of(c, dst, 1, places)
    kv4.evict_compact(c, batch, keep, new, ints(dst) if other else None, err=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 64
    got = [rows_of(c, dst, b, places) for b in range(2)]
    assert torch.equal(got[0], want[0])
    bad = [j for j in range(4) if k[1, 0, j] != j]
    assert bad == [2, 3]
    for j in range(64):
        assert torch.equal(got[1][0, j], before[0, j] if j in bad else want[1][0, j]), j
    assert torch.equal(got[1][1], want[1][1])
