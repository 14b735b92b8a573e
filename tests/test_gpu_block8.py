"""The 8-bit block-scaled cache on the GPU against the float64 oracle: codes and scales
exactly, attention within bounds counted from the roundings it makes."""
import numpy as np
import pytest
import torch

from oracle import block8_oracle as O

pytestmark = pytest.mark.gpu

FMTS = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_kv_cache_kv4_b200 import build
    build.build()


def _kv4():
    from quantized_kv_cache_kv4_b200 import kv4
    return kv4


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def paging(caps, seed, spare=3):
    """Page table (host array) over a shuffled pool with a few pages nobody owns."""
    need = [max(1, -(-c // 16)) for c in caps]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    table, at = np.full((len(caps), max(need)), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


class Model:
    """The cache as the oracle has it, fed by the same calls as the library's."""

    def __init__(self, fmt, caps, H, seed=0, G=1):
        kv4 = _kv4()
        self.fmt, self.H, self.G = fmt, H, G
        self.table, self.pages = paging(caps, seed)
        self.cfg = kv4.make_config(H * G, H, 0, 0)
        self.code = kv4.BLOCK8_INT8 if fmt == "int8" else kv4.BLOCK8_E4M3
        self.cache = kv4.allocate_block8_cache(self.code, self.cfg, self.pages)
        # what nobody has written holds e4m3 NaN codes and NaN scales
        for t in (self.cache.k, self.cache.v):
            t.view(torch.int8).fill_(0x7F)
        for t in (self.cache.k_scales, self.cache.v_scales):
            t.fill_(float("nan"))
        self.blocks = {}
        self.rows = [[] for _ in caps]  # lengths only
        self.lens = np.zeros(len(caps), np.int64)
        self.table_t = ints(self.table)
        self.err = ints([0])

    def batch(self, lens=None):
        lens = self.lens if lens is None else lens
        return _kv4().BatchTensors(self.table_t, ints(lens), None, None, int(max(1, max(lens))))

    def append(self, k, v, counts, indptr=True, **kw):
        """k, v bf16 [rows, H, 128] on the GPU; counts rows per sequence."""
        self.lens = self.lens + np.asarray(counts)
        ip = ints(np.concatenate([[0], np.cumsum(counts)])) if indptr else None
        _kv4().block8_append(self.cache, self.batch(), k, v, ip, self.err, **kw)
        at = 0
        for x, rows in (("k", k.float().cpu().numpy()), ("v", v.float().cpu().numpy())):
            at = 0
            for b, n in enumerate(counts):
                p, end = int(self.lens[b]) - n, int(self.lens[b])
                while p < end:
                    hi = min(end, p // 16 * 16 + 16)
                    for h in range(self.H):
                        blk = self.blocks.setdefault((x, b, p // 16, h), O.Block(self.fmt))
                        blk.append(p % 16, rows[at:at + hi - p, h])
                    at += hi - p
                    p = hi
        return at

    def check_pages(self):
        c = self.cache
        for x, codes, scales in (("k", c.k, c.k_scales), ("v", c.v, c.v_scales)):
            codes, scales = codes.float().cpu().numpy(), scales.float().cpu().numpy()
            for (y, b, p, h), blk in self.blocks.items():
                if y != x:
                    continue
                page, n = self.table[b, p], min(16, int(self.lens[b]) - 16 * p)
                assert scales[page, h] == blk.scale, (x, b, p, h, scales[page, h], blk.scale)
                got = codes[page, h].transpose(1, 0, 2).reshape(16, 128)
                assert np.array_equal(got[:n], blk.codes[:n]), (x, b, p, h)

    def values(self, b):
        L = int(self.lens[b])
        out = []
        for x in ("k", "v"):
            y = np.zeros((L, self.H, 128))
            for p in range(-(-L // 16)):
                for h in range(self.H):
                    blk = self.blocks[(x, b, p, h)]
                    n = min(16, L - 16 * p)
                    y[16 * p:16 * p + n, h] = blk.codes[:n] * blk.scale
            out.append(y)
        return out

    def code_sums(self, b):
        """Largest value scale times the sum of |value codes| of each kv head: [H, 128]."""
        out = np.zeros((self.H, 128))
        for h in range(self.H):
            blocks = [self.blocks[("v", b, p, h)] for p in range(-(-int(self.lens[b]) // 16))]
            if blocks:
                out[h] = max(x.scale for x in blocks) * sum(np.abs(x.codes).sum(0) for x in blocks)
        return out

    def attend(self, n, seed=1, qscale=1.0, behind=0, stream=None, workspace=None):
        """Attention of the last n[b] positions of every sequence, against the oracle."""
        kv4 = _kv4()
        Hq = self.H * self.G
        total = int(sum(n)) + behind
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = (torch.randn((total, Hq, 128), generator=g, device="cuda") * qscale).to(torch.bfloat16)
        out = torch.full_like(q, 7.0)
        o32 = torch.full((total, Hq, 128), 7.0, device="cuda")
        lse = torch.full((total, Hq), 7.0, device="cuda")
        ip = ints(np.concatenate([[0], np.cumsum(n)]))
        single = all(x == 1 for x in n) and not behind
        maxn, maxl = int(max(n)), int(max(1, max(self.lens)))
        size = kv4.block8_workspace_size(self.cfg, len(n), total, maxn, maxl)
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if workspace is None else workspace
        torch.cuda.synchronize()
        kv4.block8_attention(self.cache, self.batch(), q, out, ws, None if single else ip, maxn, o32,
                             lse, self.err, stream=stream)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0, kv4.decode_err(int(self.err.item()))
        self.compare(q, out, o32, lse, n)
        if behind:  # rows behind the last sequence
            assert torch.all(out[-behind:] == 7.0) and torch.all(o32[-behind:] == 7.0)
            assert torch.all(lse[-behind:] == 7.0)
        return out, o32, lse

    def compare(self, q, out, o32, lse, n):
        qn, out, o32, lse = (t.float().cpu().numpy() for t in (q, out, o32, lse))
        at = 0
        for b, m in enumerate(n):
            K, V = self.values(b)
            sl = slice(at, at + m)
            Or, lr, A, mag = O.attention(qn[sl], K, V, self.G)
            at += m
            # logits: fp32 sums of 128 exact products (each of up to 130 roundings 2^-24 of the
            # sum of magnitudes), the scales' products and 2^x another 2^-22 of the logit
            ds = (130 * 2.0 ** -24 + 2.0 ** -21) * mag + 2.0 ** -21
            # output: weights off by e^ds, rounded to fp16 (2^-11), sums in fp32 over L rows
            to = (2.0 ** -11 + 2 * ds[..., None] + (K.shape[0] + 64) * 2.0 ** -24) * A + 1e-30
            # the weights carry the value scales in fp16: p 2^14 vs / 2^e (up to 64 query rows of a
            # kv head) or p 2^7 vs / 2^e, with 2^e at most twice the largest scale. A subnormal of
            # that is off by at most 2^-25: 2^-38 or 2^-31 of the largest scale for each code (which
            # shows where the largest weights' values are 0)
            to += 2.0 ** (-38 if max(n) * self.G <= 64 else -31) * np.repeat(self.code_sums(b), self.G, 0)
            assert np.all(np.abs(o32[sl] - Or) <= to), (b, (np.abs(o32[sl] - Or) / to).max())
            assert np.all(np.abs(out[sl] - Or) <= to + 2.0 ** -8 * np.abs(Or)), b
            seen = np.isfinite(lr)
            assert np.array_equal(np.isneginf(lse[sl]), ~seen), b
            tl = ds + 2.0 ** -20 * np.maximum(1, np.abs(np.where(seen, lr, 0)))
            assert np.all(np.abs(lse[sl][seen] - lr[seen]) <= tl[seen]), b


def rows(total, H, seed, scale=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, total, H, 128), generator=g, device="cuda")
    if scale is not None:
        x *= scale
    return x[0].to(torch.bfloat16), x[1].to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [1, 2, 3])
def test_append_ragged_calls(fmt, H):
    """Ragged prefill (sequences without rows among them), then single tokens and chunks."""
    m = Model(fmt, [100, 40, 16, 70, 33, 5], H)
    rng = np.random.default_rng(5)
    for step, counts in enumerate([[37, 0, 15, 48, 16, 1], [1, 0, 1, 0, 0, 2], [5, 17, 0, 1, 16, 0],
                                   [0, 0, 0, 0, 0, 1], [33, 20, 0, 19, 1, 1]]):
        k, v = rows(sum(counts), H, 10 + step)
        k *= torch.as_tensor(rng.uniform(0.2, 4, (len(k), H, 1)), device="cuda").to(torch.bfloat16)
        m.append(k, v, counts)
    torch.cuda.synchronize()
    assert int(m.err.item()) == 0
    m.check_pages()


@pytest.mark.parametrize("fmt", FMTS)
def test_append_tokens_growing_scale(fmt):
    """One token at a time over page borders; rows grow, shrink, vanish, saturate the scale and
    fall into fp16's subnormal range."""
    scales = [1, 2, 4, 8, 0, 1, 1e-3, 1e3, 1e-30, 1, 0, 0, 1, 64, 2, 300,  # a page
              0, 0, 1e-6, 3e-6, 1e-5, 1e-4, 1e-3, 1, 1e6, 1e8, 1e30, 1, 1, 1, 1, 1,
              1e-7, 1e-4, 1e-4]
    m = Model(fmt, [len(scales), 2 * len(scales)], 2)
    for i, s in enumerate(scales):
        k, v = rows(2, 2, 100 + i, scale=s)
        m.append(k, v, [1, 1], indptr=False)
        torch.cuda.synchronize()
        m.check_pages()
    assert int(m.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_append_leaves_other_pages(fmt):
    m = Model(fmt, [64, 64], 2)
    before = [t.view(torch.uint8).clone() for t in (m.cache.k, m.cache.v)]
    k, v = rows(21, 2, 3)
    m.append(k, v, [21, 0])
    torch.cuda.synchronize()
    used = set(m.table[0, :2].tolist())
    for t, old in zip((m.cache.k, m.cache.v), before):
        t = t.view(torch.uint8)
        for p in range(m.pages):
            if p not in used:
                assert torch.equal(t[p], old[p]), p
        # slots behind the last row keep their bytes
        assert torch.equal(t[int(m.table[0, 1])][:, :, 5:], old[int(m.table[0, 1])][:, :, 5:])


@pytest.mark.parametrize("fmt", FMTS)
def test_append_bad_lengths_and_pages(fmt):
    """Wrong lengths and page ids are flagged and write nothing."""
    kv4 = _kv4()
    m = Model(fmt, [64, 64, 64], 2)
    k, v = rows(9, 2, 4)
    before = [t.view(torch.uint8).clone() for t in (m.cache.k, m.cache.v)]
    # fewer tokens than appended; longer than the table; a negative page
    b = m.batch([2, 65, 20])
    ip = ints([0, 3, 6, 9])
    m.table_t[2, 1] = -5
    kv4.block8_append(m.cache, b, k, v, ip, m.err)
    torch.cuda.synchronize()
    flag = int(m.err.item())
    assert flag & 2 and flag & 1
    pages = {int(m.table[2, 1])} | set(m.table[1].tolist())
    for t, old in zip((m.cache.k, m.cache.v), before):
        t = t.view(torch.uint8)
        for p in pages:
            assert torch.equal(t[p], old[p])


ATTEND = [
    # (caps, heads, G, queries of each sequence)
    ("decode-short", [1, 2, 15, 16, 17, 33, 100], 2, 4, [1] * 7),
    ("decode-gqa1", [40, 333], 4, 1, [1, 1]),
    ("decode-gqa8", [40, 333], 2, 8, [1, 1]),
    ("decode-gqa3-long", [2100, 7, 1030], 3, 3, [1, 1, 1]),
    ("decode-empty", [0, 50, 0, 3], 2, 4, [1, 1, 1, 1]),
    ("verify", [64, 100, 9, 0, 300], 2, 4, [5, 3, 9, 2, 0]),
    ("more-queries-than-rows", [4, 40], 1, 2, [9, 40]),
    ("chunk", [200, 77, 130], 1, 4, [130, 77, 33]),
    ("chunk-gqa8", [300, 20], 2, 8, [70, 20]),
    ("chunk-gqa3", [333, 257], 1, 3, [300, 1]),
    ("rows-9-to-16", [900, 40, 33, 700], 2, 4, [4, 3, 1, 4]),
    ("rows-17-to-64", [900, 40, 1500, 16], 2, 8, [8, 7, 3, 8]),
    ("rows-65", [300, 65, 400], 2, 1, [65, 65, 2]),
    ("rows-128", [300, 128, 400], 1, 4, [32, 32, 31]),
    ("prefill-ragged", [400, 1, 513], 2, 2, [400, 1, 257]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name,lens,H,G,n", ATTEND, ids=[a[0] for a in ATTEND])
def test_attention(fmt, name, lens, H, G, n):
    m = Model(fmt, lens, H, G=G)
    k, v = rows(sum(lens), H, 21)
    if len(k):
        m.append(k, v, lens)
    m.attend(n)
    out = m.attend(n, seed=2, behind=3)
    again = m.attend(n, seed=2, behind=3)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("qscale,kscale,vscale", [(2e6, 1e-6, 1.0), (1e-30, 1.0, 1e-4), (1.0, 1.0, 1e4), (6.0, 4.0, 1.0)])
def test_attention_ranges(fmt, n, qscale, kscale, vscale):
    """Large and tiny queries, keys and values; blocks whose value scales differ by 2^20."""
    m = Model(fmt, [150, 300], 2, G=4)
    k, v = rows(450, 2, 31)
    v = v * vscale
    v[60:90] *= 2.0 ** -20
    m.append((k * kscale).to(torch.bfloat16), v.to(torch.bfloat16), [150, 300])
    m.attend([min(n, 150), n], qscale=qscale)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_many_short_and_one_long(fmt):
    """More sequences than a warp share has items, and one that many warps share."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 20, 150)] + [5000]
    m = Model(fmt, lens, 1, G=2)
    k, v = rows(sum(lens), 1, 41)
    m.append(k, v, lens)
    m.attend([1] * len(lens))
    m.attend([min(3, L) for L in lens])


def test_attention_bad_page_is_left_out():
    """A page id outside the pool is flagged and its positions are left out."""
    kv4 = _kv4()
    m = Model("e4m3", [100], 2, G=2)
    k, v = rows(100, 2, 51)
    m.append(k, v, [100])
    for n in (1, 50):
        q = torch.randn((n, 4, 128), device="cuda").to(torch.bfloat16)
        o32 = torch.empty((n, 4, 128), device="cuda")
        out = torch.empty_like(q)
        ws = torch.empty(kv4.block8_workspace_size(m.cfg, 1, n, n, 100), dtype=torch.uint8, device="cuda")
        saved = m.table_t.clone()
        m.table_t[0, 1] = m.pages
        kv4.block8_attention(m.cache, m.batch(), q, out, ws, ints([0, n]), n, o32, None, m.err)
        torch.cuda.synchronize()
        assert int(m.err.item()) == 1
        m.err.zero_()
        m.table_t.copy_(saved)
        K, V = m.values(0)
        seen = np.r_[0:16, 32:100]
        qn = q.float().cpu().numpy()
        for i in (0, n - 1):
            keys = seen[seen <= 100 - n + i]
            for j in range(4):
                s = K[keys, j // 2] @ qn[i, j] / np.sqrt(128)
                p = np.exp(s - s.max())
                want = p @ V[keys, j // 2] / p.sum()
                assert np.abs(o32[i, j].cpu().numpy() - want).max() < 2e-3


def test_attention_refuses_bad_rows_and_lengths():
    """Too many queries of one sequence, rows behind total_q, a wrong length: flagged, and the
    rows are left as they were."""
    kv4 = _kv4()
    m = Model("int8", [60, 60], 1, G=4)
    k, v = rows(120, 1, 61)
    m.append(k, v, [60, 60])
    for lens, ip, maxn, alive in (([60, 60], [0, 5, 6], 4, [5]), ([60, 60], [0, 2, 9], 8, [0, 1]),
                                  ([65, 60], [0, 2, 4], 2, [2, 3]), ([-1, 60], [0, 2, 4], 2, [2, 3])):
        q = torch.randn((6, 4, 128), device="cuda").to(torch.bfloat16)
        out, lse = torch.full_like(q, 7.0), torch.full((6, 4), 7.0, device="cuda")
        ws = torch.empty(kv4.block8_workspace_size(m.cfg, 2, 6, maxn, 65), dtype=torch.uint8, device="cuda")
        kv4.block8_attention(m.cache, m.batch(lens), q, out, ws, ints(ip), maxn, None, lse, m.err)
        torch.cuda.synchronize()
        assert int(m.err.item()) == 2
        m.err.zero_()
        touched = (lse != 7.0).any(1).nonzero()[:, 0].tolist()
        # (the rows of a sequence of a wrong length are an empty sequence's)
        assert set(alive) <= set(touched) and set(touched) <= set(range(ip[-1]))
        if lens == [60, 60]:
            assert touched == alive


def test_streams_graphs_and_two_calls_at_once():
    """A captured and replayed step, and two calls on two streams with a workspace each."""
    kv4 = _kv4()
    m = Model("e4m3", [700, 90, 300], 2, G=4)
    k, v = rows(1000, 2, 71)
    m.append(k, v, [640, 80, 280])
    n = [1, 1, 1]
    ref = m.attend(n, seed=9)
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn((3, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    size = kv4.block8_workspace_size(m.cfg, 3, 3, 1, 700)
    bufs = [(torch.empty_like(q), torch.empty(size, dtype=torch.uint8, device="cuda")) for _ in range(3)]
    batch = m.batch()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (out, ws), st in zip(bufs, streams):
            kv4.block8_attention(m.cache, batch, q, out, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(out, ref[0]) for out, _ in bufs[:2])
    graph = torch.cuda.CUDAGraph()
    out, ws = bufs[2]
    kn, vn = rows(3, 2, 72)
    with torch.cuda.graph(graph):
        kv4.block8_attention(m.cache, batch, q, out, ws)
        kv4.block8_append(m.cache, batch, kn, vn)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0])


def test_decode_run():
    """Prefill, then steps of append and attention as a program runs them."""
    m = Model("int8", [120, 60, 33], 2, G=4)
    k, v = rows(150, 2, 81)
    m.append(k, v, [100, 31, 19])
    m.attend([100, 31, 19])
    for step in range(12):
        k, v = rows(3, 2, 90 + step, scale=1.0 + step % 3)
        m.append(k, v, [1, 1, 1], indptr=False)
        m.attend([1, 1, 1], seed=step)
    m.check_pages()


@pytest.mark.parametrize("n,G", [(40, 4), (9, 8), (5, 2)], ids=["tiles", "tiles-one-pipeline", "warps"])
def test_several_positions_on_streams_and_in_graphs(n, G):
    """Calls of several positions at once on two streams, replayed from a graph, and one after
    the other on one workspace that the call before left full."""
    kv4 = _kv4()
    m = Model("int8", [400, 130, 257, 64], 2, G=G)
    counts = [390, 121, 250, 60]
    k, v = rows(sum(counts), 2, 171)
    m.append(k, v, counts)
    new = [n, n // 2, n, 1]
    m.attend(new)
    total, Hq = sum(new), 2 * G
    g = torch.Generator(device="cuda").manual_seed(172)
    q = torch.randn((total, Hq, 128), generator=g, device="cuda").to(torch.bfloat16)
    ip, batch = ints(np.concatenate([[0], np.cumsum(new)])), m.batch()
    size = kv4.block8_workspace_size(m.cfg, 4, total, n, 400)

    def call(out, ws, stream=None):
        kv4.block8_attention(m.cache, batch, q, out, ws, ip, n, err=m.err, stream=stream)

    bufs = [(torch.zeros_like(q), torch.full((size,), 255, dtype=torch.uint8, device="cuda")) for _ in range(4)]
    call(*bufs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for (out, ws), s in zip(bufs[1:3], streams):
            call(out, ws, s)
    torch.cuda.synchronize()
    assert torch.equal(bufs[1][0], bufs[0][0]) and torch.equal(bufs[2][0], bufs[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*bufs[3])
        call(bufs[2][0], bufs[3][1])
    for _ in range(2):
        bufs[3][0].zero_()
        bufs[2][0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[3][0], bufs[0][0]) and torch.equal(bufs[2][0], bufs[0][0])
    m.attend(new, seed=5, workspace=bufs[3][1])
    assert int(m.err.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_pages_behind_four_gigabytes(fmt):
    """Pages whose codes lie past 2^32 bytes hold and give what those of a small pool do."""
    kv4 = _kv4()
    lens, H, G = [300, 77], 8, 4
    cfg = kv4.make_config(H * G, H, 0, 0)
    pages = [-(-L // 16) for L in lens]
    k, v = rows(sum(lens), H, 181)
    g = torch.Generator(device="cuda").manual_seed(182)
    got = []
    for pool in (sum(pages), 2 ** 32 // (2048 * H) + 40):
        cache = kv4.allocate_block8_cache(kv4.BLOCK8_INT8 if fmt == "int8" else kv4.BLOCK8_E4M3, cfg, pool)
        table = np.zeros((2, max(pages)), np.int32)
        table[0, :pages[0]] = pool - 1 - np.arange(pages[0])
        table[1, :pages[1]] = pool - 1 - pages[0] - np.arange(pages[1])
        batch = kv4.BatchTensors(ints(table), ints(lens), None, None, 300)
        err = ints([0])
        kv4.block8_append(cache, batch, k, v, ints([0, lens[0], sum(lens)]), err)
        res = [cache.k[-sum(pages):].view(torch.uint8).clone(), cache.v_scales[-sum(pages):].clone()]
        for n in (1, 4, 40):
            q = torch.randn((2 * n, H * G, 128), generator=g.manual_seed(n), device="cuda").to(torch.bfloat16)
            out = torch.zeros_like(q)
            ws = torch.empty(kv4.block8_workspace_size(cfg, 2, 2 * n, n, 300), dtype=torch.uint8, device="cuda")
            kv4.block8_attention(cache, batch, q, out, ws, ints([0, n, 2 * n]), n, err=err)
            res.append(out)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert res[2].float().abs().max() > 0.01
        got.append(res)
        del cache
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("single", [True, False], ids=["token", "rows"])
def test_append_infinities(fmt, single):
    """Infinite elements take the largest code, alone in a block and over codes that are rounded
    again; every output that sees them is finite."""
    m = Model(fmt, [20, 20], 2, G=2)
    k, v = rows(10, 2, 191)
    m.append(k, v, [5, 5])
    for step in range(3):
        k, v = rows(2, 2, 192 + step)
        if step != 1:
            k[0, 0, 3], k[1, 1, 127], v[0, 1, 0], v[1, 0, 64] = np.inf, -np.inf, -np.inf, np.inf
        m.append(k, v, [1, 1], indptr=not single)
    torch.cuda.synchronize()
    assert int(m.err.item()) == 0
    m.check_pages()
    kv4 = _kv4()
    q = torch.randn((2, 4, 128), device="cuda").to(torch.bfloat16)
    out, ws = torch.empty_like(q), torch.empty(kv4.block8_workspace_size(m.cfg, 2, 2, 1, 20), dtype=torch.uint8,
                                               device="cuda")
    kv4.block8_attention(m.cache, m.batch(), q, out, ws)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())
