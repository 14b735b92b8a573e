"""Batches large enough that every worker of the kernels takes many tiles and several units:
the block-scaled cache's attention and the attention weights against definitions in 64 bits on
the GPU (over the codes that the cache holds), and selection of rows of 8193 to 16384."""
import math

import numpy as np
import pytest
import torch

from oracle import evict_oracle as E

pytestmark = pytest.mark.gpu

FMTS = ["int8", "e4m3"]
SMS = 148


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
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def paging(lens, seed):
    need = [max(1, -(-L // 16)) for L in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + 2)
    table, at = np.full((len(lens), max(need)), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


class Batch8:
    """A block-scaled cache filled by one call; k, v bf16 [rows, H, 128]."""

    def __init__(self, fmt, lens, H, G, k, v, seed=0):
        kv4 = _kv4()
        self.lens, self.H, self.G = lens, H, G
        self.cfg = kv4.make_config(H * G, H, 0, 0)
        self.table, pages = paging(lens, seed)
        self.cache = kv4.allocate_block8_cache(kv4.BLOCK8_INT8 if fmt == "int8" else kv4.BLOCK8_E4M3, self.cfg, pages)
        self.batch = kv4.BatchTensors(ints(self.table), ints(lens), None, None, max(lens))
        self.err = ints([0])
        kv4.block8_append(self.cache, self.batch, k, v, ints(np.concatenate([[0], np.cumsum(lens)])), self.err)

    def held(self, b):
        """Codes [H, L, 128] and scales [H, L] of K and of V of sequence b, in 64 bits."""
        L = self.lens[b]
        ids = torch.as_tensor(self.table[b, :-(-L // 16)]).cuda().long()
        out = []
        for codes, scales in ((self.cache.k, self.cache.k_scales), (self.cache.v, self.cache.v_scales)):
            c = codes[ids].float().double().permute(1, 0, 3, 2, 4).reshape(self.H, -1, 128)[:, :L]
            out += [c, scales[ids].double().t().repeat_interleave(16, 1)[:, :L]]
        return out

    def check(self, n, seed, qscale=1.0, q_of=None, lost=None, flag=0, query_step=0.0):
        """Attention of the last n[b] positions of each sequence, every row. lost: {sequence: bool
        [H, n G, L]}, positions that its rows are without; flag: the error bits of the call;
        query_step: what an element of a query may be off by, of its largest."""
        kv4 = _kv4()
        Hq, total, most = self.H * self.G, sum(n), max(n)
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn((total, Hq, 128), generator=g, device="cuda") * qscale
        if q_of is not None:
            q = q_of(q)
        q = q.to(torch.bfloat16)
        out, o32 = torch.full_like(q, 7.0), torch.full(q.shape, 7.0, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        size = kv4.block8_workspace_size(self.cfg, len(n), total, most, max(self.lens))
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        ip = None if most == 1 and min(n) == 1 else ints(np.concatenate([[0], np.cumsum(n)]))
        kv4.block8_attention(self.cache, self.batch, q, out, ws, ip, most, o32, lse, self.err)
        torch.cuda.synchronize()
        assert int(self.err.item()) == flag, kv4.decode_err(int(self.err.item()))
        self.err.zero_()
        at = 0
        for b, m in enumerate(n):
            if m:
                self.compare(b, q[at:at + m], out[at:at + m], o32[at:at + m], lse[at:at + m], most * self.G <= 64,
                             None if lost is None else lost.get(b), query_step)
            at += m

    def compare(self, b, q, out, o32, lse, few, lost=None, query_step=0.0):
        L, n, H, G = self.lens[b], q.shape[0], self.H, self.G
        kc, ks, vc, vs = self.held(b)
        k, v = kc * ks[..., None], vc * vs[..., None]
        q = q.double().reshape(n, H, G, 128).permute(1, 0, 2, 3).reshape(H, n * G, 128)
        last = L - n + torch.arange(n, device="cuda").repeat_interleave(G)
        hidden = (torch.arange(L, device="cuda") > last[:, None])[None]
        if lost is not None:
            hidden = hidden | lost.cuda()
        s = (q @ k.transpose(1, 2) / math.sqrt(128)).masked_fill_(hidden, -math.inf)
        mag = (q.abs() @ k.abs().transpose(1, 2) / math.sqrt(128)).masked_fill_(hidden, 0.0).amax(-1)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m.clamp(min=-1e300))
        z = p.sum(-1, keepdim=True)
        p /= z.clamp(min=1e-300)
        want, big, lr = p @ v, p @ v.abs(), (m + torch.log(z))[..., 0]
        # logits: fp32 sums of 128 products (130 roundings of 2^-24 of the sum of magnitudes), the
        # scales' products and 2^x another 2^-22 of the logit
        ds = (130 * 2.0 ** -24 + 2.0 ** -21) * mag + 2.0 ** -21
        ds += query_step * q.abs().amax(-1) * k.abs().sum(-1).amax(1)[:, None] / math.sqrt(128)
        # weights off by e^ds and rounded to fp16 (2^-11), L products and sums in fp32, two roundings
        # of 2^-24 and a factor 2^x off by 2^-22 for each step of at least 32 positions that moves the
        # maximum or the value scales' exponent
        tol = (2.0 ** -11 + 2 * ds[..., None] + (L + 64) * 2.0 ** -24 + L / 32 * 2.0 ** -21) * big + 1e-30
        # what fp16 holds as a subnormal is off by 2^-38 (few rows) or 2^-31 of the largest scale
        tol += 2.0 ** (-38 if few else -31) * (vs.amax(1)[:, None] * vc.abs().sum(1))[:, None]
        back = lambda x: x.double().reshape(n, H, G, -1).permute(1, 0, 2, 3).reshape(H, n * G, -1)  # noqa: E731
        got, got16, gl = back(o32), back(out), back(lse)[..., 0]
        off = (got - want).abs() / tol
        assert bool((off <= 1).all()), (b, float(off.max()))
        assert bool(((got16 - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()), b
        tl = ds + 2.0 ** -20 * lr.abs().clamp(min=1) + (L + 64) * 2.0 ** -24 + L / 32 * 2.0 ** -21
        sees = torch.isfinite(lr)
        assert bool((torch.isneginf(gl) == ~sees).all()), b
        assert bool(((gl - lr).abs() <= tl)[sees].all()), (b, float(((gl - lr).abs() / tl)[sees].max()))


def rows(total, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((total, H, 128), generator=g, device="cuda") for _ in range(2)]


def key_tiles(lens, n, H, G):
    """Key tiles of 128 positions over all units of 256 query rows."""
    total = 0
    for L, m in zip(lens, n):
        for u in range(-(-m * G // 256)):
            last = min(m - 1, ((u + 1) * 256 - 1) // G)
            total += max(0, L - m + last) // 128 + 1
    return total * H


def bf(x):
    return x.to(torch.bfloat16)


MANY = [
    # lengths, kv heads, G, queries
    ("chunks", [1500, 1417, 40], 8, 4, [700, 333, 1]),
    ("gqa8", [1210, 900], 4, 8, [300, 513]),
    ("gqa3", [2000, 130, 777], 6, 3, [1111, 130, 40]),
    ("gqa1-late", [9000, 5000], 8, 1, [70, 257]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name,lens,H,G,n", MANY, ids=[m[0] for m in MANY])
def test_many_key_tiles_per_worker(fmt, name, lens, H, G, n):
    assert max(n) * G > 64 and key_tiles(lens, n, H, G) >= 4 * SMS
    m = Batch8(fmt, lens, H, G, *(bf(x) for x in rows(sum(lens), H, 5)))
    m.check(n, 6)
    m.check(n, 7, qscale=3.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_units_per_worker(fmt):
    """Short prompts: every worker goes through more units than the ring of segments holds."""
    rng = np.random.default_rng(8)
    lens = rng.integers(17, 200, 220).tolist()
    n = [int(rng.integers(0, L + 1)) for L in lens]
    n[3], n[50], n[219] = lens[3], 0, lens[219]
    assert key_tiles(lens, n, 8, 4) >= 10 * SMS
    m = Batch8(fmt, lens, 8, 4, *(bf(x) for x in rows(sum(lens), 8, 9)), seed=2)
    m.check(n, 10)


def drifting(lens, H, seed, logit, value):
    """Rows whose logits (for queries along the keys' common direction) change by `logit` and whose
    values' magnitude changes by a factor 2^`value` for each 128 positions."""
    k, v = rows(sum(lens), H, seed)
    pos = torch.cat([torch.arange(L, device="cuda") for L in lens]).float()[:, None, None] / 128
    far = max(lens) / 128
    along = torch.zeros(128, device="cuda")
    along[::2] = 1.0  # 64 dims: a query of 1 along it gives alpha * 64 / sqrt(128)
    k = 0.25 * k + along * ((pos if logit >= 0 else pos - far) * logit * math.sqrt(128) / 64)
    v = v * torch.exp2((pos if value >= 0 else pos - far) * value)
    return bf(k), bf(v), lambda q: 0.25 * q + along


@pytest.mark.parametrize("fmt", FMTS)
# logits that outgrow a row's maximum every third tile, or each; value scales that double from tile
# to tile, also under logits that fall as fast, so that old tiles keep their share; both rising
@pytest.mark.parametrize("logit,value", [(2.5, 0.0), (7.0, -1.0), (-0.7, 1.0), (0.0, 1.0), (1.0, 1.0)])
@pytest.mark.parametrize("few", [False, True], ids=["tiles", "pairs"])
def test_drifting_logits_and_value_scales(fmt, logit, value, few):
    lens, H, G = [1300, 1100], 8, 4
    k, v, q_of = drifting(lens, H, 11, logit, value)
    m = Batch8(fmt, lens, H, G, k, v)
    if few:  # a cluster of warps per unit, 8, 16 and 64 rows
        for n in ([1, 1], [4, 3], [16, 9]):
            m.check(n, 12, q_of=q_of)
    else:
        n = [600, 437]
        assert key_tiles(lens, n, H, G) >= 4 * SMS
        m.check(n, 13, q_of=q_of)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 9, 40], ids=["8-rows", "16-rows", "tiles"])
@pytest.mark.parametrize("large", [2.0 ** 8, 2.0 ** 16, 2.0 ** 24])
def test_queries_with_one_large_element(fmt, n, large):
    """An element that meets zero keys and is far larger than the others that make the logits: they
    lose bits with INT8 codes and few rows only, where the query is 23-bit fixed point (from 2^-14 of
    the largest down)."""
    lens, H, G = [500, 333], 4, 4
    k, v = rows(sum(lens), H, 22)
    k[..., 5] = 0.0
    m = Batch8(fmt, lens, H, G, bf(k), bf(v))

    def q_of(q):
        q = q.clone()
        q[..., 5] = 4 * large
        return torch.where(q.abs() < 2.0 ** -4, 2.0 ** -4, q)  # (fp16 holds down to 2^-31 of the largest)

    m.check([n, n], 23, q_of=q_of, query_step=2.0 ** -22 if fmt == "int8" and n * G <= 64 and large > 2 ** 8 else 0.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("drift", [False, True], ids=["even", "drifting"])
def test_long_shares_of_few_rows(fmt, drift):
    """Equal shares of more than 64 pages per warp, several kv heads, 8 and 16 rows per unit."""
    rng = np.random.default_rng(14)
    lens, H, G = rng.integers(3500, 8200, 48).tolist(), 8, 4
    pages = sum(-(-L // 16) for L in lens) * H
    assert len(lens) * H > 296 and pages > 64 * SMS * 3 * 4
    if drift:
        k, v, q_of = drifting(lens, H, 15, -0.1, 0.15)
    else:
        (k, v), q_of = (bf(x) for x in rows(sum(lens), H, 15)), None
    m = Batch8(fmt, lens, H, G, k, v, seed=3)
    del k, v
    for n in ([1] * 48, rng.integers(0, 5, 48).tolist(), rng.integers(2, 10, 48).tolist()):
        m.check(n, 16, q_of=q_of)


@pytest.mark.parametrize("Hq,H,S,R,B", [(32, 8, 16, 128, 48), (64, 8, 4, 100, 48), (8, 8, 0, 0, 48)],
                         ids=["gqa4", "gqa8", "gqa1"])
def test_weights_of_long_shares(Hq, H, S, R, B):
    """More than 64 tiles per warp, with two heads per warp (up to four query heads each) and one."""
    kv4 = _kv4()
    G, hpw = Hq // H, 2 if Hq // H <= 4 else 1
    lens = np.random.default_rng(18).integers(8000 // (1 if hpw == 2 else 2), 13000 // (1 if hpw == 2 else 2), B).tolist()
    assert sum(-(-L // 16) for L in lens) * H // hpw > 64 * SMS * 3 * 4
    cfg = kv4.make_config(Hq, H, S, R)
    table, pages = paging(lens, 4)
    cache = kv4.allocate_cache(cfg, pages, B, B)
    ids = ints(np.random.default_rng(19).permutation(B))
    batch = kv4.BatchTensors(ints(table), ints(lens), ids, ids, max(lens))
    err = ints([0])
    k, v = (bf(x) for x in rows(sum(lens), H, 20))
    kv4.quantize_append(cache, batch, k, v, ints(np.concatenate([[0], np.cumsum(lens)])), err)
    del k, v
    g = torch.Generator(device="cuda").manual_seed(21)
    q = bf(torch.randn((B, Hq, 128), generator=g, device="cuda"))
    out, lse = torch.empty_like(q), torch.empty((B, Hq), device="cuda")
    ws = torch.empty(kv4.workspace_size(cfg, B, max(lens)), dtype=torch.uint8, device="cuda")
    kv4.decode_attention(cache, batch, q, out, ws, None, lse, err)
    stride = max(lens) + 3
    old = torch.rand((B, H, stride), generator=g, device="cuda")
    acc = torch.full_like(old, -3.0)
    kv4.attention_weights(cache, batch, q, lse, acc, acc_in=old, err=err)
    place = old.clone()
    kv4.attention_weights(cache, batch, q, lse, place, acc_in=place, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    half = lambda x: x.view(torch.float16).double()  # noqa: E731
    for b, L in enumerate(lens):
        pg = torch.as_tensor(table[b, :-(-L // 16)]).cuda().long()
        c, par = cache.k_codes[pg], half(cache.k_params[pg])  # [n, H, 4, 16, 16], [n, H, 16, 4, 2]
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).double().transpose(2, 3)  # [n, H, 16, 4, 32]
        kk = (c * par[..., :1] + par[..., 1:]).flatten(-2).transpose(0, 1).reshape(H, -1, 128)[:, :L].clone()
        big = (15 * par[..., 0] + par[..., 1].abs()).repeat_interleave(32, -1)
        big = big.transpose(0, 1).reshape(H, -1, 128)[:, :L].clone()
        i = int(ids[b])
        for lo, hi, m, codes, sc in ((0, min(S, L), S, cache.sink_k, cache.sink_ks),
                                     (max(S, L - R), L, R, cache.ring_k, cache.ring_ks)):
            if hi > lo and m:
                t = torch.arange(lo, hi, device="cuda") % m
                x = codes[i].double().permute(0, 1, 3, 2, 4).reshape(H, -1, 128)[:, t]
                w = half(sc[i])[:, t, None]
                kk[:, lo:hi] = x * w
                big[:, lo:hi] = 127 * w
        qq, ll = q[b].double().reshape(H, G, 128), lse[b].double().reshape(H, G, 1)
        per = torch.exp(qq @ kk.transpose(1, 2) / math.sqrt(128) - ll)
        mag = qq.abs() @ big.transpose(1, 2) / math.sqrt(128) + ll.abs()
        # as for the weights' own tests: each of a logit's roundings is at most 2^-24 of its summed
        # magnitudes (128 products, 8 parameter terms, the scales' products); 2^x and the sums 2^-20
        tol = (per * (150 * 2.0 ** -24 * mag + 2.0 ** -20)).sum(1)
        want = per.sum(1) + old[b, :, :L].double()
        off = (acc[b, :, :L].double() - want).abs() / (tol + 2.0 ** -24 * want + 1e-12)
        assert bool((off <= 1).all()), (b, float(off.max()))
        assert torch.equal(place[b, :, :L], acc[b, :, :L])
        assert bool((acc[b, :, L:] == -3.0).all()) and torch.equal(place[b, :, L:], old[b, :, L:])


SELECT = [
    ([8193, 12001, 16384, 900], 2, 16, 128, 900),
    ([16384, 16383, 10000], 2, 0, 0, 9999),
    ([8193, 9000], 1, 4, 32, 36),  # no candidate stays
    ([2049, 4096, 8192], 2, 4, 32, 2048),
]


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("lens,H,S,R,budget", SELECT)
def test_select_of_long_rows(lens, H, S, R, budget, kind):
    kv4 = _kv4()
    cfg = kv4.make_config(H, H, S, R)
    B, stride = len(lens), max(lens) + 3
    rng = np.random.default_rng(sum(lens) + budget)
    acc = rng.standard_normal((B, H, stride)).astype(np.float32)
    if kind == "ties":
        acc = np.round(np.abs(acc), 1)
    elif kind == "equal":
        acc[:] = -0.5
    elif kind == "special":
        pick = rng.integers(0, 8, acc.shape)
        for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45)):
            acc[pick == i] = x
        acc[0, 0] = np.nan
    keep = torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda")
    new, err = ints([-9] * B), ints([0])
    batch = kv4.BatchTensors(ints(np.zeros((B, 1))), ints(lens), None, None, max(lens))
    kv4.evict_select(cfg, batch, torch.from_numpy(acc).cuda(), keep, new, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and new.tolist() == [min(L, budget) for L in lens]
    keep = keep.cpu().numpy()
    for b, L in enumerate(lens):
        for h in range(H):
            want = E.select(acc[b, h, :L], S, R, budget)
            assert keep[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
