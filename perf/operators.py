"""The measured cases of the 8-bit block-scaled cache and of cache eviction.

Five operators, each over a paged cache with pages of 16 positions and head_dim 128:

* ``block8_append``: new bf16 K/V rows into pages of 8-bit codes (INT8 or e4m3) with one
  fp16 scale per (page, kv head): the scale grows when a larger row arrives, and the codes
  already in the block are then rounded again under the new scale;
* ``block8_attention``: grouped-query attention over that cache, for one query per sequence
  (a decode step) or for each sequence's last n positions (a verification step of drafted
  tokens, a prefill chunk), causal;
* ``attention_weights``: each cached position's attention weight in a decode step, summed
  over the query heads of its kv head and added to a running total (INT4 pages with INT8
  sinks and recent window);
* ``evict_select``: the positions to keep per sequence and kv head: the sinks, the recent
  window, and the largest totals of the rest;
* ``evict_compact``: the kept positions' INT4 codes, parameters and totals moved to the
  front of a sequence's pages, and its ring of INT8 copies turned to the new positions.

``run`` computes each in plain torch operations, or, with ``own`` set, through the library.
Shapes are those of the decode batches in ``workload.py``: 32 query heads over 8 kv heads,
16 sinks, 128 recent positions (and the small test shape, 8 over 2 with 4 + 32).
"""
from __future__ import annotations

import math

import torch

own = False

D, PAGE, GROUP = 128, 16, 32
SCALE = 1.0 / math.sqrt(D)
MAXCODE = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = {"name": name, "op": op, "hq": 32, "hkv": 8, "sinks": 16, "recent": 128}
    c.update(kw)
    return c


def listed():
    return [
        # one new token for each sequence of the 1024-sequence rollout batch
        _case("append-token-1024", "append", fmt="int8", seqs=1024, lo=257, hi=4096, new_lo=1,
              new_hi=1, lens=11),
        # a ragged prefill: prompts and chunks that start and end inside pages
        _case("append-prefill-64", "append", fmt="e4m3", seqs=64, lo=700, hi=2048, new_lo=1,
              new_hi=1500, lens=12),
        # the smallest decode batch (the tiny test workload): latency
        _case("attend-tiny", "attend", fmt="int8", hq=8, hkv=2, seqs=4, lo=37, hi=511, new_lo=1,
              new_hi=1, lens=13),
        # a long-tail decode batch, lengths up to the 16,384-token response cap
        _case("attend-longtail-128", "attend", fmt="e4m3", seqs=128, lo=1, hi=16384, new_lo=1,
              new_hi=1, lens=14),
        # verification of a few drafted tokens per sequence over medium contexts
        _case("attend-verify-32", "attend", fmt="int8", seqs=32, lo=512, hi=8192, new_lo=2,
              new_hi=9, lens=15),
        # prefill chunks of two prompts over what is cached already
        _case("attend-prefill-2", "attend", fmt="int8", seqs=2, lo=7000, hi=8192, new_lo=3900,
              new_hi=4096, lens=16),
        # the 64 x 2048 layer batch, and a few of the longest rollouts
        _case("weights-64x2048", "weights", seqs=64, lo=2048, hi=2048, lens=17),
        _case("weights-longtail-48", "weights", seqs=48, lo=300, hi=16384, lens=18),
        # halving the contexts of a layer batch; trimming long rollouts to a quarter
        _case("select-64-to-1024", "select", seqs=64, lo=2048, hi=2048, budget=1024, lens=19),
        _case("select-128-to-4096", "select", seqs=128, lo=9001, hi=16384, budget=4096, lens=20),
        # one sequence trimmed alone (latency), and the layer batch
        _case("compact-1-to-500", "compact", seqs=1, lo=777, hi=777, budget=500, lens=21),
        _case("compact-64-to-1024", "compact", seqs=64, lo=900, hi=2048, budget=1024, lens=22),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weights", "select", "compact"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (8, 2), (16, 2), (4, 4), (12, 4)])
    s, r = rng.choice([(16, 128), (4, 32), (1, 17), (0, 100)])
    c = {"op": op, "hq": hq, "hkv": hkv, "sinks": s, "recent": r, "lens": rng.randrange(1 << 20)}
    tokens = _log(rng, 200, 500_000)  # cached positions of the batch, about
    hi = min(16384, _log(rng, 20, max(21, tokens)))
    c["hi"], c["lo"] = hi, rng.randint(1, hi)
    c["seqs"] = max(1, min(1024, tokens // hi))
    if op in ("append", "attend"):
        c["fmt"] = rng.choice(["int8", "e4m3"])
        if rng.random() < 0.5:
            c["new_lo"] = c["new_hi"] = 1
        else:  # at most as many (query, key) pairs as the largest listed case has
            top = max(2, min(hi, 40_000_000 // max(1, c["seqs"] * hi)))
            c["new_hi"] = _log(rng, 2, top)
            c["new_lo"] = rng.randint(1, c["new_hi"])
    if op in ("select", "compact"):
        c["budget"] = max(s + r, _log(rng, s + r, max(s + r, hi)))
    return c


def _lens(c):
    """Context lengths and new rows per sequence (host lists): part of the case, not of the seed."""
    g = torch.Generator().manual_seed(c["lens"])
    lens = torch.randint(c["lo"], c["hi"] + 1, (c["seqs"],), generator=g)
    new = torch.randint(c.get("new_lo", 1), c.get("new_hi", 1) + 1, (c["seqs"],), generator=g)
    return lens.tolist(), torch.minimum(new, lens).tolist()


def work(case):
    lens, new = _lens(case)
    H, Hq, S, R = case["hkv"], case["hq"], case["sinks"], case["recent"]
    T, N = sum(lens), sum(new)
    if case["op"] == "append":  # rows read, codes written, one scale per block read and written
        blocks = sum((L - 1) // PAGE - (L - n) // PAGE + 1 for L, n in zip(lens, new))
        return {"bytes": 2 * H * (N * D * (2 + 1) + 4 * blocks), "flops": 2 * N * H * D}
    if case["op"] == "attend":
        pairs = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, new))
        return {"bytes": 2 * T * H * D + N * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}
    if case["op"] == "weights":
        prot = sum(min(L, S + R) for L in lens)
        return {"bytes": H * ((T - prot) * 80 + prot * 130 + 8 * T) + len(lens) * Hq * (2 * D + 4),
                "flops": 2 * T * Hq * D}
    kept = sum(min(L, case["budget"]) for L in lens)
    if case["op"] == "select":
        return {"bytes": 4 * H * (T + kept), "flops": H * T}
    ring = sum(min(L, R) for L in lens)
    return {"bytes": H * (kept * (2 * 160 + 4 + 8) + ring * 2 * 260), "flops": H * kept}


# ------------------------------------------------------------------ inputs
def _values(g, pages, H, dev, key):
    """Rows of a page pool [pages, H, 16, 128], N(0, 1) as bf16; keys with 3 channels x10."""
    x = torch.randn((pages, H, PAGE, D), generator=g, device=dev, dtype=torch.float32)
    if key:
        x[..., torch.randperm(D, generator=g, device=dev)[:3]] *= 10.0
    return x.to(torch.bfloat16).float()


def _up16(x):
    """fp32 >= 0 to fp16, rounded up (at most 65504)."""
    h = x.clamp(max=65504.0).half()
    return torch.where(h.float() < x.clamp(max=65504.0), (h.view(torch.int16) + 1).view(torch.float16), h)


def _scale(x, fmt):
    """The fp16 scale of blocks of rows [..., 16, 128]: max|x| / (largest code), rounded up.
    (Divided by a tensor: torch takes a division by a plain number as a product.)"""
    top = x.abs().amax((2, 3))
    return _up16(top / torch.full_like(top, MAXCODE[fmt]))


def _round8(y, fmt):
    """x / scale in fp32 to the nearest code (ties to even), as numbers in fp32."""
    y = y.clamp(-MAXCODE[fmt], MAXCODE[fmt])
    return y.round() if fmt == "int8" else y.to(torch.float8_e4m3fn).float()


def _block8(x, fmt):
    """Rows [pages, H, 16, 128] to codes (fp32 numbers) and fp16 scales [pages, H]."""
    s = _scale(x, fmt)
    f = s.float()[..., None, None]
    return _round8(torch.where(f > 0, x / f, torch.zeros_like(x)), fmt), s


def _store(codes, fmt):
    """[pages, H, 16 slots, 128] numbers to the stored [pages, H, 8 strips, 16 slots, 16]."""
    dt = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    return codes.reshape(*codes.shape[:2], PAGE, 8, 16).transpose(2, 3).contiguous().to(dt)


def _rows8(codes):
    """Stored 8-bit codes [..., 8, 16 slots, 16] as fp32 numbers [..., 16 slots, 128]."""
    return codes.float().transpose(-3, -2).flatten(-2)


def _int4(x):
    """Rows [pages, H, 16, 128] to INT4 codes [pages, H, 4, 16, 16] and (scale, min) bits."""
    p, h = x.shape[:2]
    x = x.reshape(p, h, PAGE, 4, GROUP)
    mn, mx = x.amin(-1), x.amax(-1)
    m16, s16 = mn.half(), ((mx - mn) / 15).half()
    s = s16.float()[..., None]
    c = ((x - m16.float()[..., None]) / s).round().clamp(0, 15).to(torch.uint8)
    c = c.permute(0, 1, 3, 2, 4)  # [pages, H, 4, 16, 32]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), torch.stack([s16, m16], -1).view(torch.int16)


def _int8(x):
    """Rows [n, H, slots, 128] to INT8 tiles [n, H, tiles, 8, 16, 16] and scale bits [n, H, slots]."""
    n, h, m = x.shape[:3]
    s16 = (x.abs().amax(-1) / 127).half()
    c = (x / s16.float()[..., None]).round().clamp(-127, 127).to(torch.int8)
    c = c.reshape(n, h, m // PAGE, PAGE, 8, 16).transpose(3, 4).contiguous()
    return c, s16.view(torch.int16).contiguous()


def _table(g, lens, dev, spare=0):
    """Page table [B, max pages] over shuffled physical pages (-1 behind a sequence's end)."""
    need = torch.tensor([-(-n // PAGE) for n in lens])
    first = torch.cumsum(need, 0) - need
    i = torch.arange(int(need.max()))[None, :]
    t = torch.where(i < need[:, None], first[:, None] + i, torch.full_like(i, -1)).to(dev)
    pages = int(need.sum())
    perm = torch.randperm(pages + spare, generator=g, device=dev)
    return torch.where(t >= 0, perm[t.clamp(min=0)], t).to(torch.int32), pages, perm[pages:].to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lens(case)
    B, H, Hq, S, R = case["seqs"], case["hkv"], case["hq"], case["sinks"], case["recent"]
    budget = case.get("budget", 0)
    spare = sum(-(-min(n, budget) // PAGE) for n in lens) if case["op"] == "compact" else 0
    table, pages, rest = _table(g, lens, dev, spare)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": case, "table": table, "lens": ints(lens), "max_len": max(lens)}
    if case["op"] in ("append", "attend"):
        fmt = case["fmt"]
        for x, key in (("k", True), ("v", False)):
            c, sc = _block8(_values(g, pages, H, dev, key), fmt)
            s[x], s[x + "s"] = _store(c, fmt), sc
        ragged = case["new_hi"] > 1
        s["indptr"] = ints([0] + torch.tensor(new).cumsum(0).tolist()) if ragged else None
        s["new"], s["max_new"] = ints(new), max(new)
        n = sum(new)
        if case["op"] == "append":
            for x in ("k", "v"):
                s[x + "_new"] = torch.randn((n, H, D), generator=g, device=dev).to(torch.bfloat16)
        else:
            s["q"] = torch.randn((n, Hq, D), generator=g, device=dev).to(torch.bfloat16)
        return s
    if case["op"] in ("weights", "compact"):
        st, rt = -(-S // PAGE) * PAGE, -(-R // PAGE) * PAGE
        rings = B if case["op"] == "weights" else 2 * B
        side = lambda n, m: _int8(torch.randn((n, H, max(PAGE, m), D), generator=g, device=dev))  # noqa: E731
        for x in ("k", "v"):
            s["sink_" + x], s["sink_%ss" % x] = side(B, st)
            s["ring_" + x], s["ring_%ss" % x] = side(rings, rt)
            s[x], s[x + "p"] = _int4(_values(g, pages + spare, H, dev, False))
        s["ids"] = torch.randperm(B, generator=g, device=dev).to(torch.int32)
    stride = table.shape[1] * PAGE
    s["acc"] = torch.rand((B, H, stride), generator=g, device=dev) ** 8  # totals: a few large, many small
    s["acc"][torch.rand((B, H, stride), generator=g, device=dev) < 0.2] = 0.0
    if case["op"] == "weights":
        s["q"] = torch.randn((B, Hq, D), generator=g, device=dev).to(torch.bfloat16)
        s["lse"] = _cache_logits(s).logsumexp(-1).reshape(B, Hq)
        s["acc_out"] = torch.full_like(s["acc"], -1.0)
    else:
        s["keep"] = torch.full((B, H, budget), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    if case["op"] == "compact":
        s["keep"], s["new_lens"] = _select(s)
        need = -(-s["new_lens"] // PAGE)
        first = torch.cumsum(need, 0) - need
        i = torch.arange(-(-budget // PAGE), device=dev)[None, :]
        to = rest[(first[:, None] + i).clamp(max=max(0, spare - 1)).long()]
        s["to"] = torch.where(i < need[:, None], to, torch.full_like(to, -1)).contiguous()
        s["to_ids"] = s["ids"] + B
        s["acc_out"] = torch.full((B, H, budget), -1.0, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s):
    return torch.arange(s["table"].shape[1] * PAGE, device=s["table"].device)


def _cached(s, x):
    """The 8-bit cache's values, padded: fp32 [B, H, positions, 128] (rows behind a length: 0)."""
    c = _rows8(s[x]) * s[x + "s"].float()[..., None, None]
    c = c[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)
    return c.masked_fill_((_positions(s) >= s["lens"][:, None])[:, None, :, None], 0.0)


def _append(s):
    fmt, dev = s["case"]["fmt"], s["table"].device
    new, lens = s["new"].long(), s["lens"].long()
    n = s["k_new"].shape[0]
    b = torch.repeat_interleave(torch.arange(len(lens), device=dev), new, output_size=n)
    pos = (lens - new - (new.cumsum(0) - new))[b] + torch.arange(n, device=dev)
    page, slot = s["table"][b, pos // PAGE].long(), pos % PAGE
    pages = s["k"].shape[0]
    # slots of each page before this call's first row keep their codes, the others are new or free
    first = torch.full((pages,), PAGE, device=dev).scatter_reduce_(0, page, slot, "amin")
    hit = torch.zeros(pages, dtype=torch.bool, device=dev).index_fill_(0, page, True).nonzero()[:, 0]
    at = torch.full((pages,), -1, device=dev).index_put_((hit,), torch.arange(len(hit), device=dev))
    held = (torch.arange(PAGE, device=dev) < first[hit][:, None])[:, None, :, None]
    for x in ("k", "v"):
        rows = torch.zeros((len(hit), s[x].shape[1], PAGE, D), device=dev)
        rows[at[page], :, slot] = s[x + "_new"].float()
        old = s[x + "s"][hit]
        scale = _scale(rows, fmt)
        scale = torch.where(first[hit][:, None] > 0, torch.maximum(scale, old), scale)
        f = scale.float()[..., None, None]
        was = _rows8(s[x][hit])
        y = torch.where(held, was * old.float()[..., None, None], rows) / f
        codes = _round8(torch.where(f > 0, y, torch.zeros_like(y)), fmt)
        fresh = torch.zeros((len(hit), PAGE), dtype=torch.bool, device=dev)
        fresh[at[page], slot] = True
        codes = torch.where(held | fresh[:, None, :, None], codes, was)
        s[x][hit] = _store(codes, fmt)
        s[x + "s"][hit] = scale
    return {x: s[x] for x in ("k", "v", "ks", "vs")}


def _attend(s):
    c = s["case"]
    H, Hq = c["hkv"], c["hq"]
    B, n = len(s["lens"]), s["max_new"]
    i = torch.arange(n, device=s["q"].device)
    row = (s["new"].cumsum(0) - s["new"])[:, None] + i  # row of sequence b's i-th query
    live = i < s["new"][:, None]
    q = s["q"][torch.where(live, row, 0).long()].float()  # [B, n, Hq, 128]
    q = q.reshape(B, n, H, Hq // H, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    logits = q @ _cached(s, "k").transpose(-1, -2) * SCALE  # [B, H, n * G, positions]
    seen = _positions(s) <= (s["lens"] - s["new"])[:, None, None] + i[:, None]
    seen = seen.repeat_interleave(Hq // H, 1)[:, None]
    logits = logits.masked_fill_(~seen, -math.inf)
    lse = logits.logsumexp(-1)
    o = torch.exp(logits.sub_(lse[..., None])) @ _cached(s, "v")
    o = o.reshape(B, H, n, Hq // H, D).transpose(1, 2).reshape(B, n, Hq, D)
    lse = lse.reshape(B, H, n, Hq // H).transpose(1, 2).reshape(B, n, Hq)
    return {"out": o[live].to(torch.bfloat16), "lse": lse[live]}


def _cache_logits(s):
    """Logits of a decode step over the INT4 cache with its INT8 copies: fp32 [B, H, G, positions]."""
    c = s["case"]
    S, R, H, B = c["sinks"], c["recent"], c["hkv"], len(s["lens"])
    q = s["q"].float().reshape(B, H, -1, D)
    codes = torch.stack([s["k"] & 15, s["k"] >> 4], -1).flatten(-2).float()  # [pages, H, 4, 16, 32]
    p = s["kp"].view(torch.float16).float().transpose(2, 3)  # [pages, H, 4, 16, 2]
    rows = (codes * p[..., :1] + p[..., 1:]).transpose(2, 3).flatten(-2)
    rows = rows[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)
    logits = q @ rows.transpose(-1, -2) * SCALE
    pos, L = _positions(s), s["lens"][:, None]
    ids = s["ids"].long()
    copies = lambda x: (_rows8(s[x]).flatten(2, 3) * s[x + "s"].view(torch.float16).float()[..., None])[ids]  # noqa: E731
    if S:
        m = min(S, len(pos))
        logits[..., :m] = (q @ copies("sink_k").transpose(-1, -2) * SCALE)[..., :m]
    if R:
        ring = q @ copies("ring_k").transpose(-1, -2) * SCALE
        near = (pos >= torch.clamp(L - R, min=S))[:, None, None, :]
        logits = torch.where(near, ring[..., pos % R], logits)
    return logits.masked_fill((pos >= L)[:, None, None, :], -math.inf)


def _weights(s):
    B, H = s["acc"].shape[:2]
    w = torch.exp(_cache_logits(s) - s["lse"].reshape(B, H, -1, 1)).sum(2)
    return {"acc": torch.where(_positions(s) < s["lens"][:, None, None], s["acc"] + w, s["acc_out"])}


def _select(s):
    c = s["case"]
    S, R, n = c["sinks"], c["recent"], c["budget"]
    pos, L = _positions(s), s["lens"][:, None, None]
    kept = (pos < S) | (pos >= L - R)
    score = torch.where(kept, torch.full_like(s["acc"], math.inf), s["acc"])
    score = torch.where(pos < L, score, torch.full_like(score, -math.inf))
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    if best.shape[-1] < n:
        best = torch.nn.functional.pad(best, (0, n - best.shape[-1]), value=len(pos))
    best = best.sort(dim=-1).values.to(torch.int32)
    return torch.where(best < L, best, torch.full_like(best, -1)), s["lens"].clamp(max=n)


def _compact(s):
    c, dev = s["case"], s["table"].device
    S, R, n = c["sinks"], c["recent"], c["budget"]
    B, H = s["keep"].shape[:2]
    j = torch.arange(n, device=dev)
    b, jj = (j < s["new_lens"][:, None]).nonzero(as_tuple=True)  # every kept row of every sequence
    src = s["keep"].transpose(1, 2)[b, jj].long()  # [rows, H]: position of each head
    h = torch.arange(H, device=dev)
    sp, ss = s["table"][b[:, None], src // PAGE].long(), src % PAGE
    dp, ds = s["to"][b, jj // PAGE].long()[:, None], (jj % PAGE)[:, None]
    for x in ("k", "v"):
        s[x][dp, h, :, ds] = s[x][sp, h, :, ss]
        s[x + "p"][dp, h, ds] = s[x + "p"][sp, h, ss]
    s["acc_out"][b[:, None], h, jj[:, None]] = s["acc"][b[:, None], h, src]
    # the ring: the copy of the position now at p' (before: p' + what was taken out) in slot p' mod R
    slot = torch.arange(R, device=dev)
    new, old = s["new_lens"].long()[:, None], s["lens"].long()[:, None]
    p = new - 1 - (new - 1 - slot) % R if R else slot
    b, to = ((p >= S) & (p >= new - R) & (p >= 0)).nonzero(as_tuple=True)
    src = ((p + old - new) % R)[b, to] if R else to
    fr, tr = s["ids"].long()[b], s["to_ids"].long()[b]
    for x in ("k", "v"):
        s["ring_" + x][tr, :, to // PAGE, :, to % PAGE] = s["ring_" + x][fr, :, src // PAGE, :, src % PAGE]
        s["ring_%ss" % x][tr, :, to] = s["ring_%ss" % x][fr, :, src]
    return _compacted(s)


def _compacted(s):
    names = ("k", "v", "kp", "vp", "ring_k", "ring_v", "ring_ks", "ring_vs", "acc_out")
    return {x: s[x] for x in names}


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    if op == "select":
        keep, lens = _select(state)
        return {"keep": keep, "lens": lens}
    return {"append": _append, "attend": _attend, "weights": _weights, "compact": _compact}[op](state)


# ------------------------------------------------------------------ the library's calls
def _handles(s):
    """The objects that a user's program holds: the cache, the batch, the workspace."""
    from quantized_kv_cache_kv4_b200 import kv4
    if "cache" not in s:
        c = s["case"]
        cfg = kv4.make_config(c["hq"], c["hkv"], c["sinks"], c["recent"])
        ids = s.get("ids", s["lens"])
        s["batch"] = kv4.BatchTensors(s["table"], s["lens"], ids, ids, s["max_len"])
        if c["op"] in ("append", "attend"):
            fmt = kv4.BLOCK8_INT8 if c["fmt"] == "int8" else kv4.BLOCK8_E4M3
            s["cache"] = kv4.Block8Cache(fmt, cfg, s["k"], s["v"], s["ks"], s["vs"])
        elif c["op"] == "select":
            s["cache"] = cfg
        else:
            s["cache"] = kv4.Cache(cfg, s["k"], s["v"], s["kp"], s["vp"], s["sink_k"], s["sink_v"],
                                   s["sink_ks"], s["sink_vs"], s["ring_k"], s["ring_v"], s["ring_ks"],
                                   s["ring_vs"])
        if c["op"] == "attend":
            n = kv4.block8_workspace_size(cfg, c["seqs"], s["q"].shape[0], s["max_new"], s["max_len"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return kv4, s["cache"], s["batch"]


def _own_append(s):
    kv4, cache, batch = _handles(s)
    kv4.block8_append(cache, batch, s["k_new"], s["v_new"], s["indptr"])
    return {x: s[x] for x in ("k", "v", "ks", "vs")}


def _own_attend(s):
    kv4, cache, batch = _handles(s)
    kv4.block8_attention(cache, batch, s["q"], s["out"], s["workspace"], s["indptr"], s["max_new"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_weights(s):
    kv4, cache, batch = _handles(s)
    kv4.attention_weights(cache, batch, s["q"], s["lse"], s["acc_out"], acc_in=s["acc"])
    return {"acc": s["acc_out"]}


def _own_select(s):
    kv4, cfg, batch = _handles(s)
    kv4.evict_select(cfg, batch, s["acc"], s["keep"], s["new_lens"])
    return {"keep": s["keep"], "lens": s["new_lens"]}


def _own_compact(s):
    kv4, cache, batch = _handles(s)
    kv4.evict_compact(cache, batch, s["keep"], s["new_lens"], dst_page_table=s["to"], dst_ring_idx=s["to_ids"],
                      acc_in=s["acc"], acc_out=s["acc_out"])
    return _compacted(s)


_OWN = {"append": _own_append, "attend": _own_attend, "weights": _own_weights, "select": _own_select,
        "compact": _own_compact}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3(y):
    """The nearest e4m3 number to y (fp64), ties to even, from its 3 mantissa bits."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_append(s):
    """One block at a time would be slow: every touched (sequence, page) pair as one row of a batch."""
    fmt, dev = s["case"]["fmt"], s["table"].device
    top = MAXCODE[fmt]
    out = {x: s[x].double().clone() for x in ("k", "v", "ks", "vs")}
    starts = [0] + s["new"].long().cumsum(0).tolist()
    pages, rows, slots = [], [], []
    table = s["table"].cpu()
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        for p in range((L - n) // PAGE, (L - 1) // PAGE + 1):
            lo, hi = max(L - n, p * PAGE), min(L, p * PAGE + PAGE)
            pages.append(int(table[b, p]))
            rows.append(starts[b] + lo - (L - n))
            slots.append((lo - p * PAGE, hi - p * PAGE))
    pages, rows = torch.tensor(pages, device=dev), torch.tensor(rows, device=dev)
    lo, hi = torch.tensor(slots, device=dev).unbind(1)
    i = torch.arange(PAGE, device=dev)
    isnew = (i >= lo[:, None]) & (i < hi[:, None])
    at = (rows[:, None] + i - lo[:, None]).clamp(0, s["k_new"].shape[0] - 1)
    for x in ("k", "v"):
        fresh = s[x + "_new"].double()[at].transpose(1, 2)  # [blocks, H, 16, 128]
        fresh = torch.where(isnew[:, None, :, None], fresh, torch.zeros_like(fresh))
        want = fresh.abs().amax((2, 3)) / top
        e = torch.floor(torch.log2(want.clamp(min=2.0 ** -14))) - 10  # fp16's step at `want`
        want = (torch.ceil(want / torch.exp2(e)) * torch.exp2(e)).clamp(max=65504.0)
        old = out[x + "s"][pages]
        sc = torch.where(lo[:, None] > 0, torch.maximum(want, old), want)
        was = out[x][pages].transpose(2, 3).flatten(3)
        y = torch.where(isnew[:, None, :, None], fresh, was * old[..., None, None]) / sc[..., None, None]
        y = torch.where(sc[..., None, None] > 0, y, torch.zeros_like(y))
        y = torch.round(y).clamp(-top, top) if fmt == "int8" else _e4m3(y)
        y = torch.where((i < hi[:, None])[:, None, :, None], y, was)
        out[x][pages] = y.reshape(*y.shape[:3], 8, 16).transpose(2, 3)
        out[x + "s"][pages] = sc
    if fmt == "int8":
        out["k"], out["v"] = out["k"].to(torch.int8), out["v"].to(torch.int8)
    return out


def _exact_attend(s):
    c = s["case"]
    H, G = c["hkv"], c["hq"] // c["hkv"]
    out, lse, at = [], [], 0
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        ids = s["table"][b, :-(-L // PAGE)].long()
        k, v = ((s[x][ids].double() * s[x + "s"][ids].double()[..., None, None, None]).permute(1, 0, 3, 2, 4)
                .reshape(H, -1, D)[:, :L] for x in ("k", "v"))
        o_b, l_b = [], []
        for i in range(0, n, 512):
            q = s["q"][at + i:at + min(n, i + 512)].double().reshape(-1, H, G, D)
            t = torch.einsum("nhgd,hld->hgnl", q, k) * SCALE
            last = L - n + i + torch.arange(q.shape[0], device=q.device)
            t = t.masked_fill(torch.arange(L, device=q.device) > last[:, None], -math.inf)
            m = t.amax(-1, keepdim=True)
            e = torch.exp(t - m)
            z = e.sum(-1, keepdim=True)
            o_b.append(torch.einsum("hgnl,hld->nhgd", e / z, v).reshape(-1, H * G, D))
            l_b.append((m + torch.log(z)).squeeze(-1).permute(2, 0, 1).reshape(-1, H * G))
        out += o_b
        lse += l_b
        at += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_weights(s):
    c = s["case"]
    S, R, H, G = c["sinks"], c["recent"], c["hkv"], c["hq"] // c["hkv"]
    acc = s["acc_out"].double().clone()
    half = lambda x: x.view(torch.float16).double()  # noqa: E731
    for b, L in enumerate(s["lens"].tolist()):
        ids = s["table"][b, :-(-L // PAGE)].long()
        codes, par = s["k"][ids], half(s["kp"][ids])  # [n, H, 4, 16, 16], [n, H, 16, 4, 2]
        k = torch.empty((len(ids), H, PAGE, D), dtype=torch.float64, device=codes.device)
        for gr in range(4):
            for nib in range(2):
                x = ((codes[:, :, gr] >> (4 * nib)) & 15).double()
                k[..., GROUP * gr + nib:GROUP * gr + GROUP:2] = x * par[..., gr, :1] + par[..., gr, 1:]
        k = k.transpose(0, 1).reshape(H, -1, D)[:, :L]
        i = int(s["ids"][b])
        for p0, p1, name, m in ((0, min(S, L), "sink", S), (max(S, L - R), L, "ring", R)):
            if p1 > p0 and m:
                at = torch.arange(p0, p1, device=k.device) % m
                rows = s[name + "_k"][i][:, at // PAGE, :, at % PAGE].double().flatten(2)
                k[:, p0:p1] = (rows.transpose(0, 1) if rows.shape[0] != H else rows) * half(s[name + "_ks"][i])[:, at, None]
        q = s["q"][b].double().reshape(H, G, D)
        w = torch.exp(torch.einsum("hgd,hld->hgl", q, k) * SCALE - s["lse"][b].double().reshape(H, G, 1)).sum(1)
        acc[b, :, :L] = s["acc"][b, :, :L].double() + w
    return {"acc": acc}


def exact(case, seed):
    if case["op"] in ("select", "compact"):
        return None  # whole numbers, and rows that are moved: nothing is rounded
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "weights": _exact_weights}[case["op"]](s)
