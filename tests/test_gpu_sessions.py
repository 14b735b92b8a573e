"""The operators run together, as a program runs them: decode steps over a KV4 cache that is
evicted on the way, and decode and verification steps over a block-scaled 8-bit cache."""
import numpy as np
import pytest
import torch

from oracle import block8_oracle as O8
from oracle import evict_oracle as E
from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu

TOL = 2e-3  # of the output's scale, as in the parity tests of the attention


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from quantized_kv_cache_kv4_b200 import build
    build.build()


def _mods():
    from quantized_kv_cache_kv4_b200 import kv4, session, workload
    return kv4, session, workload


def magnitude(q, k, S, R):
    """Per position and query head of one kv head: the sum of magnitudes a logit is summed from
    (INT4: |q| (15 scale + |min|); INT8: |q| 127 scale), / sqrt(128). k [L, 1, 128]."""
    _, s4, m4 = O.quantize_int4(k)
    big = np.repeat(15 * s4.astype(np.float64) + np.abs(m4.astype(np.float64)), 32, -1)
    _, s8 = O.quantize_int8(k)
    prot = O.protected_mask(len(k), S, R)
    big[prot] = 127 * s8.astype(np.float64)[prot][..., None]
    return np.abs(q.astype(np.float64)) @ big[:, 0].T / np.sqrt(128)


RUNS = [  # lengths at the first step, Hq, Hkv, S, R, budget, steps after which it is evicted
    ("plain", [70, 33, 200, 1], 8, 2, 4, 32, 60, (1, 4, 5)),
    ("each-step", [90, 64, 65], 8, 2, 4, 32, 64, (0, 1, 2, 3, 4, 5, 6)),
    ("gqa1-no-sinks", [150, 31], 2, 2, 0, 16, 40, (2, 5)),
    ("gqa8-no-recent", [150, 47], 16, 2, 5, 0, 48, (2, 5)),
    ("window-only", [150, 47], 8, 2, 4, 32, 36, (0, 3)),
    ("no-protection", [80, 17], 8, 2, 0, 0, 17, (1, 2)),
]


@pytest.mark.parametrize("demotion", ["A", "B"])
@pytest.mark.parametrize("name,lens,Hq,Hkv,S,R,budget,when", RUNS, ids=[r[0] for r in RUNS])
def test_decode_steps_with_eviction(name, lens, Hq, Hkv, S, R, budget, when, demotion):
    _, session, workload = _mods()
    steps, B, G = 8, len(lens), Hq // Hkv
    wl = workload.custom_workload(lens, num_q_heads=Hq, num_kv_heads=Hkv, num_sinks=S, num_recent=R,
                                  seed=31, outlier_channels=2, outlier_scale=6.0)
    s = session.DecodeSession(wl, steps=steps, keep_streams=range(B), demotion=demotion)
    # the stream's positions that each (sequence, kv head) holds, in cache order
    held = [[list(range(L - 1)) for _ in range(Hkv)] for L in lens]
    want = [[np.zeros(L - 1) for _ in range(Hkv)] for L in lens]
    slack = [[np.zeros(L - 1) for _ in range(Hkv)] for L in lens]
    o32 = torch.empty((B, Hq, 128), device="cuda")
    lse = torch.empty((B, Hq), device="cuda")
    for step in range(steps):
        s.fused_step(step, out_f32=o32, lse=lse)
        s.weigh_step(step, lse)
        torch.cuda.synchronize()
        s.check_err()
        got, gl, totals = o32.cpu().numpy(), lse.cpu().numpy(), s.totals.cpu().numpy()
        for b, L in enumerate(lens):
            k, v = s.streams[b]
            q = s.q[step, b].float().cpu().numpy()
            for h in range(Hkv):
                held[b][h].append(L - 1 + step)
                at, hq = held[b][h], slice(h * G, h * G + G)
                K, V = O.effective_kv(k[at, h:h + 1], v[at, h:h + 1], S, R, demotion)
                ref, lr = O.attention(q[hq], K, V)
                assert np.abs(got[b, hq] - ref).max() <= TOL * max(1e-30, np.abs(ref).max()), (step, b, h)
                assert np.all(np.abs(gl[b, hq] - lr) <= TOL * np.maximum(1, np.abs(lr))), (step, b, h)
                # totals: a logit's roundings are each at most 2^-24 of its summed magnitudes (128
                # products, 8 parameter terms, the scales' products), 2^x and the sums a few 2^-22
                per = np.exp(q[hq].astype(np.float64) @ K[:, 0].T / np.sqrt(128) - gl[b, hq, None].astype(np.float64))
                mag = magnitude(q[hq], k[at, h:h + 1], S, R) + np.abs(gl[b, hq, None])
                w = E.weights(q[hq], K, gl[b, hq], G)[0]
                want[b][h] = np.append(want[b][h], 0.0) + w
                slack[b][h] = np.append(slack[b][h], 0.0) + (per * (150 * 2.0 ** -24 * mag + 2.0 ** -20)).sum(0)
                slack[b][h] += 2.0 ** -24 * want[b][h] + 1e-12
                assert np.all(np.abs(totals[b, h, :len(at)] - want[b][h]) <= slack[b][h]), (step, b, h)
                assert np.all(totals[b, h, len(at):] == 0)
        if step in when:
            keep, new = s.evict(step, budget)
            torch.cuda.synchronize()
            s.check_err()
            keep, new = keep.cpu().numpy(), new.cpu().numpy()
            for b in range(B):
                for h in range(Hkv):
                    n = len(held[b][h])
                    kept = E.select(totals[b, h, :n], S, R, budget)
                    assert new[b] == len(kept) == min(n, budget)
                    assert np.array_equal(keep[b, h, :new[b]], kept), (step, b, h)
                    held[b][h] = [held[b][h][p] for p in kept]
                    want[b][h], slack[b][h] = want[b][h][kept], slack[b][h][kept]


def test_eviction_is_refused_where_it_cannot_run():
    kv4, session, workload = _mods()
    wl = workload.custom_workload([80, 80], prompt_len=32, group_seqs=2)
    s = session.DecodeSession(wl)
    s.append_step(0)
    with pytest.raises(ValueError):
        s.evict(0, 40)  # pages of the prompt are shared
    s = session.DecodeSession(workload.custom_workload([80, 80]))
    with pytest.raises(ValueError):
        s.evict(0, 40)  # no totals yet
    s = session.BaselineSession(workload.custom_workload([80, 80]), kv4.BASELINE_KV8)
    with pytest.raises(NotImplementedError):
        s.weigh_step(0, torch.zeros((2, 8), device="cuda"))
    with pytest.raises(NotImplementedError):
        s.evict(0, 40)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,prompt,group", [([75, 33, 130, 1], 0, 1), ([90, 49, 64, 200], 32, 2)],
                         ids=["own-prompts", "shared-prompts"])
def test_block8_session(fmt, lens, prompt, group):
    """Decode steps, then the last positions of every sequence verified in one call."""
    kv4, session, workload = _mods()
    wl = workload.custom_workload(lens, seed=5, prompt_len=prompt, group_seqs=group)
    B, steps, H, Hq = len(lens), 6, wl.num_kv_heads, wl.num_q_heads
    G = Hq // H
    s = session.Block8Session(wl, fmt=kv4.BLOCK8_INT8 if fmt == "int8" else kv4.BLOCK8_E4M3, steps=steps,
                              keep_streams=range(B))
    blocks = {}

    def appended(b, p, end):  # one call's positions
        while p < end:
            hi = min(end, p // 16 * 16 + 16)
            for x in range(2):
                for h in range(H):
                    blk = blocks.setdefault((b, x, h, p // 16), O8.Block(fmt))
                    blk.append(p % 16, s.streams[b][x][p:hi, h])
            p = hi

    def values(b, L):
        out = np.zeros((2, L, H, 128))
        for p in range(0, L, 16):
            for x in range(2):
                for h in range(H):
                    blk = blocks[(b, x, h, p // 16)]
                    out[x, p:p + 16, h] = (blk.codes * blk.scale)[:L - p]
        return out

    def close(got, lse, ref, lr, A, mag, L):
        # counted as for the attention's own tests: logits, weights as fp16, fp32 sums; weights that
        # fp16 holds as subnormals are off by 2^-38 of the largest value scale (below 1 here), times
        # codes of at most 448, over at most L rows
        ds = (130 * 2.0 ** -24 + 2.0 ** -21) * mag + 2.0 ** -21
        tol = (2.0 ** -11 + 2 * ds[..., None] + (L + 64) * 2.0 ** -24) * A + L * 2.0 ** -29
        assert np.all(np.abs(got - ref) <= tol)
        assert np.all(np.abs(lse - lr) <= ds + 2.0 ** -20 * np.maximum(1, np.abs(lr)))

    for b, L in enumerate(lens):
        P = prompt if prompt else 0
        appended(b, 0, min(P, L - 1))
        appended(b, P, L - 1)
    o32, lse = torch.empty((B, Hq, 128), device="cuda"), torch.empty((B, Hq), device="cuda")
    for step in range(steps):
        s.step(step, out_f32=o32, lse=lse)
        torch.cuda.synchronize()
        s.check_err()
        for b, L in enumerate(lens):
            appended(b, L - 1 + step, L + step)
            K, V = values(b, L + step)
            ref = O8.attention(s.q[step, b:b + 1].float().cpu().numpy(), K, V, G)
            close(o32[b].cpu().numpy(), lse[b].cpu().numpy(), *(x[0] for x in ref), L + step)
    n = [min(steps, L) for L in lens]
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((sum(n), Hq, 128), generator=g, device="cuda").to(torch.bfloat16)
    out, o32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    ip = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    s.verify_step(steps - 1, q, out, ip, max(n), s.verify_workspace(sum(n), max(n)), o32, lse)
    torch.cuda.synchronize()
    s.check_err()
    at = 0
    for b, L in enumerate(lens):
        K, V = values(b, L + steps - 1)
        ref = O8.attention(q[at:at + n[b]].float().cpu().numpy(), K, V, G)
        close(o32[at:at + n[b]].cpu().numpy(), lse[at:at + n[b]].cpu().numpy(), *ref, L + steps - 1)
        at += n[b]
    with pytest.raises(NotImplementedError):
        s.evict(0, 40)


def test_eviction_on_the_steps_stream():
    """Steps, weights and evictions on a side stream that lags behind, next to work on the current
    stream: nothing of them runs, or reads a length, before the step that it follows."""
    _, session, workload = _mods()
    steps, budget, runs = 5, 70, []
    for side in (None, torch.cuda.Stream()):
        wl = workload.custom_workload([90, 200, 33], num_q_heads=8, num_kv_heads=2, num_sinks=4, num_recent=32,
                                      seed=33)
        s = session.DecodeSession(wl, steps=steps)
        outs = [torch.zeros((3, 8, 128), device="cuda") for _ in range(steps)]
        lse = torch.zeros((3, 8), device="cuda")
        torch.cuda.synchronize()
        kept = []
        for step in range(steps):
            if side is not None:
                with torch.cuda.stream(side):
                    torch.cuda._sleep(20_000_000)  # ~10 ms: what does not follow the step runs before it
            s.fused_step(step, out_f32=outs[step], lse=lse, stream=side)
            s.weigh_step(step, lse, stream=side)
            if step in (1, 3):
                kept += s.evict(step, budget, stream=side)
        torch.cuda.synchronize()
        s.check_err()
        runs.append(outs + kept + [s.totals, s.step_lens])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert int(runs[0][-1][-1].max()) == budget + 1
