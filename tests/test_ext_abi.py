"""Host-side checks of the block-scaled cache's and the eviction's entry points: refused calls
return before anything is launched, so these run without a GPU."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def kv4():
    from quantized_kv_cache_kv4_b200 import build
    build.build()
    from quantized_kv_cache_kv4_b200 import kv4 as m
    return m


FAKE = 0x10000  # an aligned address nothing reads: every call here is refused


def structs(kv4, **kw):
    cfg = kv4.make_config(kw.pop("hq", 8), kw.pop("hkv", 2), kw.pop("S", 4), kw.pop("R", 32))
    pool = kv4.PagedPool(FAKE, FAKE, FAKE, FAKE, 10)
    int4 = kv4.Int4Pool(FAKE, FAKE, FAKE, FAKE, 10)
    side = kv4.Int8Side(FAKE, FAKE, FAKE, FAKE, 2, FAKE, FAKE, FAKE, FAKE, 2)
    batch = kv4.Batch(FAKE, 4, FAKE, FAKE, FAKE, kw.pop("B", 2), kw.pop("max_len", 64), 0)
    assert not kw
    return cfg, pool, int4, side, batch


def test_block8_append_refusals(kv4):
    cfg, pool, _, _, batch = structs(kv4)
    r = ctypes.byref

    def call(fmt=1, c=cfg, p=pool, b=batch, k=FAKE, v=FAKE, ip=None, n=2):
        return kv4._lib.kv4_block8_append(fmt, r(c) if c else None, r(p) if p else None, r(b) if b else None,
                                          k, v, ip, n, None, None)

    for bad in (dict(fmt=0), dict(fmt=3), dict(c=None), dict(p=None), dict(b=None), dict(k=None), dict(v=None),
                dict(k=FAKE + 2), dict(n=-1), dict(n=3)):
        assert call(**bad) == -1, bad
    for field in ("k", "v", "k_scales", "v_scales"):
        for value in (0, FAKE + 8):
            broken = kv4.PagedPool(FAKE, FAKE, FAKE, FAKE, 10)
            setattr(broken, field, value)
            assert call(p=broken) == -1, (field, value)
    shape = kv4.make_config(8, 3, 0, 0)
    assert call(c=shape) == -2
    wide = kv4.make_config(18, 2, 0, 0)
    assert call(c=wide) == -2
    assert call(ip=FAKE, n=0) == 0  # nothing to do
    empty = kv4.Batch(FAKE, 4, FAKE, FAKE, FAKE, 0, 64, 0)
    assert call(b=empty, n=0) == 0


def test_block8_attention_refusals(kv4):
    cfg, pool, _, _, batch = structs(kv4)
    r = ctypes.byref
    size = kv4.block8_workspace_size(cfg, 2, 2, 1, 64)

    def call(fmt=1, c=cfg, p=pool, b=batch, q=FAKE, ip=None, n=2, m=1, out=FAKE, f=None, ws=FAKE, bytes_=size):
        return kv4._lib.kv4_block8_attention(fmt, r(c), r(p), r(b), q, ip, n, m, out, f, None, ws, bytes_, None,
                                             None)

    for bad in (dict(fmt=7), dict(q=None), dict(out=None), dict(ws=None), dict(ws=FAKE + 16), dict(q=FAKE + 4),
                dict(out=FAKE + 4), dict(f=FAKE + 4), dict(n=-1), dict(m=-1), dict(n=3), dict(m=2)):
        assert call(**bad) == -1, bad
    assert call(bytes_=size - 1) == -4
    assert call(ip=FAKE, n=0) == 0 and call(ip=FAKE, n=2, m=0) == 0


def test_block8_workspace_grows_with_the_batch(kv4):
    rng = np.random.default_rng(1)
    for hq, hkv in ((32, 8), (8, 2), (4, 4), (16, 2), (9, 3)):
        cfg = kv4.make_config(hq, hkv, 0, 0)
        for _ in range(300):
            big = [int(2 ** x) for x in rng.uniform(0, [11, 13, 13, 15])]
            small = [int(rng.integers(0, x + 1)) for x in big]
            assert kv4.block8_workspace_size(cfg, *small) <= kv4.block8_workspace_size(cfg, *big), (small, big)
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1)):
        with pytest.raises(kv4.KV4Error):
            kv4.block8_workspace_size(cfg, *bad)
    assert kv4.block8_workspace_size(cfg, 1024, 1024, 1, 1 << 20) < 64 << 20


def test_weights_refusals(kv4):
    cfg, _, pool, side, batch = structs(kv4)
    r = ctypes.byref

    def call(c=cfg, p=pool, q=FAKE, lse=FAKE, out=FAKE, stride=64):
        return kv4._lib.kv4_attention_weights(r(c), r(p) if p else None, r(side), r(batch), q, lse, None, out,
                                              stride, None, None)

    for bad in (dict(p=None), dict(q=None), dict(lse=None), dict(out=None), dict(q=FAKE + 8), dict(stride=-1)):
        assert call(**bad) == -1, bad
    assert call(c=kv4.make_config(8, 2, 100, 45)) == -3


def test_select_refusals(kv4):
    cfg, _, _, _, batch = structs(kv4)
    r = ctypes.byref

    def call(c=cfg, b=batch, acc=FAKE, stride=64, budget=40, keep=FAKE, new=FAKE):
        return kv4._lib.kv4_evict_select(r(c), r(b) if b else None, acc, stride, budget, keep, new, None, None)

    for bad in (dict(b=None), dict(acc=None), dict(stride=-1), dict(budget=35), dict(budget=0), dict(keep=None),
                dict(new=None)):
        assert call(**bad) == -1, bad
    none = kv4.make_config(8, 2, 0, 0)
    assert call(c=none, budget=0) == -1


def test_compact_refusals(kv4):
    cfg, _, pool, side, batch = structs(kv4)
    r = ctypes.byref
    other = FAKE + 0x1000

    def call(keep=FAKE, budget=40, new=other, to=None, pages=0, a=None, sa=0, z=None, sz=0):
        return kv4._lib.kv4_evict_compact(r(cfg), r(pool), r(side), r(batch), keep, budget, new, to, pages, None,
                                          a, sa, z, sz, None, None)

    for bad in (dict(keep=None), dict(budget=0), dict(new=None), dict(new=FAKE), dict(to=FAKE, pages=0),
                dict(a=FAKE), dict(z=FAKE), dict(a=FAKE, z=FAKE, sa=5, sz=6), dict(a=FAKE, z=other, sa=-1, sz=6),
                dict(a=FAKE, z=FAKE, sa=5, sz=5, to=other, pages=3)):
        assert call(**bad) == -1, bad


def test_binding_refuses_wrong_types_and_shapes(kv4):
    """Types and shapes are refused by the binding before it takes a pointer; so are tensors
    that are not on a GPU."""
    import torch
    t = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    for dtype, shape in ((torch.float32, (2, 2, 128)), (torch.bfloat16, (2, 3, 128)), (torch.bfloat16, (2, 2)),
                         (torch.bfloat16, (2, 2, None))):  # (the last: host memory)
        with pytest.raises(ValueError):
            kv4._addr(t, "x", dtype, shape)
    with pytest.raises(ValueError):
        kv4._addr(None, "x", torch.bfloat16, (2, 2, 128))
    assert kv4._addr_or_null(None, "x", torch.bfloat16, (2, 2, 128)) is None
    with pytest.raises(ValueError):
        kv4.allocate_block8_cache(5, kv4.make_config(8, 2, 0, 0), 4, device="cpu")
    with pytest.raises(ValueError):
        kv4.allocate_block8_cache(kv4.BLOCK8_INT8, kv4.make_config(8, 2, 0, 0), 4, device="cpu")


def test_block8_workspace_at_the_largest_lengths(kv4):
    """Rounding a length up to pages must not run over: the size never falls."""
    cfg = kv4.make_config(32, 8, 0, 0)
    top = 2 ** 31 - 1
    for n, q, m in ((1, 1, 1), (4, 16, 4), (4, 400, 100)):
        sizes = [kv4.block8_workspace_size(cfg, n, q, m, L) for L in (0, 1, 1000, 2 ** 30, top - 15, top - 1, top)]
        assert sizes == sorted(sizes) and sizes[-1] == sizes[-4]


def test_binding_refuses_several_devices(kv4):
    """Every tensor of a call, the error word among them, has to be on one device."""
    import torch

    class On(torch.Tensor):  # a tensor that says it is on a GPU
        is_cuda = True
        gpu = 0

        def get_device(self):
            return self.gpu

    def on(gpu, *shape, dtype=torch.int32):
        t = torch.zeros(shape, dtype=dtype).as_subclass(On)
        t.gpu = gpu
        return t

    called = []
    with pytest.raises(ValueError, match="different devices"):
        kv4._launch(lambda *a: called.append(a), (), on(1, 1), None, on(0, 4))
    with pytest.raises(ValueError, match="different devices"):
        kv4._launch(lambda *a: called.append(a), (), None, None, on(0, 4), None, on(2, 4))
    cfg = kv4.make_config(8, 2, 0, 0)
    codes = [on(g, 3, 2, 8, 16, 16, dtype=torch.int8) for g in (0, 1)]
    scales = [on(0, 3, 2, dtype=torch.float16) for _ in range(2)]
    with pytest.raises(ValueError, match="several devices"):
        kv4.Block8Cache(kv4.BLOCK8_INT8, cfg, *codes, *scales)
    assert not called


class _On:
    """Tensors that say they are on a GPU."""

    def __init__(self):
        import torch

        class On(torch.Tensor):
            is_cuda = True
            gpu = 0

            def get_device(self):
                return self.gpu

        self.cls, self.torch = On, torch

    def __call__(self, shape, dtype, gpu=0):
        return self.of(self.torch.zeros(shape, dtype=dtype), gpu)

    def of(self, t, gpu=0):
        t = t.as_subclass(self.cls)
        t.gpu = gpu
        return t


def _kv4_cache(kv4, on, S=4, R=40, pages=5, H=2, sets=3):
    import torch
    cpu = kv4.allocate_cache(kv4.make_config(8, H, S, R), pages, sets, sets, device="cpu")
    names = [n for n in vars(cpu) if isinstance(getattr(cpu, n), torch.Tensor)]
    assert len(names) == 12
    for n in names:
        setattr(cpu, n, on.of(getattr(cpu, n)))
    return cpu, names


def test_eviction_checks_every_tensor_of_the_cache(kv4):
    """Another type, shape, order or device of any of the twelve tensors, and of the batch's own, is
    refused before a pointer is taken; a tensor set anew is looked at again."""
    import torch
    on = _On()
    lens, ids = on((3,), torch.int32), on((3,), torch.int32)
    q, lse = on((3, 8, 128), torch.bfloat16), on((3, 8), torch.float32)
    acc, keep, new = on((3, 2, 60), torch.float32), on((3, 2, 44), torch.int32), on((3,), torch.int32)
    launched = []

    def refused(cache, batch, match=None):
        with pytest.MonkeyPatch.context() as mp:
            mp.setattr(kv4, "_launch", lambda *a: launched.append(a) or 0)
            for call in (lambda: kv4.attention_weights(cache, batch, q, lse, acc),
                         lambda: kv4.evict_compact(cache, batch, keep, new)):
                with pytest.raises(ValueError, match=match):
                    call()
        assert not launched

    def taken(cache, batch):
        with pytest.MonkeyPatch.context() as mp:
            mp.setattr(kv4, "_launch", lambda *a: launched.append(a) or 0)
            kv4.attention_weights(cache, batch, q, lse, acc)
            kv4.evict_compact(cache, batch, keep, new)
        assert len(launched) == 2
        launched.clear()

    batch = kv4.BatchTensors(on((3, 4), torch.int32), lens, ids, ids, 60)
    cache, names = _kv4_cache(kv4, on)
    taken(cache, batch)
    for name in names:
        good = getattr(cache, name)
        wide = torch.zeros(good.shape[:-1] + (2 * good.shape[-1],), dtype=good.dtype)
        for bad in (on(good.shape, good.dtype, gpu=1), on(good.shape, torch.int64), on.of(wide[..., ::2]),
                    on(good.shape[:-1], good.dtype), on(good.shape[:1] + (3,) + good.shape[2:], good.dtype),
                    torch.zeros(good.shape, dtype=good.dtype)):
            setattr(cache, name, bad)
            refused(cache, batch)
        setattr(cache, name, good)
        taken(cache, batch)
    # a store that the configuration does not use may be anything
    plain, _ = _kv4_cache(kv4, on, S=0, R=0)
    plain.sink_k = plain.ring_vs = on((1,), torch.int64)
    taken(plain, kv4.BatchTensors(on((3, 4), torch.int32), lens, on((3,), torch.int64), None, 60))
    table = torch.zeros((3, 8), dtype=torch.int32)
    for field, bad in (("page_table", on.of(table[:, :4])), ("page_table", on((3, 4), torch.int64)),
                       ("page_table", on((3, 4), torch.int32, gpu=1)), ("page_table", on((2, 4), torch.int32)),
                       ("page_table", None), ("seq_lens", on((3,), torch.int64)),
                       ("seq_lens", on.of(torch.zeros(1, dtype=torch.int32).expand(3))),
                       ("ring_idx", on((3,), torch.int64)), ("ring_idx", on((2,), torch.int32)),
                       ("ring_idx", on((3,), torch.int32, gpu=1))):
        broken = kv4.BatchTensors(on((3, 4), torch.int32), lens, ids, ids, 60)
        broken.check(rings=True, sinks=True)
        setattr(broken, field, bad)
        refused(cache, broken)
    # rows that the batch does not have are not read
    taken(cache, kv4.BatchTensors(on((9, 4), torch.int32), lens, on((7,), torch.int32), None, 60))


def test_block8_and_select_check_the_batch(kv4):
    import torch
    on = _On()
    cfg = kv4.make_config(8, 2, 0, 0)
    codes = [on((5, 2, 8, 16, 16), torch.int8) for _ in range(2)]
    scales = [on((5, 2), torch.float16) for _ in range(2)]
    cache = kv4.Block8Cache(kv4.BLOCK8_INT8, cfg, *codes, *scales)
    k, q, out = on((3, 2, 128), torch.bfloat16), on((3, 8, 128), torch.bfloat16), on((3, 8, 128), torch.bfloat16)
    ws, acc = on((100,), torch.uint8), on((3, 2, 60), torch.float32)
    keep, new = on((3, 2, 9), torch.int32), on((3,), torch.int32)
    table, lens = on((3, 4), torch.int32), on((3,), torch.int32)
    sliced = on.of(torch.zeros((3, 8), dtype=torch.int32)[:, :4])
    launched = []
    with pytest.MonkeyPatch.context() as mp:
        mp.setattr(kv4, "_launch", lambda *a: launched.append(a) or 0)
        for t, n in ((sliced, lens), (on((3, 4), torch.int64), lens), (table, on((3,), torch.int64)),
                     (table, on.of(torch.zeros(6, dtype=torch.int32)[::2]))):
            b = kv4.BatchTensors(t, n, None, None, 60)
            with pytest.raises(ValueError):
                kv4.block8_append(cache, b, k, k)
            with pytest.raises(ValueError):
                kv4.block8_attention(cache, b, q, out, ws)
            if n is not lens:
                with pytest.raises(ValueError):
                    kv4.evict_select(cfg, b, acc, keep, new)
        assert not launched
        b = kv4.BatchTensors(table, lens, None, None, 60)
        kv4.block8_append(cache, b, k, k)
        kv4.block8_attention(cache, b, q, out, ws)
        kv4.evict_select(cfg, kv4.BatchTensors(sliced, lens, None, None, 60), acc, keep, new)
        assert len(launched) == 3


def test_checked_objects_are_copied(kv4):
    """What has been checked is no part of a copy or a comparison."""
    import copy

    import torch
    on = _On()
    b = kv4.BatchTensors(on((3, 4), torch.int32), on((3,), torch.int32), None, None, 60)
    b.check()
    import dataclasses
    c = dataclasses.replace(b, seq_lens=on((3,), torch.int64))
    with pytest.raises(ValueError):
        c.check()
    d = copy.copy(b)
    d.seq_lens = on((3,), torch.int64)
    with pytest.raises(ValueError):
        d.check()
    b.check()


def test_select_refuses_the_lengths_as_its_output(kv4):
    """A unit of the grid would read the lengths that another has already written."""
    cfg, _, _, _, batch = structs(kv4)
    r = ctypes.byref

    def call(new, B=2):
        batch.num_seqs = B
        return kv4._lib.kv4_evict_select(r(cfg), r(batch), FAKE, 64, 40, FAKE, new, None, None)

    assert call(batch.seq_lens) == -1
    assert call(batch.seq_lens, B=0) == 0  # nothing to do


def test_compact_refuses_the_batchs_own_pages_as_others(kv4):
    """Rows that go to other pages move in any order: the batch's own table is not another."""
    cfg, _, pool, side, batch = structs(kv4)
    r = ctypes.byref
    assert kv4._lib.kv4_evict_compact(r(cfg), r(pool), r(side), r(batch), FAKE, 40, FAKE + 0x1000, batch.page_table,
                                      4, None, None, 0, None, 0, None, None) == -1
