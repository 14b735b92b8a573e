"""Thin Python binding of libkv4.so (include/kv4.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
allocates device tensors with PyTorch (plumbing), fills the C structs with raw
pointers and forwards the caller's CUDA stream. There is no fallback: if the library
cannot be loaded, importing this module raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkv4.so")

KV4_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape",
          -3: "protected set larger than 144 positions", -4: "workspace too small",
          -5: "CUDA error"}
DEVERR = {1: "page id", 2: "seq len", 4: "side index", 8: "q range", 16: "workspace",
          32: "timeout", 64: "keep index"}
MAX_PROTECTED = 144
HEAD_DIM = 128
PAGE = 16
GROUP = 32

EXPORTS = ("kv4_workspace_size", "kv4_chunk_pages_for", "kv4_quantize_append",
           "kv4_decode_attention", "kv4_decode_step", "kv4_regional_merge",
           "kv4_status_string", "kv4_version",
           "kv4_decode_attention_noalloc", "kv4_noalloc_scratch_bytes",
           "kv4_baseline_append", "kv4_baseline_workspace_size",
           "kv4_baseline_decode_attention", "kv4_test_withhold_copy",
           "kv4_block8_append", "kv4_block8_workspace_size", "kv4_block8_attention",
           "kv4_attention_weights", "kv4_evict_select", "kv4_evict_compact")

BASELINE_BF16 = 1  # kv4_baseline_format
BASELINE_KV8 = 2
BLOCK8_INT8 = 1  # kv4_block8_format
BLOCK8_E4M3 = 2


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("num_sinks", ctypes.c_int32),
                ("num_recent", ctypes.c_int32), ("chunk_pages", ctypes.c_int32),
                ("demotion", ctypes.c_int32), ("prefix_mode", ctypes.c_int32)]


class Int4Pool(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_params", ctypes.c_void_p), ("v_params", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class Int8Side(ctypes.Structure):
    _fields_ = [("sink_k", ctypes.c_void_p), ("sink_v", ctypes.c_void_p),
                ("sink_ks", ctypes.c_void_p), ("sink_vs", ctypes.c_void_p),
                ("num_sink_sets", ctypes.c_int32),
                ("ring_k", ctypes.c_void_p), ("ring_v", ctypes.c_void_p),
                ("ring_ks", ctypes.c_void_p), ("ring_vs", ctypes.c_void_p),
                ("num_rings", ctypes.c_int32)]


class Batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("sink_idx", ctypes.c_void_p),
                ("ring_idx", ctypes.c_void_p), ("num_seqs", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("plan_reuse", ctypes.c_int32)]


class PagedPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libkv4.so not built at {path}: run "
                          "`python -m quantized_kv_cache_kv4_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    lib.kv4_workspace_size.restype = ctypes.c_size_t
    lib.kv4_workspace_size.argtypes = [ctypes.POINTER(Config), ctypes.c_int32, ctypes.c_int32]
    lib.kv4_chunk_pages_for.restype = ctypes.c_int32
    lib.kv4_chunk_pages_for.argtypes = [ctypes.POINTER(Config), ctypes.c_int32, ctypes.c_int32]
    lib.kv4_quantize_append.restype = ctypes.c_int
    lib.kv4_quantize_append.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Int4Pool),
                                        ctypes.POINTER(Int8Side), ctypes.POINTER(Batch),
                                        P, P, P, ctypes.c_int32, P, P]
    lib.kv4_decode_attention.restype = ctypes.c_int
    lib.kv4_decode_attention.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Int4Pool),
                                         ctypes.POINTER(Int8Side), ctypes.POINTER(Batch),
                                         P, P, P, P, P, ctypes.c_size_t, P, P]
    lib.kv4_decode_step.restype = ctypes.c_int
    lib.kv4_decode_step.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Int4Pool),
                                    ctypes.POINTER(Int8Side), ctypes.POINTER(Batch),
                                    P, P, P, P, P, P, P, ctypes.c_size_t, P, P]
    lib.kv4_regional_merge.restype = ctypes.c_int
    lib.kv4_regional_merge.argtypes = [P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       P, P, P, P]
    lib.kv4_decode_attention_noalloc.restype = ctypes.c_int
    lib.kv4_decode_attention_noalloc.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Int4Pool),
                                                 ctypes.POINTER(Int8Side), ctypes.POINTER(Batch),
                                                 P, P, P, P, P, P]
    lib.kv4_noalloc_scratch_bytes.restype = ctypes.c_size_t
    lib.kv4_noalloc_scratch_bytes.argtypes = []
    lib.kv4_baseline_append.restype = ctypes.c_int
    lib.kv4_baseline_append.argtypes = [ctypes.c_int, ctypes.POINTER(Config),
                                        ctypes.POINTER(PagedPool), ctypes.POINTER(Batch),
                                        P, P, P, ctypes.c_int32, P, P]
    lib.kv4_baseline_workspace_size.restype = ctypes.c_size_t
    lib.kv4_baseline_workspace_size.argtypes = [ctypes.POINTER(Config), ctypes.c_int32,
                                                ctypes.c_int32]
    lib.kv4_baseline_decode_attention.restype = ctypes.c_int
    lib.kv4_baseline_decode_attention.argtypes = [ctypes.c_int, ctypes.POINTER(Config),
                                                  ctypes.POINTER(PagedPool),
                                                  ctypes.POINTER(Batch), P, P, P, P, P,
                                                  ctypes.c_size_t, P, P]
    I = ctypes.c_int32
    lib.kv4_block8_append.restype = ctypes.c_int
    lib.kv4_block8_append.argtypes = [I, ctypes.POINTER(Config), ctypes.POINTER(PagedPool),
                                      ctypes.POINTER(Batch), P, P, P, I, P, P]
    lib.kv4_block8_workspace_size.restype = ctypes.c_size_t
    lib.kv4_block8_workspace_size.argtypes = [ctypes.POINTER(Config), I, I, I, I]
    lib.kv4_block8_attention.restype = ctypes.c_int
    lib.kv4_block8_attention.argtypes = [I, ctypes.POINTER(Config), ctypes.POINTER(PagedPool),
                                         ctypes.POINTER(Batch), P, P, I, I, P, P, P, P,
                                         ctypes.c_size_t, P, P]
    cache4 = [ctypes.POINTER(Config), ctypes.POINTER(Int4Pool), ctypes.POINTER(Int8Side),
              ctypes.POINTER(Batch)]
    lib.kv4_attention_weights.restype = ctypes.c_int
    lib.kv4_attention_weights.argtypes = cache4 + [P, P, P, P, I, P, P]
    lib.kv4_evict_select.restype = ctypes.c_int
    lib.kv4_evict_select.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Batch), P, I, I, P, P,
                                     P, P]
    lib.kv4_evict_compact.restype = ctypes.c_int
    lib.kv4_evict_compact.argtypes = cache4 + [P, I, P, P, I, P, P, I, P, I, P, P]
    lib.kv4_test_withhold_copy.restype = None
    lib.kv4_test_withhold_copy.argtypes = [ctypes.c_int32, ctypes.c_uint32]
    lib.kv4_status_string.restype = ctypes.c_char_p
    lib.kv4_status_string.argtypes = [ctypes.c_int]
    lib.kv4_version.restype = ctypes.c_int32
    lib.kv4_version.argtypes = []
    return lib


_lib = load_library()


class KV4Error(RuntimeError):
    pass


def _check(status: int, what: str):
    if status != KV4_OK:
        raise KV4Error(f"{what}: {_lib.kv4_status_string(status).decode()} ({status})")


def _ptr(t):
    """Device pointer of a tensor argument (None -> NULL). The library reads every array
    densely from its first element, so a tensor must be a contiguous CUDA tensor."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("kv4 arguments must be contiguous CUDA tensors "
                         f"(got device={t.device}, contiguous={t.is_contiguous()})")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


DEMOTION = {"A": 0, "B": 1}  # kv4_config.demotion
PREFIX = {"off": 0, "shared": 1}  # kv4_config.prefix_mode


def make_config(num_q_heads, num_kv_heads, num_sinks, num_recent, chunk_pages=0,
                demotion="A", prefix="off") -> Config:
    return Config(num_q_heads, num_kv_heads, HEAD_DIM, PAGE, GROUP, num_sinks, num_recent,
                  chunk_pages, DEMOTION[demotion], PREFIX[prefix])


def _dense(t, what, itemsize, shape, dev):
    """Raises unless t is a contiguous CUDA tensor on device `dev` (None: any), of elements of
    `itemsize` bytes (a dtype: of that type), of this shape (None in it: any size)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: a tensor is wanted, not {type(t).__name__}")
    if t.dtype is not itemsize if isinstance(itemsize, torch.dtype) else t.element_size() != itemsize:
        raise ValueError(f"{what}: elements of {itemsize} are wanted, not {t.dtype}"
                         if isinstance(itemsize, torch.dtype) else
                         f"{what}: elements of {itemsize} bytes are wanted, not {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{what}: shape {tuple(shape)} is wanted, not {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA tensor is wanted "
                         f"(got device={t.device}, contiguous={t.is_contiguous()})")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{what}: kv4 arguments on different devices ({t.get_device()}, not {dev})")


class _Checked:
    """Remembers what of an object has been checked, until one of its attributes is set anew."""

    _seen = None

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_seen":
            object.__setattr__(self, "_seen", None)


@dataclasses.dataclass
class Cache(_Checked):
    """Device storage of one layer's cache, in the library's format (see kv4.h)."""

    cfg: Config
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_params: torch.Tensor
    v_params: torch.Tensor
    sink_k: torch.Tensor
    sink_v: torch.Tensor
    sink_ks: torch.Tensor
    sink_vs: torch.Tensor
    ring_k: torch.Tensor
    ring_v: torch.Tensor
    ring_ks: torch.Tensor
    ring_vs: torch.Tensor

    @property
    def num_pages(self):
        return self.k_codes.shape[0]

    def check(self):
        """Raises unless all its tensors have the format's shapes and element sizes, dense on one
        device (a side store that the configuration does not use may be anything)."""
        H, S, R = self.cfg.num_kv_heads, self.cfg.num_sinks, self.cfg.num_recent
        if self._seen == (H, S, R):
            return
        _dense(self.k_codes, "k_codes", 1, (None, H, 4, PAGE, 16), None)
        pages, dev = self.k_codes.shape[0], self.k_codes.get_device()
        _dense(self.v_codes, "v_codes", 1, (pages, H, 4, PAGE, 16), dev)
        _dense(self.k_params, "k_params", 2, (pages, H, PAGE, 4, 2), dev)
        _dense(self.v_params, "v_params", 2, (pages, H, PAGE, 4, 2), dev)
        for name, slots in (("sink", S), ("ring", R)):
            if slots == 0:
                continue
            tiles, sets = (slots + PAGE - 1) // PAGE, getattr(self, name + "_k").shape[0]
            for x in ("_k", "_v"):
                _dense(getattr(self, name + x), name + x, 1, (sets, H, tiles, 8, PAGE, 16), dev)
                _dense(getattr(self, name + x + "s"), name + x + "s", 2, (sets, H, tiles * PAGE), dev)
        self._seen = (H, S, R)

    def pool_struct(self) -> Int4Pool:
        return Int4Pool(self.k_codes.data_ptr(), self.v_codes.data_ptr(),
                        self.k_params.data_ptr(), self.v_params.data_ptr(), self.num_pages)

    def side_struct(self) -> Int8Side:
        return Int8Side(self.sink_k.data_ptr(), self.sink_v.data_ptr(),
                        self.sink_ks.data_ptr(), self.sink_vs.data_ptr(), self.sink_k.shape[0],
                        self.ring_k.data_ptr(), self.ring_v.data_ptr(),
                        self.ring_ks.data_ptr(), self.ring_vs.data_ptr(), self.ring_k.shape[0])


def allocate_cache(cfg: Config, num_pages: int, num_sink_sets: int, num_rings: int,
                   device="cuda") -> Cache:
    """Zero-initialised cache tensors (int8/uint8 codes, fp16 bits as int16)."""
    H = cfg.num_kv_heads
    st = max(1, (cfg.num_sinks + PAGE - 1) // PAGE)
    rt = max(1, (cfg.num_recent + PAGE - 1) // PAGE)
    z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
    return Cache(
        cfg=cfg,
        k_codes=z((num_pages, H, 4, PAGE, 16), torch.uint8),
        v_codes=z((num_pages, H, 4, PAGE, 16), torch.uint8),
        k_params=z((num_pages, H, PAGE, 4, 2), torch.int16),
        v_params=z((num_pages, H, PAGE, 4, 2), torch.int16),
        sink_k=z((max(1, num_sink_sets), H, st, 8, PAGE, 16), torch.int8),
        sink_v=z((max(1, num_sink_sets), H, st, 8, PAGE, 16), torch.int8),
        sink_ks=z((max(1, num_sink_sets), H, st * PAGE), torch.int16),
        sink_vs=z((max(1, num_sink_sets), H, st * PAGE), torch.int16),
        ring_k=z((max(1, num_rings), H, rt, 8, PAGE, 16), torch.int8),
        ring_v=z((max(1, num_rings), H, rt, 8, PAGE, 16), torch.int8),
        ring_ks=z((max(1, num_rings), H, rt * PAGE), torch.int16),
        ring_vs=z((max(1, num_rings), H, rt * PAGE), torch.int16))


@dataclasses.dataclass
class BatchTensors(_Checked):
    page_table: torch.Tensor  # int32 [B, max_pages]
    seq_lens: torch.Tensor    # int32 [B]
    sink_idx: torch.Tensor | None  # int32 [B]; None where there are no sinks
    ring_idx: torch.Tensor | None
    max_seq_len: int
    plan_reuse: bool = False  # use the work list the last call on the workspace left

    def check(self, table=True, sinks=False, rings=False):
        """Raises unless the lengths, and what else the call reads, are dense int32 tensors on one
        device with an entry for each sequence."""
        want = 1 | 2 * table | 4 * sinks | 8 * rings
        seen = self._seen or 0
        if seen & want == want:
            return
        _dense(self.seq_lens, "seq_lens", torch.int32, (None,), None)
        B, dev = self.seq_lens.shape[0], self.seq_lens.get_device()
        for wanted, name, dims in ((table, "page_table", 2), (sinks, "sink_idx", 1), (rings, "ring_idx", 1)):
            t = getattr(self, name)
            if wanted and (t is not None or name == "page_table"):
                _dense(t, name, torch.int32, (None,) * dims, dev)
                if t.shape[0] < B:
                    raise ValueError(f"{name}: {t.shape[0]} entries for {B} sequences")
        self._seen = seen | want

    def struct(self) -> Batch:
        return Batch(self.page_table.data_ptr(), self.page_table.shape[1],
                     self.seq_lens.data_ptr(),
                     0 if self.sink_idx is None else self.sink_idx.data_ptr(),
                     0 if self.ring_idx is None else self.ring_idx.data_ptr(),
                     self.seq_lens.shape[0], int(self.max_seq_len), int(self.plan_reuse))


def workspace_size(cfg: Config, num_seqs: int, max_seq_len: int) -> int:
    n = _lib.kv4_workspace_size(ctypes.byref(cfg), num_seqs, max_seq_len)
    if n == 0 and num_seqs > 0:
        raise KV4Error("kv4_workspace_size: invalid arguments")
    return n


def chunk_pages_for(cfg: Config, num_seqs: int, max_seq_len: int) -> int:
    """The INT4 chunk length (pages) the library uses for such a batch."""
    n = _lib.kv4_chunk_pages_for(ctypes.byref(cfg), num_seqs, max_seq_len)
    if n < 0:
        raise KV4Error("kv4_chunk_pages_for: invalid arguments")
    return n


def quantize_append(cache: Cache, batch: BatchTensors, k_new: torch.Tensor, v_new: torch.Tensor,
                    new_indptr: torch.Tensor | None = None, err: torch.Tensor | None = None,
                    stream=None):
    """k_new, v_new: bf16 [rows, Hkv, 128]; new_indptr int32 [B+1] or None (one row per seq)."""
    pool, side, bs = cache.pool_struct(), cache.side_struct(), batch.struct()
    st = _lib.kv4_quantize_append(ctypes.byref(cache.cfg), ctypes.byref(pool), ctypes.byref(side),
                                  ctypes.byref(bs), _ptr(k_new), _ptr(v_new), _ptr(new_indptr),
                                  int(k_new.shape[0]), _ptr(err), _stream(stream))
    _check(st, "kv4_quantize_append")


def decode_attention(cache: Cache, batch: BatchTensors, q: torch.Tensor, out: torch.Tensor,
                     workspace: torch.Tensor, out_f32: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, err: torch.Tensor | None = None,
                     stream=None):
    """q, out: bf16 [B, Hq, 128]; workspace: uint8 device tensor (256-byte aligned)."""
    pool, side, bs = cache.pool_struct(), cache.side_struct(), batch.struct()
    st = _lib.kv4_decode_attention(ctypes.byref(cache.cfg), ctypes.byref(pool),
                                   ctypes.byref(side), ctypes.byref(bs), _ptr(q), _ptr(out),
                                   _ptr(out_f32), _ptr(lse), _ptr(workspace),
                                   workspace.numel(), _ptr(err), _stream(stream))
    _check(st, "kv4_decode_attention")


def decode_step(cache: Cache, batch: BatchTensors, k_new: torch.Tensor, v_new: torch.Tensor,
                q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                out_f32: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                err: torch.Tensor | None = None, stream=None):
    """One decode step: quantize_append of one token per sequence (k_new, v_new bf16
    [B, Hkv, 128]) then decode_attention, in one library call (one launch builds the
    attention's work list and appends the tokens). batch.lens: lengths after the
    append."""
    pool, side, bs = cache.pool_struct(), cache.side_struct(), batch.struct()
    st = _lib.kv4_decode_step(ctypes.byref(cache.cfg), ctypes.byref(pool), ctypes.byref(side),
                              ctypes.byref(bs), _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(out),
                              _ptr(out_f32), _ptr(lse), _ptr(workspace), workspace.numel(),
                              _ptr(err), _stream(stream))
    _check(st, "kv4_decode_step")


def decode_attention_noalloc(cache: Cache, batch: BatchTensors, q: torch.Tensor,
                             out: torch.Tensor, out_f32: torch.Tensor | None = None,
                             lse: torch.Tensor | None = None, err: torch.Tensor | None = None,
                             stream=None):
    """decode_attention without a workspace argument, for callers that cannot allocate
    device memory: the library's fixed scratch array (kv4_noalloc_scratch_bytes()) is
    used instead. Calls that overlap on the GPU race on that array."""
    pool, side, bs = cache.pool_struct(), cache.side_struct(), batch.struct()
    st = _lib.kv4_decode_attention_noalloc(ctypes.byref(cache.cfg), ctypes.byref(pool),
                                           ctypes.byref(side), ctypes.byref(bs), _ptr(q),
                                           _ptr(out), _ptr(out_f32), _ptr(lse), _ptr(err),
                                           _stream(stream))
    _check(st, "kv4_decode_attention_noalloc")


def noalloc_scratch_bytes() -> int:
    return int(_lib.kv4_noalloc_scratch_bytes())


def regional_merge(partials: torch.Tensor, region_offsets: torch.Tensor, group: int,
                   out: torch.Tensor, out_f32: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, stream=None):
    """partials fp32 [regions, group, 132]; region_offsets int32 [units+1]."""
    n_units = region_offsets.shape[0] - 1
    st = _lib.kv4_regional_merge(_ptr(partials), _ptr(region_offsets), n_units, group, HEAD_DIM,
                                 _ptr(out), _ptr(out_f32), _ptr(lse), _stream(stream))
    _check(st, "kv4_regional_merge")


def decode_err(flag: int) -> list[str]:
    return [name for bit, name in DEVERR.items() if flag & bit]


# ----------------------------------------------------------------------------
# comparison baselines (BF16 and all-INT8 paged caches)
# ----------------------------------------------------------------------------

@dataclasses.dataclass
class BaselineCache:
    """Device storage of one layer's BF16 or KV8 paged cache (layouts in kv4.h)."""

    fmt: int
    cfg: Config
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor | None
    v_scales: torch.Tensor | None

    @property
    def num_pages(self):
        return self.k.shape[0]

    def pool_struct(self) -> PagedPool:
        ks = 0 if self.k_scales is None else self.k_scales.data_ptr()
        vs = 0 if self.v_scales is None else self.v_scales.data_ptr()
        return PagedPool(self.k.data_ptr(), self.v.data_ptr(), ks, vs, self.num_pages)


def allocate_baseline_cache(fmt: int, cfg: Config, num_pages: int, device="cuda") -> BaselineCache:
    """Zero-initialised BF16 ([pages, Hkv, 16 octets, 16 slots, 8]) or KV8 ([pages, Hkv,
    8 strips, 16 slots, 16] int8 + fp16 scales [pages, Hkv, 16]) page pool."""
    H = cfg.num_kv_heads
    z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
    if fmt == BASELINE_BF16:
        return BaselineCache(fmt, cfg, z((num_pages, H, 16, PAGE, 8), torch.bfloat16),
                             z((num_pages, H, 16, PAGE, 8), torch.bfloat16), None, None)
    if fmt == BASELINE_KV8:
        return BaselineCache(fmt, cfg, z((num_pages, H, 8, PAGE, 16), torch.int8),
                             z((num_pages, H, 8, PAGE, 16), torch.int8),
                             z((num_pages, H, PAGE), torch.int16),
                             z((num_pages, H, PAGE), torch.int16))
    raise ValueError(f"unknown baseline format {fmt}")


def baseline_workspace_size(cfg: Config, num_seqs: int, max_seq_len: int) -> int:
    n = _lib.kv4_baseline_workspace_size(ctypes.byref(cfg), num_seqs, max_seq_len)
    if n == 0 and num_seqs > 0:
        raise KV4Error("kv4_baseline_workspace_size: invalid arguments")
    return n


def baseline_append(cache: BaselineCache, batch: BatchTensors, k_new: torch.Tensor,
                    v_new: torch.Tensor, new_indptr: torch.Tensor | None = None,
                    err: torch.Tensor | None = None, stream=None):
    pool, bs = cache.pool_struct(), batch.struct()
    st = _lib.kv4_baseline_append(cache.fmt, ctypes.byref(cache.cfg), ctypes.byref(pool),
                                  ctypes.byref(bs), _ptr(k_new), _ptr(v_new), _ptr(new_indptr),
                                  int(k_new.shape[0]), _ptr(err), _stream(stream))
    _check(st, "kv4_baseline_append")


def baseline_decode_attention(cache: BaselineCache, batch: BatchTensors, q: torch.Tensor,
                              out: torch.Tensor, workspace: torch.Tensor,
                              out_f32: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                              err: torch.Tensor | None = None, stream=None):
    pool, bs = cache.pool_struct(), batch.struct()
    st = _lib.kv4_baseline_decode_attention(cache.fmt, ctypes.byref(cache.cfg),
                                            ctypes.byref(pool), ctypes.byref(bs), _ptr(q),
                                            _ptr(out), _ptr(out_f32), _ptr(lse), _ptr(workspace),
                                            workspace.numel(), _ptr(err), _stream(stream))
    _check(st, "kv4_baseline_decode_attention")


# ----------------------------------------------------------------------------
# 8-bit block-scaled cache
# ----------------------------------------------------------------------------

def _addr(t, what, dtype, shape):
    """Address of a contiguous CUDA tensor of this type and shape (None in a shape: any size)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: a tensor is wanted, not {type(t).__name__}")
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} is wanted, not {t.dtype}")
    if t.shape != shape and (t.dim() != len(shape) or any(
            n is not None and n != m for n, m in zip(shape, t.shape))):
        raise ValueError(f"{what}: shape {tuple(shape)} is wanted, not {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous CUDA tensor is wanted "
                         f"(got device={t.device}, contiguous={t.is_contiguous()})")
    return t.data_ptr()


def _addr_or_null(t, what, dtype, shape):
    return None if t is None else _addr(t, what, dtype, shape)


def _launch(fn, args, err, stream, *tensors):
    """fn(*args, err, stream) with the tensors' device current: a launch goes to the current
    device, whichever the caller left current."""
    dev = tensors[0].get_device()
    e = _addr_or_null(err, "err", torch.int32, (1,))
    for t in tensors + (err,):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"kv4 arguments on different devices: {tensors[0].device} and {t.device}")
    if dev == torch.cuda.current_device():
        return fn(*args, e, torch.cuda.current_stream(dev).cuda_stream if stream is None
                  else stream.cuda_stream)
    with torch.cuda.device(dev):
        return fn(*args, e, torch.cuda.current_stream(dev).cuda_stream if stream is None
                  else stream.cuda_stream)


@dataclasses.dataclass(frozen=True)
class Block8Cache:
    """Device storage of one layer's 8-bit block-scaled cache (layout in kv4.h): codes
    [pages, Hkv, 8 strips, 16 slots, 16] as int8 (BLOCK8_INT8) or float8_e4m3fn
    (BLOCK8_E4M3), scales float16 [pages, Hkv]. Its tensors are checked once, here."""

    fmt: int
    cfg: Config
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    pool: PagedPool = dataclasses.field(init=False, repr=False, compare=False)

    def __post_init__(self):
        if self.fmt not in _BLOCK8_DTYPES:
            raise ValueError(f"unknown block8 format {self.fmt}")
        code, pages, H = _BLOCK8_DTYPES[self.fmt], self.k.shape[0], self.cfg.num_kv_heads
        codes, scales = (pages, H, 8, PAGE, 16), (pages, H)
        object.__setattr__(self, "pool", PagedPool(
            _addr(self.k, "k", code, codes), _addr(self.v, "v", code, codes),
            _addr(self.k_scales, "k_scales", torch.float16, scales),
            _addr(self.v_scales, "v_scales", torch.float16, scales), pages))
        if len({t.get_device() for t in (self.k, self.v, self.k_scales, self.v_scales)}) > 1:
            raise ValueError("a block8 cache on several devices")

    @property
    def num_pages(self):
        return self.k.shape[0]

    def pool_struct(self) -> PagedPool:
        return self.pool


_BLOCK8_DTYPES = {BLOCK8_INT8: torch.int8, BLOCK8_E4M3: torch.float8_e4m3fn}


def allocate_block8_cache(fmt: int, cfg: Config, num_pages: int, device="cuda") -> Block8Cache:
    """Zero-initialised block-scaled page pool."""
    if fmt not in _BLOCK8_DTYPES:
        raise ValueError(f"unknown block8 format {fmt}")
    H = cfg.num_kv_heads
    codes = lambda: torch.zeros((num_pages, H, 8, PAGE, 16), dtype=torch.int8,
                                device=device).view(_BLOCK8_DTYPES[fmt])
    scales = lambda: torch.zeros((num_pages, H), dtype=torch.float16, device=device)
    return Block8Cache(fmt, cfg, codes(), codes(), scales(), scales())


def block8_append(cache: Block8Cache, batch: BatchTensors, k_new: torch.Tensor,
                  v_new: torch.Tensor, new_indptr: torch.Tensor | None = None,
                  err: torch.Tensor | None = None, stream=None):
    """k_new, v_new: bf16 [rows, Hkv, 128]; new_indptr int32 [B+1] or None (one row per seq)."""
    batch.check()
    n, bs = k_new.shape[0], batch.struct()
    rows = (n, cache.cfg.num_kv_heads, HEAD_DIM)
    args = (cache.fmt, ctypes.byref(cache.cfg), ctypes.byref(cache.pool), ctypes.byref(bs),
            _addr(k_new, "k_new", torch.bfloat16, rows), _addr(v_new, "v_new", torch.bfloat16, rows),
            _addr_or_null(new_indptr, "new_indptr", torch.int32, (bs.num_seqs + 1,)), n)
    _check(_launch(_lib.kv4_block8_append, args, err, stream, cache.k, batch.page_table,
                   batch.seq_lens, k_new, v_new, new_indptr), "kv4_block8_append")


def block8_workspace_size(cfg: Config, num_seqs: int, total_q: int, max_q_len: int,
                          max_seq_len: int) -> int:
    n = _lib.kv4_block8_workspace_size(ctypes.byref(cfg), num_seqs, total_q, max_q_len, max_seq_len)
    if n == 0:
        raise KV4Error("kv4_block8_workspace_size: invalid arguments")
    return n


def block8_attention(cache: Block8Cache, batch: BatchTensors, q: torch.Tensor, out: torch.Tensor,
                     workspace: torch.Tensor, q_indptr: torch.Tensor | None = None,
                     max_q_len: int = 1, out_f32: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, err: torch.Tensor | None = None,
                     stream=None):
    """q, out: bf16 [rows, Hq, 128]; q_indptr int32 [B+1]: sequence b's rows are its last
    positions, at most max_q_len of them, causal (None: one per sequence); out_f32 fp32 like
    out; lse fp32 [rows, Hq]; workspace: uint8, block8_workspace_size(...) bytes."""
    batch.check()
    n, Hq, bs = q.shape[0], cache.cfg.num_q_heads, batch.struct()
    rows = (n, Hq, HEAD_DIM)
    args = (cache.fmt, ctypes.byref(cache.cfg), ctypes.byref(cache.pool), ctypes.byref(bs),
            _addr(q, "q", torch.bfloat16, rows),
            _addr_or_null(q_indptr, "q_indptr", torch.int32, (bs.num_seqs + 1,)), n, max_q_len,
            _addr(out, "out", torch.bfloat16, rows),
            _addr_or_null(out_f32, "out_f32", torch.float32, rows),
            _addr_or_null(lse, "lse", torch.float32, (n, Hq)),
            _addr(workspace, "workspace", torch.uint8, (None,)), workspace.numel())
    _check(_launch(_lib.kv4_block8_attention, args, err, stream, cache.k, batch.page_table,
                   batch.seq_lens, q, out, workspace, q_indptr, out_f32, lse), "kv4_block8_attention")


# ----------------------------------------------------------------------------
# eviction by accumulated attention weight
# ----------------------------------------------------------------------------

def attention_weights(cache: Cache, batch: BatchTensors, q: torch.Tensor, lse: torch.Tensor,
                      acc_out: torch.Tensor, acc_in: torch.Tensor | None = None,
                      err: torch.Tensor | None = None, stream=None):
    """acc_out = acc_in + each position's attention weight in this decode step. q bf16
    [B, Hq, 128]; lse fp32 [B, Hq] as decode_attention wrote it; acc_in, acc_out fp32
    [B, Hkv, positions] (may be the same; None: zeros)."""
    cfg = cache.cfg
    cache.check()
    batch.check(sinks=cfg.num_sinks > 0, rings=cfg.num_recent > 0)
    bs = batch.struct()
    B, stride = bs.num_seqs, acc_out.shape[-1]
    total = (B, cfg.num_kv_heads, stride)
    pool, side = cache.pool_struct(), cache.side_struct()
    args = (ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(side), ctypes.byref(bs),
            _addr(q, "q", torch.bfloat16, (B, cfg.num_q_heads, HEAD_DIM)),
            _addr(lse, "lse", torch.float32, (B, cfg.num_q_heads)),
            _addr_or_null(acc_in, "acc_in", torch.float32, total),
            _addr(acc_out, "acc_out", torch.float32, total), stride)
    _check(_launch(_lib.kv4_attention_weights, args, err, stream, cache.k_codes,
                   batch.page_table, batch.seq_lens, q, lse, acc_out, acc_in), "kv4_attention_weights")


def evict_select(cfg: Config, batch: BatchTensors, acc: torch.Tensor, keep: torch.Tensor,
                 new_lens: torch.Tensor, err: torch.Tensor | None = None, stream=None):
    """The positions to keep: acc fp32 [B, Hkv, positions]; keep int32 [B, Hkv, budget]
    (ascending, -1 behind the last) and new_lens int32 [B] are written."""
    batch.check(table=False)
    bs = batch.struct()
    B, H, stride, budget = bs.num_seqs, cfg.num_kv_heads, acc.shape[-1], keep.shape[-1]
    if B and new_lens.data_ptr() == bs.seq_lens:
        raise ValueError("new_lens must not be the batch's seq_lens")
    args = (ctypes.byref(cfg), ctypes.byref(bs), _addr(acc, "acc", torch.float32, (B, H, stride)), stride,
            budget, _addr(keep, "keep", torch.int32, (B, H, budget)),
            _addr(new_lens, "new_lens", torch.int32, (B,)))
    _check(_launch(_lib.kv4_evict_select, args, err, stream, acc, batch.seq_lens, keep, new_lens),
           "kv4_evict_select")


def evict_compact(cache: Cache, batch: BatchTensors, keep: torch.Tensor, new_lens: torch.Tensor,
                  dst_page_table: torch.Tensor | None = None,
                  dst_ring_idx: torch.Tensor | None = None, acc_in: torch.Tensor | None = None,
                  acc_out: torch.Tensor | None = None, err: torch.Tensor | None = None,
                  stream=None):
    """Moves the kept rows (keep, new_lens as evict_select wrote them) to the front of the pages
    of dst_page_table int32 [B, pages] (None: the sequence's own), the recent window's INT8
    copies to ring dst_ring_idx int32 [B] (None: its own), and the totals to acc_out."""
    cfg = cache.cfg
    cache.check()
    batch.check(rings=cfg.num_recent > 0)
    bs = batch.struct()
    B, H, budget = bs.num_seqs, cfg.num_kv_heads, keep.shape[-1]
    pages = 0 if dst_page_table is None else dst_page_table.shape[-1]
    s_in, s_out = (0 if t is None else t.shape[-1] for t in (acc_in, acc_out))
    pool, side = cache.pool_struct(), cache.side_struct()
    args = (ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(side), ctypes.byref(bs),
            _addr(keep, "keep", torch.int32, (B, H, budget)), budget,
            _addr(new_lens, "new_lens", torch.int32, (B,)),
            _addr_or_null(dst_page_table, "dst_page_table", torch.int32, (B, pages)), pages,
            _addr_or_null(dst_ring_idx, "dst_ring_idx", torch.int32, (B,)),
            _addr_or_null(acc_in, "acc_in", torch.float32, (B, H, s_in)), s_in,
            _addr_or_null(acc_out, "acc_out", torch.float32, (B, H, s_out)), s_out)
    _check(_launch(_lib.kv4_evict_compact, args, err, stream, cache.k_codes, batch.page_table,
                   batch.seq_lens, keep, new_lens, dst_page_table, dst_ring_idx, acc_in, acc_out),
           "kv4_evict_compact")
