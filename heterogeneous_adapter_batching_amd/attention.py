"""The attention between a layer's q/k/v product and its o product over the C
ABI (argument marshalling only): the plan of a batch over a paged cache, rotary
positions with the new keys and values into the pages, attention over them."""
from __future__ import annotations

import ctypes
import functools

import numpy as np

try:
    import torch
except ImportError:                    # batches can be planned without it
    torch = None

from ._lib import (ROTARY_LAYOUTS, ROTARY_SCALINGS, AttnDesc, KvCache, RotaryDesc, check, load)
from .api import _DTYPES, _i32, _torch_dtype
from .layer import _code, _enqueue, _new, _Tensor

_i32p = ctypes.POINTER(ctypes.c_int32)


def _lens(values, name):
    """Lengths as the library's 32-bit integers, each of them checked."""
    a = np.asarray(values)
    if a.ndim != 1 or (a.size and a.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of integers")
    if a.size and (int(a.min()) < -(1 << 31) or int(a.max()) >= 1 << 31):
        raise ValueError(f"{name} does not fit 32 bits")
    return np.ascontiguousarray(a, dtype=np.int32)


class AttentionPlan:
    """The plan of one batch's attention over a paged cache (built on the
    host): new_lens[s] tokens of sequence s, in order, at the end of its
    kv_lens[s] keys.

    heads query heads share kv_heads key heads; a page holds page_size tokens
    (a multiple of 16).  causal: a token sees the keys up to its own, the last
    `window` of them unless that is 0; else all of its sequence's keys (an
    encoder's states; new_lens and kv_lens are then independent).  max_kv: the
    most keys of any later rebuild, so that a captured graph may be replayed
    after rebuild(the same new_lens, other kv_lens).upload(the same ws); the
    page table then has room for max_kv keys.  A rebuild that fails leaves the
    plan as it was.  A workspace that any other plan, an adapter plan too, has
    been uploaded over is refused until this one is uploaded again."""

    def __init__(self, heads, kv_heads, head_dim, page_size, new_lens, kv_lens, *, dtype="bf16",
                 causal=True, window=0, max_kv=0):
        self.lib = load()
        self._h = ctypes.c_void_p()
        self.ws = None
        self.heads, self.kv_heads, self.head_dim, self.page_size = heads, kv_heads, head_dim, page_size
        self.page_shape = (kv_heads, page_size, head_dim)
        self.q_width, self.k_width = heads * head_dim, kv_heads * head_dim
        if torch:
            self.dtype = _torch_dtype(dtype)
        self.desc = AttnDesc(_DTYPES[dtype], _i32(heads, "heads"), _i32(kv_heads, "kv_heads"),
                             _i32(head_dim, "head_dim"), _i32(page_size, "page_size"),
                             int(bool(causal)), _i32(window, "window"), _i32(max_kv, "max_kv"))
        self._build(lambda *a: self.lib.attn_plan_create(ctypes.byref(self._h),
                                                         ctypes.byref(self.desc), *a),
                    new_lens, kv_lens)

    def _build(self, fn, new_lens, kv_lens):
        new, kv = _lens(new_lens, "new_lens"), _lens(kv_lens, "kv_lens")
        if new.shape != kv.shape:
            raise ValueError("new_lens and kv_lens must have one entry per sequence each")
        check(fn(new.ctypes.data_as(_i32p), kv.ctypes.data_as(_i32p), len(new)))
        self.num_seqs, self.num_tokens = len(new), int(new.sum())

    def rebuild(self, new_lens, kv_lens):
        """Re-plan for the next batch in place; upload again before the next
        call."""
        self._build(lambda *a: self.lib.attn_plan_rebuild(self._h, *a), new_lens, kv_lens)
        return self

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self.lib.attn_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def workspace_bytes(self) -> int:
        return int(self.lib.attn_plan_workspace_bytes(self._h))

    def stats(self) -> dict:
        vals = [ctypes.c_int32() for _ in range(4)]
        check(self.lib.attn_plan_stats(self._h, *[ctypes.byref(v) for v in vals]))
        return dict(zip(("tokens", "units", "joins", "max_kv"), [v.value for v in vals]))

    def upload(self, ws=None, stream=None, device="cuda"):
        """Copy the plan into a device workspace (made on `device` unless
        given, from the memory of the stream that the copy is queued on).  Not
        while the stream is being captured."""
        if ws is None:
            device = torch.device(device) if stream is None else stream.device
            if device.index is None:
                device = torch.device(device.type, torch.cuda.current_device())
            ws = _new((self.workspace_bytes(),), torch.uint8, device, stream)
        elif not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous CUDA tensor")
        _enqueue(self.lib.attn_plan_upload, (self._h, ws.data_ptr(), ws.nbytes), ws.device, stream)
        self.ws, self.device = ws, ws.device
        return self


@functools.lru_cache(maxsize=1024)
def _rotary_desc(rotary_dim, layout, magnitude):
    return ctypes.byref(RotaryDesc(_i32(rotary_dim, "rotary_dim"),
                                   _code(ROTARY_LAYOUTS, layout, "layout"), magnitude))


def rotary_frequencies(rotary_dim, *, base=10000.0, scaling="none", factor=1.0, original_length=0,
                       low=1.0, high=32.0, device=None):
    """Radians that each of a head's rotary_dim / 2 pairs turns by a position,
    in 64 bits: base^(-2 i / rotary_dim), or scaled for long contexts.
    scaling "linear" divides them by factor; "by_parts" leaves pairs that make
    at least `high` turns in original_length positions, divides those of at
    most `low`, and blends between them."""
    f = np.empty(min(max(_i32(rotary_dim, "rotary_dim"), 2), 256) // 2, np.float64)
    check(load().rotary_frequencies(
        f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), rotary_dim, base,
        _code(ROTARY_SCALINGS, scaling, "scaling"), factor, original_length, low, high))
    return torch.from_numpy(f).to(device) if device is not None else torch.from_numpy(f)


# A layer makes these calls with tensors of a dozen properties each, so the
# properties are asked for once, in the cheapest form, and what is wrong is told
# apart only when something is.
def _refuse(t, name, plan, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != plan.dtype:
        raise TypeError(f"{name} must be {plan.dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _device(plan, t):
    """The device of a call: the plan's (one that was not uploaded is refused
    by the library)."""
    if plan.ws is not None:
        return plan.device
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("q, k and v must be CUDA tensors")
    return t.device


def _call(fn, plan, args, device, stream):
    """A call on `stream` keeps the plan's workspace until it is done (what the
    caller holds, and the current stream's order, the caller sees to)."""
    _enqueue(fn, (plan.handle, *args), device, stream)
    if stream is not None and plan.ws is not None:
        plan.ws.record_stream(stream)


def _heads(t, name, plan, width, device):
    """A matrix of the plan's tokens (and rows past them): pointer, stride."""
    if not isinstance(t, _Tensor) or t.get_device() != device.index or t.dtype != plan.dtype:
        _refuse(t, name, plan, device)
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or shape[0] < plan.num_tokens:
        raise ValueError(f"{name} must be [{plan.num_tokens} or more][{width}], got {list(shape)}")
    ld, step = t.stride()
    if step != 1:
        raise ValueError(f"{name} rows must be contiguous")
    return t.data_ptr(), (ld if shape[0] > 1 else width)


def _pages_of(t, name, plan, device):
    """A cache's shape and its page, head and token strides."""
    if not isinstance(t, _Tensor) or t.get_device() != device.index or t.dtype != plan.dtype:
        _refuse(t, name, plan, device)
    shape = t.shape
    if shape[1:] != plan.page_shape:
        raise ValueError(f"{name} must be [pages]{list(plan.page_shape)}, got {list(shape)}")
    page, head, tok, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: a token's elements must be contiguous")
    # (a dimension of one has any stride)
    return shape[0], 0 if shape[0] == 1 else page, 0 if plan.kv_heads == 1 else head, tok


# (one descriptor per distinct set of values, as the library only reads them)
@functools.lru_cache(maxsize=1024)
def _kv_desc(k, v, k_pages, v_pages):
    if k_pages[0] != v_pages[0]:
        raise ValueError("k_cache and v_cache must have the same pages")
    return ctypes.byref(KvCache(k, v, *k_pages[1:], *v_pages[1:], _i32(k_pages[0], "pages")))


def _cache(plan, k_cache, v_cache, pages, device):
    """The library's arguments of a cache and its page table."""
    desc = _kv_desc(k_cache.data_ptr() if isinstance(k_cache, _Tensor) else 0,
                    v_cache.data_ptr() if isinstance(v_cache, _Tensor) else 0,
                    _pages_of(k_cache, "k_cache", plan, device),
                    _pages_of(v_cache, "v_cache", plan, device))
    if not isinstance(pages, _Tensor) or pages.dtype != torch.int32:
        raise TypeError("pages must be an int32 CUDA tensor")
    if pages.get_device() != device.index:
        raise ValueError(f"pages is on {pages.device}, not on {device}")
    shape = pages.shape
    if len(shape) != 2 or shape[0] < plan.num_seqs:
        raise ValueError(f"pages must be [{plan.num_seqs} or more][pages of a sequence], got "
                         f"{list(shape)}")
    rows, count = shape
    ld, step = pages.stride()
    if step != 1 and count > 1:
        raise ValueError("pages must have contiguous rows")
    return desc, pages.data_ptr(), (ld if rows > 1 else count), _i32(count, "pages of a sequence")


def _vector(t, name, dtype, least, device):
    """A contiguous vector's pointer and length."""
    if not isinstance(t, _Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    shape = t.shape
    if len(shape) != 1 or shape[0] < least or (shape[0] > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {least} or more")
    return t.data_ptr(), shape[0]


def _padded(q, plan, device, stream):
    """A tensor like q for a call's results; rows past the plan's tokens are
    zeros."""
    t = _new(q.shape, q.dtype, device, stream)
    if q.shape[0] > plan.num_tokens:
        with torch.cuda.stream(stream):
            t[plan.num_tokens:].zero_()
    return t


def paged_attention(plan, q, k_cache, v_cache, pages, *, scale=None, o=None, stream=None):
    """Attention of the plan's tokens over their sequences' keys in the cache:

        o = softmax(scale q . k) v

    for every query head, over the keys that the plan lets the token see; zeros
    where there are none, NaN where all of them score -inf.  q and o are [tokens][heads * head_dim] (q may be a
    slice of the q/k/v product; rows past the plan's tokens are not looked at
    and stay as they are, or are zeros in a new o), k_cache and v_cache
    [pages][kv_heads][page_size][head_dim] with contiguous elements and any
    strides of multiples of 8, pages int32 [sequences][pages of a sequence].
    scale defaults to head_dim^-0.5.  What a token does not see does not reach
    it, also where it is infinite or NaN; a page outside the cache counts as
    absent.  Calls that share a plan's workspace must not overlap.  Inference
    only.  Returns o."""
    device = _device(plan, q)
    qp, ldq = _heads(q, "q", plan, plan.q_width, device)
    scale = plan.head_dim ** -0.5 if scale is None else float(scale)
    if o is None:
        o = _padded(q, plan, device, stream)
    op, ldo = _heads(o, "o", plan, plan.q_width, device)
    _call(plan.lib.paged_attention, plan,
          (qp, ldq, *_cache(plan, k_cache, v_cache, pages, device), scale, op, ldo), device, stream)
    return o


def rotary_append(plan, q, k, v, k_cache, v_cache, pages, freqs, *, layout="half", magnitude=1.0,
                  positions=None, q_out=None, stream=None):
    """Rotary positions on the plan's tokens, and their keys and values into
    the pages.  With angle a = position * freqs[i], pair (x, y) of a head's
    first 2 len(freqs) elements becomes

        magnitude * (x cos a - y sin a, y cos a + x sin a).

    layout "half": the pair is elements i and i + len(freqs); "interleaved":
    2 i and 2 i + 1.  q is returned rotated, in q_out (which may be q) or a new
    tensor; k goes rotated, and v as it is, to the places of the plan's tokens
    in the cache.  freqs: float64 on the device (rotary_frequencies), or None
    to append alone.  positions: int32 [tokens], or None for the tokens' places
    among their keys.  q may be None (an encoder's keys and values), or k, v,
    both caches and pages together (queries alone).  A cache in which two
    places have elements in common is refused.  Other arguments as
    paged_attention."""
    if q is None and k is None:
        raise ValueError("neither q nor k")
    device = _device(plan, k if q is None else q)
    qp = ldq = op = ldo = kp = ldk = vp = ldv = pp = fp = n = 0
    if q is not None:
        qp, ldq = _heads(q, "q", plan, plan.q_width, device)
        if q_out is None:
            q_out = _padded(q, plan, device, stream)
        op, ldo = _heads(q_out, "q_out", plan, plan.q_width, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    absent = (k is None) + (v is None) + (k_cache is None) + (v_cache is None) + (pages is None)
    if absent == 0:
        kp, ldk = _heads(k, "k", plan, plan.k_width, device)
        vp, ldv = _heads(v, "v", plan, plan.k_width, device)
        cache = _cache(plan, k_cache, v_cache, pages, device)
    elif absent == 5:
        cache = (None, 0, 0, 0)
    else:
        raise ValueError("k, v, k_cache, v_cache and pages are given together or not at all")
    if positions is not None:
        pp, _ = _vector(positions, "positions", torch.int32, plan.num_tokens, device)
    if freqs is not None:
        fp, n = _vector(freqs, "freqs", torch.float64, 1, device)
    desc = _rotary_desc(2 * n, layout, float(magnitude))
    _call(plan.lib.rotary_append, plan, (desc, qp, ldq, op, ldo, kp, ldk, vp, ldv, *cache, pp, fp),
          device, stream)
    return q_out
