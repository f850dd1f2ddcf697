"""The operators around the delta over the C ABI (argument marshalling only):
the residual stream's norms, the frozen layer's product, and the product with
the delta inside its activation.

A decode step makes hundreds of such calls, each a few microseconds on the
GPU, so what is the same from call to call (descriptors, device checks) is
made once and each tensor is asked for each of its properties once."""
from __future__ import annotations

import ctypes
import functools

try:
    import torch
except ImportError:                    # sizes can be asked for without it
    torch = None

from ._lib import (ACTS, GATE_ACTS, LORA_BF16, LORA_F32, NORMS, LinearDesc, NormDesc, check, load)
from .api import _DTYPES, _i32, _offsets, _projs

_f32 = ctypes.c_float
_CODES = {torch.bfloat16: LORA_BF16, torch.float32: LORA_F32} if torch else {}
_Tensor = torch.Tensor if torch else ()


def _dtype_code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    return code


def _matrix(t, name, shape, dtype, device):
    """A 2-D CUDA tensor with contiguous rows, as (pointer, row stride); None
    for shape, dtype or device: any."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    s = t.shape
    if s != shape and (shape is not None or len(s) != 2):
        raise ValueError(f"{name} must be {list(shape) if shape else '2-D'}, got {list(s)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    rows, cols = s
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} rows must be contiguous")
    return t.data_ptr(), (ld if rows > 1 else cols)


def _vector(t, name, n, dtype, device):
    """A contiguous vector of n elements, or None: its pointer (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def _code(table, key, what):
    if key not in table:
        raise ValueError(f"{what} {key!r} is not one of {', '.join(map(repr, table))}")
    return table[key]


def _enqueue(fn, args, device, stream):
    """Calls the library with `stream` (None: the device's current one) as the
    last argument, with `device` current for the launches."""
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, not on {device}")
        handle = stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        check(fn(*args, handle))
    else:
        with torch.cuda.device(device):
            check(fn(*args, handle))


def _new(shape, dtype, device, stream):
    """A tensor for a launch on `stream` (None: the current one).  Memory is
    given out again in the order of the stream it was made on, with its last
    owner's work perhaps still queued there, so it is made on the launch's own
    stream; and it goes back only behind the uses that the caller's current
    stream has of it by then."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


# (descriptors are only read by the library: one per distinct set of values,
# which have to be plain ones: a tensor is remembered by what it is, not by
# the value it holds)
@functools.lru_cache(maxsize=1024)
def _norm_desc(dtype, stream_dtype, T, d, post, pre, gate_act, unit_offset, alpha, beta, eps):
    return ctypes.byref(NormDesc(
        dtype, stream_dtype, _i32(T, "num_tokens"), _i32(d, "width"),
        _code(NORMS, post, "post norm"), _code(NORMS, pre, "pre norm"),
        _code(GATE_ACTS, gate_act, "gate_act"), int(unit_offset), alpha, beta, eps))


def block_norm(h, o=None, *, post="none", post_weight=None, post_bias=None, gate=None,
               gate_act="none", alpha=1.0, beta=1.0, pre="rms", pre_weight=None, pre_bias=None,
               eps=1e-5, unit_offset=False, h_out=None, u=None, stream=None):
    """The residual stream past a block and the next block's input, in one pass:

        h_out = beta h + alpha gate_act(gate) * N_post(o),   u = N_pre(h_out)

    h [T][d] is the residual stream, o [T][d] the block's output (None: there
    is none yet).  post and pre name the norms ("none", "rms", "layer"), each
    with an optional weight and bias [d]; gate is a vector [d] or a row per
    token [T][d], through gate_act ("none", "sigmoid", "tanh").  bfloat16 or
    float32, with a float32 stream beside bfloat16 blocks if h is float32.
    u is formed from the unrounded h_out.  Returns (h_out, u), in the tensors
    given or new ones; h_out may be h itself.  Without a block output and
    with beta 1 the stream is unchanged: h itself is returned unless h_out is
    given.  u is None with pre="none".  Inference only."""
    hp, ldh = _matrix(h, "h", None, None, None)
    shape, dev, hdt = h.shape, h.device, h.dtype
    T, d = shape
    dt = hdt
    for t in (o, u, pre_weight, pre_bias):
        if t is not None:
            dt = t.dtype
            break
    # (the values now, also of scales that are held in tensors)
    alpha, beta, eps = _f32(alpha).value, _f32(beta).value, _f32(eps).value
    desc = _norm_desc(_dtype_code(dt, "o"), _dtype_code(hdt, "h"), T, d, post, pre, gate_act,
                      bool(unit_offset), alpha, beta, eps)
    op, ldo = _matrix(o, "o", shape, dt, dev) if o is not None else (0, d)
    gp, ldg = 0, 0
    if gate is not None:
        if gate.dim() == 1:
            gp = _vector(gate, "gate", d, dt, dev)
        else:
            gp, ldg = _matrix(gate, "gate", shape, dt, dev)
    unchanged = o is None and beta == 1.0 and h_out is None
    if h_out is None and not unchanged:
        h_out = _new(shape, hdt, dev, stream)
    if u is None and pre != "none":
        u = _new(shape, dt, dev, stream)
    hop, ldho = _matrix(h_out, "h_out", shape, hdt, dev) if h_out is not None else (0, d)
    up, ldu = _matrix(u, "u", shape, dt, dev) if u is not None else (0, d)
    _enqueue(load().block_norm,
             (desc, hp, ldh, op, ldo, _vector(post_weight, "post_weight", d, dt, dev),
              _vector(post_bias, "post_bias", d, dt, dev), gp, ldg,
              _vector(pre_weight, "pre_weight", d, dt, dev),
              _vector(pre_bias, "pre_bias", d, dt, dev), hop, ldho, up, ldu), dev, stream)
    return (h if unchanged else h_out), u


@functools.lru_cache(maxsize=1024)
def _linear_desc(num_tokens, n, k, dtype, glu, act="none"):
    return ctypes.byref(LinearDesc(dtype, _i32(num_tokens, "num_tokens"), _i32(n, "n"), _i32(k, "k"),
                                   _code(ACTS, act, "act"), int(glu)))


def linear_workspace_bytes(num_tokens: int, n: int, k: int, dtype: str = "bf16",
                           glu: bool = False, up_to: bool = False) -> int:
    """Bytes of workspace a frozen_linear call of these sizes takes (0: none);
    n is the width of y.  A smaller batch may take more (it runs in more parts
    along k): with up_to, what is enough for every call of at most num_tokens
    tokens, found by trying each of them (once, when a server starts)."""
    lib = load()
    ask = lib.frozen_linear_max_workspace_bytes if up_to else lib.frozen_linear_workspace_bytes
    return int(ask(_linear_desc(num_tokens, n, k, _DTYPES[dtype], bool(glu))))


def sgmv_linear_workspace_bytes(pool, num_tokens: int, n: int, k: int, nproj: int,
                                glu: bool = False, plan=None, up_to: bool = False) -> int:
    """The same for sgmv_linear over nproj projections of the pool: what is
    enough for any batch of num_tokens tokens over its adapters (with up_to,
    for those of fewer tokens too), or what the given plan takes, which for a
    prompt is a fraction of it."""
    desc = _linear_desc(num_tokens, n, k, pool.desc.dtype, bool(glu))
    nproj = _i32(nproj, "nproj")
    lib = load()
    if plan is not None:
        if up_to:
            raise ValueError("a plan is one batch: plan and up_to exclude each other")
        return int(lib.sgmv_linear_plan_workspace_bytes(pool.handle, plan.handle, desc, nproj))
    ask = lib.sgmv_linear_max_workspace_bytes if up_to else lib.sgmv_linear_workspace_bytes
    return int(ask(pool.handle, desc, nproj))


def _linear_call(x, w, bias, act, glu, residual, y, ws, stream, need, fn, head, beside=()):
    """Checks the tensors of a product call, makes y and the workspace where
    they are not given, and calls fn(*head, descriptor, tensors, stream).
    beside: what else the call reads, as (name, tensor or None)."""
    xp, ldx = _matrix(x, "x", None, None, None)
    dev, dt = x.device, x.dtype
    for name, t in beside:
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")
    wp, ldw = _matrix(w, "w", None, dt, dev)
    (T, k), (wide, kw) = x.shape, w.shape
    if kw != k:
        raise ValueError(f"w has rows of {kw}, x of {k}")
    if glu and wide % 2:
        raise ValueError(f"w must hold a gate and an up of the same rows, got {wide}")
    n = wide // 2 if glu else wide
    shape = (T, n)
    desc = _linear_desc(T, n, k, _dtype_code(dt, "x"), bool(glu), act)
    bp = _vector(bias, "bias", wide, dt, dev)
    rp, ldr = _matrix(residual, "residual", shape, dt, dev) if residual is not None else (0, n)
    if y is None:
        y = _new(shape, dt, dev, stream)
    yp, ldy = _matrix(y, "y", shape, dt, dev)
    if ws is None:
        size = need(desc)
        ws = _new((size,), torch.uint8, dev, stream) if size else None
    elif not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    wsp, wsn = (ws.data_ptr(), ws.nbytes) if ws is not None else (0, 0)
    _enqueue(fn, (*head, desc, xp, ldx, wp, ldw, bp, rp, ldr, yp, ldy, wsp, wsn), dev, stream)
    return y


def frozen_linear(x, w, *, bias=None, act="none", glu=False, residual=None, y=None, ws=None,
                  stream=None):
    """The frozen layer's product with its epilogue, rounded once:

        y = act(x w^T + bias) + residual
        y = act(x wg^T + bias_g) * (x wu^T + bias_u) + residual     (glu)

    x [T][k], w [n][k] (with glu [2 n][k]: the gate's rows, then the up's),
    bias [rows of w], residual and y [T][n], all of one type, bfloat16 or
    float32; k and the row strides of x and w are multiples of 8.  act is
    "none", "relu", "silu", "gelu" or "gelu_tanh".  residual may be y.  ws: a
    workspace of linear_workspace_bytes (made per call if not given).
    Inference only.  Returns y."""
    lib = load()
    return _linear_call(x, w, bias, act, glu, residual, y, ws, stream,
                        lib.frozen_linear_workspace_bytes, lib.frozen_linear, ())


def sgmv_linear(pool, plan, layer, projs, y_offsets, x, w, *, bias=None, act="none", glu=False,
                residual=None, y=None, ws=None, stream=None):
    """frozen_linear with every token's LoRA delta inside the activation:
    before it, columns y_offsets[i] .. + h_out of x w^T + bias get
    s B (A x) of projection projs[i] (with glu the columns are the gate's n,
    then the up's n).  plan: a plain or weighted plan of x's tokens.  ws: a
    workspace of sgmv_linear_workspace_bytes (made per call, of the plan's
    size, if not given)."""
    lib = pool.lib
    count, parr = _projs(projs)
    if len(y_offsets) != count:
        raise ValueError("y_offsets must have one entry per projection")
    return _linear_call(
        x, w, bias, act, glu, residual, y, ws, stream,
        lambda d: lib.sgmv_linear_plan_workspace_bytes(pool.handle, plan.handle, d, count),
        lib.sgmv_linear,
        (pool.handle, plan.handle, _i32(layer, "layer"), count, parr, _offsets(y_offsets)),
        (("the pool", pool.slab), ("the plan's workspace", plan.ws)))
