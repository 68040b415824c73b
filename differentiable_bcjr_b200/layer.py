"""Calls around a quantised layer (C ABI in include/bcjr_layer.h): the AdamW
step that trains weight preimages and codebooks, the 4-bit group quantiser,
the packing of hard-decoded trellis states, and products with either kind of
packed weights.

As in the rest of the binding, tensors must be contiguous CUDA tensors of one
device, every call is asynchronous on that device's current stream, malformed
arguments raise before anything is launched, and nothing falls back to
PyTorch.  The products have no gradient: they serve frozen layers, and refuse
tensors that want one (outside torch.no_grad()).
"""
from __future__ import annotations

from array import array
import ctypes

import torch

from . import BCJRError, lib

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
STATE_BLOCK = 256  # elements of a block of optimiser state


_calls = {}


def _call(name, index, *args):
    """The library's call `name` on the current stream of device `index`."""
    call = _calls.get(name)
    if call is None:
        call = _calls[name] = getattr(lib(), name)
    if _current_device() == index:
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _raw_stream(index))
    if status:
        raise BCJRError(status, name)


def _on_device(t, name):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (libbcjr has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return index


def _like(t, name, shape, dtype, index):
    if t.get_device() == index and t.dtype is dtype and t.is_contiguous() and t.shape == shape:  # the usual case
        return
    if _on_device(t, name) != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _tokens(x):
    """x [..., cols] as (device index, type code, leading sizes, cols)."""
    index, kind = x.get_device(), _DTYPE.get(x.dtype)
    if index < 0 or kind is None or not x.is_contiguous():
        _on_device(x, "x")
        _dtype(x, "x")
    lead = list(x.shape)
    if not lead or lead[-1] < 1:
        raise ValueError("x must be [..., cols]")
    return index, kind, lead, lead.pop()


def _dtype(t, name):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    return code


class _AdamWOptions(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("step_ptr", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p), ("seed", ctypes.c_uint32)]


def adamw_state(params, state_bits=32):
    """Zeroed states for `adamw_step` on `params`: (exp_avg, exp_avg_sq, scales or None)."""
    params = list(params)
    if state_bits not in (8, 32):
        raise ValueError("state_bits must be 8 or 32")
    if not params:
        raise ValueError("there are no parameters")
    blocks = sum(-(-p.numel() // STATE_BLOCK) for p in params)
    dev = params[0].device
    kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
    first = torch.zeros(blocks * STATE_BLOCK, dtype=torch.float32 if state_bits == 32 else torch.uint8, device=dev).view(kind)
    second = torch.zeros_like(first)
    return first, second, torch.zeros((2, blocks), device=dev) if state_bits == 8 else None


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
               scales=None, grad_scale=None, seed=0):
    """One AdamW step of every tensor of `params`, in place, in one launch.

    `params` and `grads` are lists of as many tensors: float32 parameters with
    gradients of any float type, or 16-bit ones with gradients of the same
    type or float32.  A gradient may be None: that parameter and its states
    are left as they are.  The states are flat (see `adamw_state`; tensor i
    starts at the next multiple of 256 elements): float32, or float8_e4m3fn
    codes with `scales` float32 [2][blocks].  With 8-bit states `exp_avg_sq`
    holds the root of the second moment, and codes are rounded stochastically
    from a hash of `seed`, the step and the element's index.  The library
    refuses states that share memory with one another, a parameter or a gradient.

    `step` counts from 1; it is a number, or an int64 CUDA tensor of one
    element that the kernel reads (what a captured graph needs: with a number,
    capture is refused, because every replay would repeat that step).
    `grad_scale`, a float32 CUDA tensor of one element, multiplies every
    gradient (clipping or loss scaling without a synchronisation).
    """
    plan = _adamw_plan(params, grads, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay, scales, grad_scale, seed)
    if plan is not None:
        _adamw_run(plan)


def _adamw_plan(params, grads, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay, scales, grad_scale, seed):
    """The arguments of `adamw_step` checked and laid out for `_adamw_run`; None if there is nothing to do."""
    n = len(params)
    if len(grads) != n:
        raise ValueError(f"{n} parameters and {len(grads)} gradients")
    if n == 0:
        return None
    given = [g for g in grads if g is not None]
    both = list(params) + given
    index = params[0].get_device()
    if index < 0 or set(map(_get_device, both)) != {index}:
        raise ValueError("parameters and gradients must be CUDA tensors of one device (libbcjr has no CPU path)")
    if not all(map(_is_contiguous, both)):
        raise ValueError("parameters and gradients must be contiguous")
    kind = _one_dtype(params, "parameters")
    gkind = _one_dtype(given, "gradients") if given else kind
    if kind != torch.float32 and gkind not in (torch.float32, kind):
        raise ValueError(f"{kind} parameters take gradients of {kind} or float32, not {gkind}")
    numel = list(map(_numel, params))
    if len(given) == n:
        gp, same = list(map(_data_ptr, grads)), list(map(_numel, grads)) == numel
    else:
        gp = [0 if g is None else g.data_ptr() for g in grads]
        same = all(g is None or g.numel() == m for g, m in zip(grads, numel))
    if not same:
        raise ValueError("every gradient must have as many elements as its parameter")
    pp = list(map(_data_ptr, params))
    blocks = sum([m + 255 >> 8 for m in numel])
    bits = 32 if scales is None else 8
    held = torch.float32 if bits == 32 else torch.float8_e4m3fn
    flat = (blocks * STATE_BLOCK,)
    _like(exp_avg, "exp_avg", flat, held, index)
    _like(exp_avg_sq, "exp_avg_sq", flat, held, index)
    if scales is not None:
        _like(scales, "scales", (2, blocks), torch.float32, index)
    o = _AdamWOptions(lr, betas[0], betas[1], eps, weight_decay, 0, None, None, seed & 0xFFFFFFFF)
    if isinstance(step, torch.Tensor):
        _like(step, "step", step.shape, torch.int64, index)
        if step.numel() != 1:
            raise ValueError("step must have one element")
        o.step_ptr = step.data_ptr()
    else:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("a captured step needs its count in a CUDA tensor")
        o.step = int(step)
    if grad_scale is not None:
        _like(grad_scale, "grad_scale", grad_scale.shape, torch.float32, index)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one element")
        o.grad_scale = grad_scale.data_ptr()
    table = array("Q", bytes(24 * n))
    table[0::3] = array("Q", pp)
    table[1::3] = array("Q", gp)
    table[2::3] = array("Q", numel)
    return (index, table, (_DTYPE[kind], _DTYPE[gkind], bits, exp_avg.data_ptr(), exp_avg_sq.data_ptr(),
                           None if scales is None else scales.data_ptr(), ctypes.byref(o)),
            params, params if len(given) == n else [p for p, g in zip(params, grads) if g is not None])


def _adamw_check(plan):
    """Raises if the library refuses the plan's types or hyperparameters (by a call without tensors, which launches nothing)."""
    index, _, args, _, _ = plan
    _call("bcjr_adamw_step", index, None, 0, *args)


def _adamw_run(plan):
    index, table, args, params, moved = plan
    try:
        _call("bcjr_adamw_step", index, table.buffer_info()[0], len(params), *args)
    except BCJRError:
        size = 4 if params[0].dtype == torch.float32 else 2
        spans = sorted((a, a + m * size) for a, m in zip(table[0::3], table[2::3]) if m)
        if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
            raise ValueError("parameters must not overlap") from None
        raise
    _increment_version(moved)


_get_device, _is_contiguous, _numel, _data_ptr = (torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.numel,
                                                  torch.Tensor.data_ptr)
_get_dtype = torch.Tensor.dtype.__get__
_increment_version = torch.autograd.graph.increment_version


def _one_dtype(ts, name):
    kinds = set(map(_get_dtype, ts))
    if len(kinds) != 1 or not kinds <= _DTYPE.keys():
        raise ValueError(f"{name} must all be float32, float16 or bfloat16, not {sorted(map(str, kinds))}")
    return kinds.pop()


def _into(out, shape, x, index, name, weights):
    """Checks an output of the caller's, into which nothing may be written that is still read for other rows."""
    _like(out, "out", tuple(shape), x.dtype, index)
    a = out.data_ptr()
    for what, t in (("x", x), *weights):
        if t is not None:
            b = t.data_ptr()
            if a < b + t.numel() * t.element_size() and b < a + out.numel() * out.element_size():
                raise ValueError(f"out must not overlap {what}")
    if out.requires_grad:
        _no_gradient(name)
    return out


def _no_gradient(name):
    """For a call of which some tensor wants a gradient."""
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no gradient: call it under torch.no_grad(), or with detached tensors")


def _groups(cols, group_size):
    if group_size < 0 or (group_size % 128 and group_size not in (32, 64)):
        raise ValueError("group_size must be 32, 64, a multiple of 128, or 0 for the whole row")
    return -(-cols // group_size) if group_size else 1


def int4_quantize(w, group_size=128, zero_point=False, scale_dtype=None):
    """w [rows][cols] rounded to 4 bits with one scale a group of `group_size`
    columns (32, 64, a multiple of 128, or 0 for the whole row).  Returns
    (packed uint8 [ceil(rows/16)][ceil(cols/128)][1024], scales [groups][rows]
    of `scale_dtype` (w's by default), zeros uint8 [groups][rows] or None).
    Symmetric codes stand for -7..7 (8 is zero); with `zero_point` a group's
    range from its least to its largest value (0 among them) takes codes 0..15.
    bcjr_layer.h gives the layout of the packed tiles."""
    index = _on_device(w, "w")
    if w.dim() != 2 or w.shape[1] < 1:
        raise ValueError("w must be [rows][cols]")
    rows, cols = w.shape
    groups = _groups(cols, group_size)
    kind = w.dtype if scale_dtype is None else scale_dtype
    if kind not in _DTYPE:
        raise ValueError(f"scale_dtype must be float32, float16 or bfloat16, not {kind}")
    dev = w.device
    packed = torch.empty((-(-rows // 16), -(-cols // 128), 1024), dtype=torch.uint8, device=dev)
    scales = torch.empty((groups, rows), dtype=kind, device=dev)
    zeros = torch.empty((groups, rows), dtype=torch.uint8, device=dev) if zero_point else None
    _call("bcjr_int4_quantize", index, w.data_ptr(), _dtype(w, "w"), rows, cols, group_size, packed.data_ptr(),
          scales.data_ptr(), _DTYPE[kind], None if zeros is None else zeros.data_ptr())
    return packed, scales, zeros


def int4_matmul(x, packed, scales, zeros=None, group_size=128, out=None):
    """x [..., cols] times the transpose of 4-bit weights: [..., rows] of x's
    type, sums in float32.  `packed`, `scales`, `zeros` and `group_size` as
    `int4_quantize` gives and takes them."""
    index, kind, lead, cols = _tokens(x)
    grouped = scales.shape
    if len(grouped) != 2 or grouped[0] != _groups(cols, group_size):
        raise ValueError("scales must be [groups][rows]")
    rows = grouped[1]
    if scales.get_device() != index or not scales.is_contiguous():
        _like(scales, "scales", grouped, scales.dtype, index)
    _like(packed, "packed", (rows + 15 >> 4, cols + 127 >> 7, 1024), torch.uint8, index)
    if zeros is not None:
        _like(zeros, "zeros", grouped, torch.uint8, index)
    lead.append(rows)
    if x.requires_grad or scales.requires_grad:
        _no_gradient("int4_matmul")
    if out is None:
        y = x.new_empty(lead)
    else:
        y = _into(out, lead, x, index, "int4_matmul", (("packed", packed), ("scales", scales), ("zeros", zeros)))
    _call("bcjr_int4_matmul", index, x.data_ptr(), kind, x.numel() // cols, rows, cols, packed.data_ptr(),
          scales.data_ptr(), _dtype(scales, "scales"), None if zeros is None else zeros.data_ptr(), group_size,
          y.data_ptr())
    if out is not None:
        _increment_version(out)
    return y


def _trellis(state_bits, k):
    if not (1 <= k <= 4 and k <= state_bits <= 16):
        raise ValueError("packed trellis codes need 1 <= k <= 4 and k <= state_bits <= 16")


def _trellis_groups(cols, seq_len, group_size):
    if not group_size:
        return 1
    if group_size < 0 or not ((group_size % seq_len == 0 and cols % group_size == 0) or
                              (group_size % 16 == 0 and seq_len % group_size == 0)):
        raise ValueError("group_size must be 0, a multiple of seq_len that divides cols, or a multiple of 16 that divides seq_len")
    return cols // group_size


def trellis_words(state_bits, k, seq_len):
    """32-bit words that a packed sequence of seq_len states takes."""
    _trellis(state_bits, k)
    return (seq_len * k + state_bits - k + 31) // 32


def trellis_pack(states, state_bits, k, check=False):
    """Hard-decoded states (int32 [n_seq][seq_len], as `viterbi_decode` gives
    them) as one bit stream a sequence, k bits a step after the first:
    int32 [n_seq][trellis_words(state_bits, k, seq_len)].  With `check` the
    call waits for the GPU and raises if the states are no path of the trellis;
    without it the words of such a sequence mean nothing."""
    index = _on_device(states, "states")
    if states.dim() != 2 or states.shape[1] < 1 or states.dtype != torch.int32:
        raise ValueError("states must be int32 [n_seq][seq_len]")
    n_seq, n = states.shape
    packed = states.new_empty((n_seq, trellis_words(state_bits, k, n)))
    bad = torch.zeros(1, dtype=torch.int32, device=states.device) if check else None
    _call("bcjr_trellis_pack", index, states.data_ptr(), state_bits, k, n, n_seq, packed.data_ptr(),
          None if bad is None else bad.data_ptr())
    if check and bad.item():
        raise ValueError("the states are not a path of the bitshift trellis")
    return packed


def trellis_matmul(x, packed, codebook, state_bits, k, seq_len, scales=None, group_size=0, out=None):
    """x [..., cols] times the transpose of packed trellis weights: [..., rows]
    of x's type.  A row's weights are cols / seq_len sequences of `packed`
    (int32 [rows * cols / seq_len][words], see `trellis_pack`) read through
    `codebook` [2^state_bits], each times `scales` (float32 [cols /
    group_size][rows]) when given.  group_size: 0 for one scale a row, a
    multiple of seq_len that divides cols, or a multiple of 16 that divides
    seq_len.  Products and sums are float32."""
    index, kind, lead, cols = _tokens(x)
    if seq_len < 1 or cols % seq_len:
        raise ValueError("a row must be whole sequences")
    seqs = cols // seq_len
    words = trellis_words(state_bits, k, seq_len)
    if packed.dim() != 2 or packed.shape[0] % seqs:
        raise ValueError("packed must be [rows * cols / seq_len][words]")
    rows = packed.shape[0] // seqs
    _like(packed, "packed", (rows * seqs, words), torch.int32, index)
    if codebook.get_device() != index or not codebook.is_contiguous() or codebook.shape != (1 << state_bits,):
        _like(codebook, "codebook", (1 << state_bits,), codebook.dtype, index)
    if scales is not None:
        _like(scales, "scales", (_trellis_groups(cols, seq_len, group_size), rows), torch.float32, index)
    lead.append(rows)
    if x.requires_grad or codebook.requires_grad or (scales is not None and scales.requires_grad):
        _no_gradient("trellis_matmul")
    if out is None:
        y = x.new_empty(lead)
    else:
        y = _into(out, lead, x, index, "trellis_matmul", (("packed", packed), ("codebook", codebook), ("scales", scales)))
    _call("bcjr_trellis_matmul", index, x.data_ptr(), kind, x.numel() // cols, rows, cols, packed.data_ptr(),
          codebook.data_ptr(), _dtype(codebook, "codebook"), state_bits, k, seq_len,
          None if scales is None else scales.data_ptr(), group_size, y.data_ptr())
    if out is not None:
        _increment_version(out)
    return y
