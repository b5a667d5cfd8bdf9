"""AdamW over many tensors in one launch (the C entry point fljsd_adamw_step)."""
from __future__ import annotations

from operator import attrgetter

import numpy as np
import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._streams import Memory, hand_over, on, require_cuda
from .api import _DT
from .clip import check_max_norm, table, workspace

_BLOCK = 128  # elements of one 8-bit state block

# the layout of fljsd_adamw_tensor
_ENTRY = np.dtype([(n, np.uint64) for n in ("grad", "param", "master", "exp_avg", "exp_avg_sq",
                                            "exp_avg_scale", "exp_avg_sq_scale")] +
                  [("n", np.int64)])


_DTYPE, _DEVICE = attrgetter("dtype"), torch.Tensor.get_device  # (-1 off the GPUs)


def _ptrs(ts):
    return list(map(torch.Tensor.data_ptr, ts))


class AdamW:
    """AdamW for a list of parameters of one dtype (fp32 or bf16) on one device.

    ``state_bits``: 32 (fp32 moments) or 8 (e4m3 codes of the first moment and of the
    second's root, one fp32 scale for 128 elements; a root below about 2^-19 of its block's
    largest is held as 0, and the next step then divides by the new gradient's part and
    ``eps`` alone, so ``eps`` bounds it). ``master``: True to keep fp32
    weights beside bf16 parameters, or a list of them. The states may be given
    (``exp_avg``, ``exp_avg_sq`` and, in 8 bits, their scales, with ``step`` the number
    of steps they have taken, or a list of each parameter's), e.g. from a checkpoint: they
    are stepped in place.

    ``step(grads)`` takes the gradients in the parameters' order, or the parameters'
    ``.grad``; a gradient of None leaves its parameter, its states and its number of steps
    (``param_steps``) as they are. ``steps`` is the number of steps that moved any. ``lr``
    and ``weight_decay`` may be changed between steps.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, *,
                 state_bits=32, master=None, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None,
                 exp_avg_sq_scale=None, step=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        p0 = self.params[0]
        self.device, self.dtype = p0.device, p0.dtype
        if self.dtype not in _DT:
            raise ValueError(f"parameters have dtype {self.dtype}, expected one of {list(_DT)}")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is {state_bits}, expected 8 or 32")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits = state_bits
        self.grad_norm = None  # of the last step that was given a max_norm
        counts = np.array(step, dtype=np.int64) if isinstance(step, (list, tuple, np.ndarray)) else None
        if counts is not None and counts.shape != (len(self.params),):
            raise ValueError(f"step has {counts.size} numbers, expected {len(self.params)}")
        self.steps = int(step) if counts is None else int(counts.max())
        # steps that a parameter has not taken part in (None: all have in each)
        self._missed = None if counts is None or (counts == self.steps).all() else self.steps - counts
        self._check("params", self.params, self.dtype)
        own_master = master is True
        if own_master:
            master = [p.detach().float() for p in self.params]
        self._master = tuple(master) if master else None
        if self.master and self.dtype != torch.bfloat16:
            raise ValueError("master weights are kept beside bf16 parameters")
        sd = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        given = (exp_avg is not None, exp_avg_sq is not None, exp_avg_scale is not None,
                 exp_avg_sq_scale is not None)
        if any(given) and given != (True, True, state_bits == 8, state_bits == 8):
            raise ValueError("states are given all together, with scales in 8 bits")
        self._exp_avg = tuple(exp_avg) if exp_avg is not None else self._zeros(sd)
        self._exp_avg_sq = tuple(exp_avg_sq) if exp_avg_sq is not None else self._zeros(sd)
        self._exp_avg_scale = self._exp_avg_sq_scale = None
        if state_bits == 8:
            self._exp_avg_scale = tuple(exp_avg_scale) if exp_avg_scale is not None else self._scales()
            self._exp_avg_sq_scale = (tuple(exp_avg_sq_scale) if exp_avg_sq_scale is not None
                                      else self._scales())
        sizes = [p.numel() for p in self.params]
        for name, ts, dt, want in (
                ("master", self.master, torch.float32, sizes), ("exp_avg", self.exp_avg, sd, sizes),
                ("exp_avg_sq", self.exp_avg_sq, sd, sizes),
                ("exp_avg_scale", self.exp_avg_scale, torch.float32, None),
                ("exp_avg_sq_scale", self.exp_avg_sq_scale, torch.float32, None)):
            if ts is not None:
                self._check(name, ts, dt, want or [-(-n // _BLOCK) for n in sizes])
        made = [] if exp_avg is not None else [*self.exp_avg, *self.exp_avg_sq,
                                               *(self.exp_avg_scale or ()), *(self.exp_avg_sq_scale or ())]
        made += self.master if own_master else ()
        self._memory = Memory(made) if made and self.device.type == "cuda" else None
        self._sizes = sizes
        # (what the table points at is kept, whatever becomes of the tensors)
        self._storages = [t.untyped_storage() for ts in (self.master, self.exp_avg, self.exp_avg_sq,
                                                         self.exp_avg_scale, self.exp_avg_sq_scale)
                          for t in ts or ()]
        self._stepped = [*self.params, *(self.master or ())]
        self._table = np.zeros(len(sizes), dtype=_ENTRY)
        t = self._table
        self._table_at = t.ctypes.data
        self._at = _ptrs(self.params)
        t["param"], t["n"] = self._at, sizes
        t["exp_avg"], t["exp_avg_sq"] = _ptrs(self.exp_avg), _ptrs(self.exp_avg_sq)
        if self.master:
            t["master"] = _ptrs(self.master)
        if state_bits == 8:
            t["exp_avg_scale"] = _ptrs(self.exp_avg_scale)
            t["exp_avg_sq_scale"] = _ptrs(self.exp_avg_sq_scale)

    # The weights and states that are stepped, where they lay at construction: their contents
    # may be written, but no other tensor put in their place.
    master = property(lambda self: self._master)
    exp_avg = property(lambda self: self._exp_avg)
    exp_avg_sq = property(lambda self: self._exp_avg_sq)
    exp_avg_scale = property(lambda self: self._exp_avg_scale)
    exp_avg_sq_scale = property(lambda self: self._exp_avg_sq_scale)

    @property
    def param_steps(self):
        """The number of steps that each parameter has taken."""
        if self._missed is None:
            return [self.steps] * len(self.params)
        return (self.steps - self._missed).tolist()

    def _zeros(self, dtype):
        return tuple(torch.zeros(p.numel(), dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                                 device=self.device).view(dtype) for p in self.params)

    def _scales(self):
        return tuple(torch.zeros(-(-p.numel() // _BLOCK), dtype=torch.float32, device=self.device)
                     for p in self.params)

    def _check(self, name, ts, dtype, sizes=None):
        if sizes is not None and len(ts) != len(sizes):
            raise ValueError(f"{name} has {len(ts)} tensors, expected {len(sizes)}")
        for i, t in enumerate(ts):
            if t.device != self.device or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be a contiguous {dtype} tensor on {self.device}")
            if sizes is not None and t.numel() != sizes[i]:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements, expected {sizes[i]}")

    def step(self, grads=None, *, grad_scale=None, max_norm=None, stream=None):
        """One step. ``grad_scale``: an fp32 scalar on the device that every gradient is
        multiplied by. ``max_norm``: the step goes by gradients scaled (after that) to at
        most this norm of all of them together, as :func:`clip_grads` does; the gradients
        stay as they are, and ``grad_norm`` is their norm before that, an fp32 scalar on
        the device (0 without any gradients). A norm of NaN makes every stepped value NaN.
        The norm is that of this call's gradients alone. Several objects that share one (say of
        bf16 and of fp32 parameters) take its factor each: ``norm = grad_norm(all gradients)``,
        ``step(..., grad_scale=(max_norm / (norm + 1e-6)).clamp(max=1))``."""
        if max_norm is not None:
            check_max_norm(max_norm)
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self._sizes):
            raise ValueError(f"{len(grads)} gradients for {len(self._sizes)} parameters")
        t = self._table
        at = _ptrs(self.params)
        if at != self._at:  # parameters whose storage was replaced (p.data = ...)
            self._check("params", self.params, self.dtype, self._sizes)
            self._at = at
            t["param"] = at
            self._stepped = [*self.params, *(self.master or ())]
        live, sizes, stepped, out = grads, self._sizes, self._stepped, None
        try:
            t["grad"] = _ptrs(grads)
        except TypeError:  # some are None: those parameters stay as they are
            out = np.array([g is None for g in grads])
            t = t[~out]
            live = [g for g in grads if g is not None]
            sizes = [n for g, n in zip(grads, sizes) if g is not None]
            stepped = [x for x, g in zip(stepped, grads * 2) if g is not None]
            if not live:
                if max_norm is not None:  # (the norm of none)
                    require_cuda("params[0]", self.params[0])
                    with on(stream, self.device):
                        self.grad_norm = torch.zeros((), dtype=torch.float32, device=self.device)
                    hand_over((self.grad_norm,), stream, self.device)
                return
            t["grad"] = _ptrs(live)
        dt, dev = live[0].dtype, self.device
        require_cuda("params[0]", self.params[0])
        # (whole-list checks: a step of many small tensors is bound by this function)
        if (dt not in _DT or set(map(_DTYPE, live)) != {dt} or set(map(_DEVICE, live)) != {dev.index}
                or not all(map(torch.Tensor.is_contiguous, live))
                or list(map(torch.Tensor.numel, live)) != sizes):
            raise ValueError(f"gradients must be contiguous, of one dtype of {list(_DT)}, on {dev}, "
                             "and as large as their parameters")
        if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                       or grad_scale.device != dev):
            raise ValueError(f"grad_scale must be one fp32 value on {dev}")
        at = self._table_at if out is None else t.ctypes.data
        o = _lib.make_adamw_options(self.lr, *self.betas, self.eps, self.weight_decay,
                                    self.steps + 1, _DT[self.dtype], _DT[dt], self.state_bits,
                                    int(self.master is not None))
        with on(stream, dev):
            if self._memory is not None:
                self._memory.use()
            if max_norm is not None:
                both = torch.empty(2, dtype=torch.float32, device=dev)  # norm, factor
                g = table(t["grad"], t["n"], dt)
                _lib.fljsd_grad_norm(g.ctypes.data, len(g), _lib.FLJSD_NORM_2, max_norm, grad_scale,
                                     both[0], both[1], workspace(len(g), dev))
                self.grad_norm, grad_scale = both[0], both[1]
            if self._missed is None:
                _lib.fljsd_adamw_step(o, at, len(t), grad_scale)
            else:
                missed = self._missed if out is None else self._missed[~out]
                steps = self.steps + 1 - missed
                _lib.fljsd_adamw_step_each(o, at, steps.ctypes.data, len(t), grad_scale)
        if max_norm is not None:
            hand_over((self.grad_norm,), stream, dev)
        # autograd's own check of what it saved: these have changed
        increment_version(stepped)
        self.steps += 1
        if out is not None:
            self._missed = out + (0 if self._missed is None else self._missed)


__all__ = ["AdamW"]
