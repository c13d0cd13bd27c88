"""AdamW over the framework's flat parameter and gradient buffers.

`AdamW` keeps the table of tensors, the optimiser's states and the step count
(on the device, so that a captured step counts its replays); `step` is one
call of eaga_adamw_step.  With bf16 weights it keeps fp32 master copies unless
told not to.  `LayerBuffers.optimizer` and `BlockBuffers.optimizer`
(buffers.py) make one over a layer's or a block's weights and gradients.
"""
from __future__ import annotations

import ctypes

import torch

from . import eaga

BLOCK = 256          # elements of an 8-bit state that share a scale


def _flat(sizes, dtype, device, per=1):
    """One zero buffer and a view of ceil(n / per) elements in it for each n, on 16-byte boundaries."""
    lens = [-(-n // per) for n in sizes]
    offs, off = [], 0
    for n in lens:
        offs.append(off)
        off += -(-n // 16) * 16
    flat = torch.zeros(off, dtype=dtype, device=device)
    return [flat[o:o + n] for o, n in zip(offs, lens)]


class AdamW:
    """params, grads: lists of contiguous tensors on one device, alike in number
    of elements (grads fp32 or bf16, params fp32 or bf16, one dtype each).

    weight_decay: a number, or one per tensor.  bits: 32 or 8, of the states.
    master: fp32 copies of bf16 weights (default: made from the weights), a list
    of them, or False for none.  m, v (with bits = 8 also m_scale, v_scale): the
    states of an earlier run; `step` its number of steps.  counters: where each
    tensor's elements begin in the count that seeds 8-bit rounding.
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, master=None,
                 m=None, v=None, m_scale=None, v_scale=None, counters=None, seed=0, step=0):
        params, grads = list(params), list(grads)
        if not params:
            raise ValueError("params: at least one tensor is required")
        if bits not in (8, 32):
            raise ValueError(f"bits: {bits}, expected 8 or 32")
        k = len(params)
        sizes = [p.numel() for p in params]
        pd, gd = params[0].dtype, grads[0].dtype if grads else None
        self.device = params[0].device
        if pd not in (torch.float32, torch.bfloat16) or gd not in (torch.float32, torch.bfloat16):
            raise ValueError(f"params and grads are fp32 or bf16 (got {pd}, {gd})")

        def take(ts, name, dtype, lens=sizes):
            ts = list(ts)
            if len(ts) != k:
                raise ValueError(f"{name}: {len(ts)} tensors, expected {k}")
            for i, (t, n) in enumerate(zip(ts, lens)):
                if t.device != self.device or not t.is_cuda:
                    raise ValueError(f"{name}[{i}]: on {t.device}, expected the params' CUDA device")
                if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
                    raise ValueError(f"{name}[{i}]: {n} contiguous elements of {dtype} expected "
                                     f"(got {t.numel()} of {t.dtype})")
            return ts

        self.params, self.grads = take(params, "params", pd), take(grads, "grads", gd)
        if pd == torch.float32:
            if master:
                raise ValueError("master: fp32 weights have no master copies")
            self.master = None
        elif master is False:
            self.master = None
        elif master is None:
            self.master = _flat(sizes, torch.float32, self.device)
            for a, p in zip(self.master, params):
                a.copy_(p.detach().reshape(-1))
        else:
            self.master = take(master, "master", torch.float32)
        sd = torch.float32 if bits == 32 else torch.uint8
        blocks = [-(-n // BLOCK) for n in sizes]
        self.m = take(m, "m", sd) if m is not None else _flat(sizes, sd, self.device)
        self.v = take(v, "v", sd) if v is not None else _flat(sizes, sd, self.device)
        self.m_scale = self.v_scale = None
        if bits == 8:
            new = lambda: _flat(sizes, torch.float32, self.device, BLOCK)
            self.m_scale = take(m_scale, "m_scale", torch.float32, blocks) if m_scale is not None else new()
            self.v_scale = take(v_scale, "v_scale", torch.float32, blocks) if v_scale is not None else new()
        decay = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * k
        if len(decay) != k:
            raise ValueError(f"weight_decay: {len(decay)} values, expected {k}")
        if counters is None:
            counters, off = [], 0
            for n in sizes:
                counters.append(off)
                off += n
        self.config = eaga.AdamwConfig(lr, betas[0], betas[1], eps, 1.0,
                                       eaga.EAGA_BF16 if pd == torch.bfloat16 else eaga.EAGA_FP32,
                                       eaga.EAGA_BF16 if gd == torch.bfloat16 else eaga.EAGA_FP32, bits, seed)
        self.sizes = sizes
        self.state = torch.tensor([step, 0], dtype=torch.int64, device=self.device)
        at = lambda ts, i: ts[i].data_ptr() if ts is not None else None
        self._table = (eaga.AdamwTensor * k)(*(
            eaga.AdamwTensor(at(self.params, i), at(self.master, i), at(self.grads, i), at(self.m, i), at(self.v, i),
                             at(self.m_scale, i), at(self.v_scale, i), sizes[i], counters[i], decay[i])
            for i in range(k)))

    @property
    def steps(self) -> int:
        """The number of steps taken (waits for the device)."""
        return int(self.state[0].item())

    def step(self, lr=None, grad_scale=1.0, stream=None):
        """One step.  lr: None for the constructor's, a number, or a device tensor of
        one fp32 value that the step reads when it runs (for captured steps)."""
        on_device = lr if isinstance(lr, torch.Tensor) else None
        c = self.config
        if grad_scale != c.grad_scale or (lr is not None and on_device is None):
            c = eaga.AdamwConfig.from_buffer_copy(c)
            c.grad_scale = grad_scale
            if on_device is None and lr is not None:
                c.lr = lr
        eaga.adamw_step(c, self._table, len(self.sizes), self.state, on_device, stream)

    def unpack(self, m_out=None, v_out=None, stream=None):
        """The 8-bit states as fp32: lists of tensors, the given ones filled or new ones."""
        if m_out is None:
            m_out = _flat(self.sizes, torch.float32, self.device)
        if v_out is None:
            v_out = _flat(self.sizes, torch.float32, self.device)
        self.unpacker(m_out, v_out)(stream)
        return m_out, v_out

    def unpacker(self, m_out, v_out):
        """`unpack` into the given tensors as a function to call again (its table is made once)."""
        if self.config.state_bits != 8:
            raise ValueError("unpack: the states are in 32 bits")
        k = len(self.sizes)
        if len(m_out) != k or len(v_out) != k:
            raise ValueError(f"{len(m_out)} and {len(v_out)} tensors, expected {k}")
        table = (eaga.AdamwTensor * k)()
        ctypes.memmove(table, self._table, ctypes.sizeof(table))
        for i, (a, b, n) in enumerate(zip(m_out, v_out, self.sizes)):
            for t, name in ((a, "m_out"), (b, "v_out")):
                if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous() or t.device != self.device:
                    raise ValueError(f"{name}[{i}]: {n} contiguous fp32 elements on {self.device} expected")
            table[i].p, table[i].master = a.data_ptr(), b.data_ptr()
        held = (list(m_out), list(v_out), self)

        def run(stream=None, held=held):
            if torch.cuda.current_device() != self.device.index:     # the call has no tensor of its own to tell by
                raise ValueError(f"unpack: on {self.device}, but the current device is cuda:{torch.cuda.current_device()}")
            eaga.adamw_unpack(table, k, stream)
        return run

    def state_dict(self) -> dict:
        """What a checkpoint needs: the states as they are held, the masters, the step."""
        clone = lambda ts: None if ts is None else [t.detach().clone() for t in ts]
        return {"bits": int(self.config.state_bits), "step": self.steps,
                **{k: clone(getattr(self, k)) for k in ("master", "m", "v", "m_scale", "v_scale")}}

    def load_state_dict(self, s: dict):
        if s["bits"] != self.config.state_bits:
            raise ValueError(f"states in {s['bits']} bits, expected {self.config.state_bits}")
        names = ("master", "m", "v", "m_scale", "v_scale")
        like = lambda ts: None if ts is None else [(t.numel(), t.dtype) for t in ts]
        for k in names:                                 # all before any is loaded
            if like(getattr(self, k)) != like(s[k]):
                raise ValueError(f"{k}: not the states of these tensors")
        for k in names:
            for a, b in zip(getattr(self, k) or (), s[k] or ()):
                a.detach().copy_(b.reshape(a.shape))
        self.state.copy_(torch.tensor([s["step"], 0], dtype=torch.int64))
