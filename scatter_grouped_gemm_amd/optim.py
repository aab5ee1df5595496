"""AdamW over many tensors in one launch, with states in fp32 or in 8 bits.

The update, the 8-bit format and its rounding are moe_adamw_step's
(include/moe.h).  The tensors' addresses go into a plan on the device once, so a
step is one kernel launch whatever their number, reads nothing back to the host
and can be captured in a HIP graph: the step count, the learning rate and the
gradient scale live on the device and are read by the kernel.
"""
from __future__ import annotations

import bisect
import ctypes

import torch

from . import _lib as L

GROUP = 128  # elements that share a scale in the 8-bit states


class AdamW:
    """AdamW with decoupled weight decay.

    params, grads    lists of contiguous tensors of equal sizes on one device,
                     16-byte aligned; params bf16 or fp32, none overlapping
                     another or a gradient; grads bf16 or fp32.  A
                     bf16 parameter is the rounding of an fp32 master that this
                     class holds; both stay where they are between steps (write
                     new gradients into the same buffers).
    weight_decay     one number, or one for each tensor
    state_bits       32, or 8: 2 bytes an element instead of 8
    seed             of the 8-bit states' rounding

    ``lr`` (fp32 [1]) and ``steps`` (int64 [1]) are device tensors and may be
    written between steps.  ``master``, ``m``, ``v`` (and ``m_scale``,
    ``v_scale``) are flat over all tensors, tensor i at ``offsets[i]``, a
    multiple of 128; ``v`` holds the codes of its root where state_bits is 8.
    ``master`` has the places of fp32 parameters too (unused zeros); give them an
    optimizer of their own where that memory counts.
    ``state_dict`` gives what a checkpoint has to keep (and the fp32 parameters,
    which are the caller's), the seed among it: a run that is taken up again rounds
    as it would have.
    """

    def __init__(self, params, grads, *, lr: float = 1e-3, betas=(0.9, 0.95), eps: float = 1e-8,
                 weight_decay=0.0, state_bits: int = 32, seed: int = 0):
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise ValueError(f"{len(params)} parameters and {len(grads)} gradients")
        if not params:
            raise ValueError("no parameters")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is 8 or 32, not {state_bits!r}")
        wd = [float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(wd) != len(params):
            raise ValueError(f"{len(params)} parameters and {len(wd)} weight decays")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0) or not ctypes.c_float(eps).value > 0.0:
            raise ValueError("betas lie in [0, 1) and eps is positive (in fp32)")
        dev = params[0].device
        code = {torch.bfloat16: L.MOE_DTYPE_BF16, torch.float32: L.MOE_DTYPE_FP32}
        for i, (p, g) in enumerate(zip(params, grads)):
            if p.dtype not in code or g.dtype not in code:
                raise ValueError(f"tensor {i}: parameters and gradients are bf16 or fp32")
            if p.shape != g.shape:
                raise ValueError(f"tensor {i}: parameter {tuple(p.shape)}, gradient {tuple(g.shape)}")
            if p.device != dev or g.device != dev:
                raise ValueError(f"tensor {i}: all tensors are on one device")
            if not p.is_contiguous() or not g.is_contiguous():
                raise ValueError(f"tensor {i}: must be contiguous")
            if p.data_ptr() % 16 or g.data_ptr() % 16:
                raise ValueError(f"tensor {i}: must be 16-byte aligned")
        held = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size(), i)
                      for i, p in enumerate(params) if p.numel())
        for (_, end, i), (start, _, j) in zip(held, held[1:]):
            if start < end:          # two updates of one element would race
                raise ValueError(f"parameters {i} and {j} share memory")
        starts = [h[0] for h in held]
        for j, g in enumerate(grads):
            lo = g.data_ptr()
            hi = lo + g.numel() * g.element_size()
            k = bisect.bisect_left(starts, hi) - 1       # the last parameter that begins before its end
            if g.numel() and k >= 0 and held[k][1] > lo and held[k] != (lo, hi, j):
                # read by one workgroup while another writes (its own parameter itself is
                # read and written by the same lanes)
                raise ValueError(f"gradient {j} and parameter {held[k][2]} share memory")
        self.params, self.grads = params, grads
        self.betas, self.eps, self.seed, self.state_bits = (float(betas[0]), float(betas[1])), float(eps), int(seed), state_bits
        self.offsets, total = [], 0
        for p in params:
            self.offsets.append(total)
            total += -(-p.numel() // GROUP) * GROUP
        low = state_bits == 8
        zeros = lambda n, dt: torch.zeros(n, dtype=dt, device=dev)  # noqa: E731
        self.m = zeros(total, torch.uint8 if low else torch.float32)
        self.v = zeros(total, torch.uint8 if low else torch.float32)
        self.m_scale = zeros(total // GROUP, torch.uint8) if low else None
        self.v_scale = zeros(total // GROUP, torch.uint8) if low else None
        self.master = zeros(total, torch.float32) if any(p.dtype is torch.bfloat16 for p in params) else None
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=dev)
        self._counter = zeros(2, torch.int64)
        self.steps = self._counter[:1]
        self.reset_master()
        tensors = []
        for i, (p, g, at) in enumerate(zip(params, grads, self.offsets)):
            bf16 = p.dtype is torch.bfloat16
            tensors.append(L.AdamwTensor(
                param=p.data_ptr(), master=self.master.data_ptr() + 4 * at if bf16 else None, grad=g.data_ptr(),
                m=self.m.data_ptr() + at * self.m.element_size(), v=self.v.data_ptr() + at * self.v.element_size(),
                m_scale=self.m_scale.data_ptr() + at // GROUP if low else None,
                v_scale=self.v_scale.data_ptr() + at // GROUP if low else None,
                numel=p.numel(), weight_decay=wd[i], param_dtype=code[p.dtype], grad_dtype=code[g.dtype],
                state_bits=state_bits))
        self._plan = L.moe_adamw_plan(tensors).to(dev)

    @torch.no_grad()
    def reset_master(self):
        """Take the masters of bf16 parameters from the parameters (after loading new ones)."""
        for p, at in zip(self.params, self.offsets):
            if p.dtype is torch.bfloat16:
                self.master[at:at + p.numel()].copy_(p.reshape(-1))

    def state_dict(self) -> dict:
        """The state's tensors (not copies): what a checkpoint has to keep."""
        names = ("master", "m", "v", "m_scale", "v_scale", "lr")
        return {"steps": self.steps, "offsets": list(self.offsets), "state_bits": self.state_bits, "seed": self.seed,
                **{n: getattr(self, n) for n in names if getattr(self, n) is not None}}

    @torch.no_grad()
    def load_state_dict(self, state: dict):
        """Take over another run's state_dict (same tensors, same state_bits) and its
        seed (this one's stays if it holds none); bf16 parameters become their
        masters' roundings.  A step captured before keeps the seed it was captured
        with: capture it again if they differ."""
        mine = self.state_dict()
        seed = state.get("seed", self.seed)
        if not isinstance(seed, int):
            raise ValueError(f"seed: want a whole number, got {seed!r}")
        state = {**state, "seed": seed}
        if state.keys() != mine.keys() or state["state_bits"] != self.state_bits or list(state["offsets"]) != self.offsets:
            raise ValueError("the state is of other tensors or another state_bits")
        for n, t in mine.items():
            if isinstance(t, torch.Tensor):
                if state[n].shape != t.shape or state[n].dtype != t.dtype:
                    raise ValueError(f"{n}: want {t.dtype} {tuple(t.shape)}, got {state[n].dtype} {tuple(state[n].shape)}")
        self.seed = seed
        for n, t in mine.items():
            if isinstance(t, torch.Tensor):
                t.copy_(state[n])
        for p, at in zip(self.params, self.offsets):
            if p.dtype is torch.bfloat16:
                p.copy_(self.master[at:at + p.numel()].view(p.shape))

    def step(self, grad_scale: torch.Tensor | None = None):
        """Update every parameter from its gradient, times grad_scale (device fp32 [1]) if given."""
        L.moe_adamw_step(self._plan, self.lr, self._counter, self.betas[0], self.betas[1], self.eps, self.seed,
                         grad_scale)
