"""ZeroAdam: the page's optimizer object over the C ABI, N ranks emulated on one GPU.

Same surface as the class in "ZeRO and FSDP" -> "Implementing ZeRO's Adam from
scratch": ZeroAdam(params, lr, betas=(0.9, 0.999), eps=1e-8), step(),
zero_grad(), state_bytes().  The flat layout is the page's (numel, shard =
ceil(numel/world), zero-padded tail); the differences are GB300-first:

- the parameters become views into one flat bf16 buffer, which is where the
  kernel's all-gather writes, so there is no unflatten copy;
- each emulated rank k owns a flat bf16 gradient buffer (grads_of(k) gives
  per-parameter views of it, for that rank's backward pass to fill);
- the fp32 master weights, m and v of all ranks live in three flat buffers;
- step() is one zero_adam_step launch on the current stream (no collectives:
  the ranks are buffers in this GPU's memory).

TensorAdamW is the same surface over a list of tensors that keep their own
storage (a rank's FSDP2-style row shards, or a whole model on one card): AdamW
with decoupled weight decay, clipping by the global norm, and moments in 32 or
8 bits.

This module only allocates (through PyTorch) and marshals; the arithmetic runs
in libzeroadam.so.
"""
from __future__ import annotations

import torch

from . import (ZERO_ALL_RANKS, ZERO_MOMENT_BLOCK, adamw_tensors, check_device,
               grad_norm_workspace, pointer_array, zero_adam_step, zero_adamw_state_f32,
               zero_adamw_step, zero_grad_norm, zero_plan)


class ZeroAdam:
    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, world=1):
        self.params = list(params)
        self.lr, self.betas, self.eps, self.t = lr, betas, eps, 0
        self.world = world
        dev = self.params[0].device
        if dev.type != "cuda":
            raise ValueError("ZeroAdam keeps its state in GPU memory: give it CUDA parameters")
        self.numel = sum(p.numel() for p in self.params)
        self.plan = zero_plan(self.numel, world)
        self.shard = self.plan.shard
        padded = self.plan.padded
        # fp32 master weights of every rank's shard (the page keeps only the own
        # slice per process; here all N slices live side by side), moments at zero
        self.master = torch.zeros(padded, dtype=torch.float32, device=dev)
        self.m = torch.zeros_like(self.master)
        self.v = torch.zeros_like(self.master)
        self.flat_params = torch.empty(self.numel, dtype=torch.bfloat16, device=dev)
        self.grads = [torch.zeros(padded, dtype=torch.bfloat16, device=dev) for _ in range(world)]
        self._grad_ptrs = pointer_array(self.grads)
        off = 0
        with torch.no_grad():
            for p in self.params:
                n = p.numel()
                self.master[off:off + n] = p.detach().reshape(-1).float()
                view = self.flat_params[off:off + n].view(p.shape)
                view.copy_(p.detach())
                p.data = view
                off += n

    def grads_of(self, k):
        """Per-parameter views into emulated rank k's flat bf16 gradient buffer."""
        out, off = [], 0
        for p in self.params:
            out.append(self.grads[k][off:off + p.numel()].view(p.shape))
            off += p.numel()
        return out

    def step(self, stream=None, check=False):
        """One ZeRO-2 step of every rank: reduce-scatter + average, Adam, all-gather.

        With check=True the call waits for the device and raises ZeroError
        (ZERO_E_TIMEOUT) if a kernel gave up a bounded wait, i.e. if some element
        of the step was not updated."""
        self.t += 1
        b1, b2 = self.betas
        if any(a is not b for a, b in zip(self.grads, self._grad_ptrs.buffers)):
            self._grad_ptrs = pointer_array(self.grads)   # a gradient buffer was replaced
        zero_adam_step(self.plan, ZERO_ALL_RANKS, self._grad_ptrs, self.master, self.m, self.v,
                       self.flat_params, lr=self.lr, beta1=b1, beta2=b2, eps=self.eps, t=self.t,
                       stream=stream)
        if check:
            check_device("ZeroAdam.step")

    def zero_grad(self):
        for g in self.grads:
            g.zero_()

    def state_bytes(self):
        """fp32 master + m + v bytes one rank holds (12 x shard)."""
        return 3 * 4 * self.shard


class TensorAdamW:
    """AdamW over a list of bf16 CUDA tensors: one norm (with max_norm) and one step launch
    per 384 tensors.

    Each parameter has an fp32 master copy and fp32 moments, or with eight_bit=True
    8-bit ones (2 + 8/256 bytes a parameter instead of 8).  weight_decay is applied to
    tensors of two or more dimensions.  Gradients are bf16 or fp32 tensors of the
    parameters' sizes: those of `grads`, filled by the caller, or else each
    parameter's .grad at step()."""

    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, max_norm=None,
                 eight_bit=False, grads=None, seed=0):
        self.params = list(params)
        if not self.params or any(p.device.type != "cuda" for p in self.params):
            raise ValueError("TensorAdamW keeps its state in GPU memory: give it CUDA parameters")
        if any(p.dtype != torch.bfloat16 or not p.is_contiguous() for p in self.params):
            raise ValueError("the parameters are contiguous bf16 tensors")
        self.lr, self.betas, self.eps, self.max_norm, self.t = lr, betas, eps, max_norm, 0
        self.decay = [weight_decay if p.dim() > 1 else 0.0 for p in self.params]
        self.eight_bit, self.seed, self.grads = eight_bit, seed, grads
        dev = self.params[0].device
        like = dict(dtype=torch.uint8 if eight_bit else torch.float32, device=dev)
        self.master = [p.detach().float() for p in self.params]
        self.m = [torch.zeros(p.shape, **like) for p in self.params]
        self.v = [torch.zeros(p.shape, **like) for p in self.params]
        self.m_scale = self.v_scale = None
        if eight_bit:
            blocks = [-(-p.numel() // ZERO_MOMENT_BLOCK) for p in self.params]
            self.m_scale = [torch.zeros(b, dtype=torch.float32, device=dev) for b in blocks]
            self.v_scale = [torch.zeros(b, dtype=torch.float32, device=dev) for b in blocks]
        self.norm = torch.zeros(2, dtype=torch.float32, device=dev)  # of the last step, and its clip
        self._workspace = grad_norm_workspace(dev)
        self._list = self._at = None

    def _tensors(self):
        grads = self.grads if self.grads is not None else [p.grad for p in self.params]
        if any(g is None for g in grads):
            raise ValueError("a parameter has no gradient")
        columns = (grads, self.params, self.master, self.m, self.v, self.m_scale or (),
                   self.v_scale or ())
        at = [t.data_ptr() for c in columns for t in c] + [g.dtype for g in grads]
        if self._list is None or at != self._at:  # marshalled anew once anything has moved
            self._list = adamw_tensors(grads, self.master, self.m, self.v, params=self.params,
                                       m_scale=self.m_scale, v_scale=self.v_scale,
                                       weight_decay=self.decay)
            self._at = at
        return self._list

    def step(self, stream=None):
        """One step: the gradients' global norm and its clip (with max_norm), then AdamW."""
        tensors = self._tensors()
        self.t += 1
        scale = None
        if self.max_norm is not None:
            zero_grad_norm(tensors, self.norm, max_norm=self.max_norm, workspace=self._workspace,
                           stream=stream)
            scale = self.norm[1:]
        b1, b2 = self.betas
        zero_adamw_step(tensors, lr=self.lr, beta1=b1, beta2=b2, eps=self.eps, t=self.t,
                        grad_scale=scale, seed=self.seed + self.t, stream=stream)

    def zero_grad(self):
        for g in self.grads if self.grads is not None else [p.grad for p in self.params]:
            if g is not None:
                g.zero_()

    def moments(self):
        """(m, v) of every parameter as fp32, for a checkpoint."""
        if not self.eight_bit:
            return self.m, self.v
        out = [[torch.empty(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
               for _ in range(2)]
        # (the parameters in place of gradients, which may be None: only their sizes are used)
        codes = adamw_tensors(self.params, self.master, self.m, self.v, m_scale=self.m_scale,
                              v_scale=self.v_scale)
        zero_adamw_state_f32(codes, *out)
        return out[0], out[1]

    def state_bytes(self):
        """Bytes of master weights and moments."""
        lists = (self.master, self.m, self.v, self.m_scale or [], self.v_scale or [])
        return sum(t.numel() * t.element_size() for x in lists for t in x)
