"""One attention layer's training step on packed sequences with shared key heads, composed from C-ABI calls.

Call order only: rotary positions and norm of queries and keys, attention forward; attention backward, then the positions'
and norm's gradients, in place. Sequences of any lengths lie one after another in one row of tokens, without padding.
Nothing is read back on the host, so a step can be captured as one CUDA graph.
"""
from __future__ import annotations

import torch

from . import (packed_plan_size, packed_workspace_size, scfa_get_device_status, scfa_packed_bwd, scfa_packed_fwd,
               scfa_packed_plan_self, workspace)


class PackedStep:
    """Buffers and the launch sequence of a layer's step for N token rows in up to R sequences."""

    def __init__(self, N: int, R: int, Hq: int, Hkv: int, D: int, window: int = 0, rope=None, norm: bool = False,
                 eps: float = 1e-6, dtype=torch.bfloat16, device="cuda", plan_of=None):
        """window: keys that a query sees at most (0: all before it). rope: a Rope, whose positions the calls then take.
        norm: queries and keys pass a root-mean-square norm per head first, with weights that the calls take (needs a
        rope; Rope(0) turns nothing). plan_of: another PackedStep of the same sizes and window, another layer's, whose plan
        this one reads: a batch is planned once, by plan() of either. Each layer's step keeps its own results and workspace."""
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"PackedStep: rows are bf16 or fp16, not {dtype}")
        if norm and rope is None:
            raise ValueError("PackedStep: the norm comes with the rotary positions; Rope(0) turns nothing")
        nbytes = packed_plan_size(N, N, R, Hq, Hkv) if N >= 1 else 0
        nws = packed_workspace_size(True, N, N, R, Hq, Hkv, D) if nbytes else 0
        if not nws:
            raise ValueError(f"PackedStep: {N} tokens, {R} sequences, {Hq} query heads on {Hkv} key heads of {D} channels are "
                             "not supported")
        # with its index: "cuda" is the device that is current now, not the one that is at a later call
        self.device = dev = torch.empty(0, device=device).device
        self.N, self.R, self.Hq, self.Hkv, self.D, self.window = N, R, Hq, Hkv, D, window
        self.rope, self.norm, self.eps, self.dtype = rope, bool(norm), float(eps), dtype
        row = dict(dtype=dtype, device=dev)
        self.o = torch.zeros((N, Hq, D), **row)
        self.lse = torch.zeros((N, Hq), dtype=torch.float32, device=dev)
        # the gradients of a fused projection's output: queries, keys, values
        self.dqkv = torch.zeros((N, Hq + 2 * Hkv, D), **row)
        self.dq, self.dk, self.dv = self.dqkv[:, :Hq], self.dqkv[:, Hq:Hq + Hkv], self.dqkv[:, Hq + Hkv:]
        self.q_r = self.k_r = self.dwq = self.dwk = self.ws_rope = None
        if rope is not None:
            if rope.rot > D:
                raise ValueError(f"PackedStep: {rope.rot} channels to turn, a head has {D}")
            self.q_r, self.k_r = torch.zeros((N, Hq, D), **row), torch.zeros((N, Hkv, D), **row)
        if norm:
            self.dwq, self.dwk = (torch.zeros(D, dtype=torch.float32, device=dev) for _ in range(2))
            self.ws_rope = rope.workspace(N, Hq, Hkv, D)
        if plan_of is not None:
            mine = (N, R, Hq, Hkv, window, dev)
            theirs = (plan_of.N, plan_of.R, plan_of.Hq, plan_of.Hkv, plan_of.window, plan_of.device)
            if mine != theirs:
                raise ValueError(f"PackedStep: a plan of (tokens, sequences, query heads, key heads, window, device) {theirs} "
                                 f"is none of {mine}")
        self.plan_buf = workspace(nbytes, dev) if plan_of is None else plan_of.plan_buf
        self.count = self.plan_buf[4:8].view(torch.int32)  # tokens of the batch, by the plan; 0 if it is refused
        self.ws = workspace(nws, dev)
        self.ws[:4].zero_()  # the status word: nothing has run yet
        if plan_of is None:
            self.plan_buf[:256].zero_()  # no plan, whatever the memory held: steps before plan() are refused

    def plan(self, starts, stream=None):
        """The batch's sequences: starts [R + 1] int32, from 0; tokens starts[r] .. starts[r + 1] are sequence r (a shorter
        batch repeats its end). To be called before the first step, which is refused otherwise, and whenever `starts`
        changes; one plan serves any number of layers' steps (plan_of). Starts that fall, leave the N rows or do not begin
        at 0 show in status(), and steps then write no row (dwq and dwk, sums over no rows, become zero)."""
        if starts.numel() != self.R + 1:
            raise ValueError(f"PackedStep.plan: {self.R + 1} starts expected, got {starts.numel()}")
        scfa_packed_plan_self(starts, self.N, self.Hq, self.Hkv, self.window, self.plan_buf, stream)

    def _args(self, pos, wq, wk):
        if (pos is None) != (self.rope is None):
            raise ValueError("PackedStep: positions come with a rope, and only with one")
        if (wq is None) == self.norm or (wk is None) == self.norm:
            raise ValueError("PackedStep: weights come with the norm, and only with it")

    def forward(self, q, k, v, scale, pos=None, wq=None, wk=None, stream=None):
        """o [N, Hq, D], lse [N, Hq] (this object's buffers) of q [N, Hq, D], k, v [N, Hkv, D], which may be views of a fused
        projection; pos [N] int32 with a rope, wq, wk [D] fp32 with the norm. Rows behind the last sequence stay as they
        were."""
        self._args(pos, wq, wk)
        if self.rope is not None:
            self.rope.fwd(q, k, pos, self.q_r, self.k_r, wq, wk, self.eps, self.count, stream)
            q, k = self.q_r, self.k_r
        scfa_packed_fwd(q, k, v, self.plan_buf, scale, self.o, self.lse, self.ws, 0, stream)
        return self.o, self.lse

    def backward(self, q, k, v, do, scale, pos=None, wq=None, wk=None, stream=None):
        """Gradients of the last forward (same arguments) for do [N, Hq, D], into dq, dk, dv (views of dqkv) and with the
        norm dwq, dwk. Rows behind the last sequence stay as they were."""
        self._args(pos, wq, wk)
        qa, ka = (q, k) if self.rope is None else (self.q_r, self.k_r)
        scfa_packed_bwd(qa, ka, v, self.o, self.lse, do, self.plan_buf, scale, self.dq, self.dk, self.dv, self.ws, 0, stream)
        if self.rope is not None:
            kw = dict(q=q, k=k, wq=wq, wk=wk, eps=self.eps, dwq=self.dwq, dwk=self.dwk, ws=self.ws_rope) if self.norm else {}
            self.rope.bwd(self.dq, self.dk, pos, self.dq, self.dk, count=self.count, stream=stream, **kw)
        return self.dqkv

    def run(self, q, k, v, do, scale, pos=None, wq=None, wk=None, stream=None):
        """Forward and backward."""
        self.forward(q, k, v, scale, pos, wq, wk, stream)
        self.backward(q, k, v, do, scale, pos, wq, wk, stream)
        return self

    def capture(self, q, k, v, do, scale, pos=None, wq=None, wk=None):
        """run() on these tensors as a CUDA graph, which must stay alive and in place, as must this object; plan() is not
        part of it and may be called between replays. Nothing is run."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.device(self.device), torch.cuda.graph(g):
            self.run(q, k, v, do, scale, pos, wq, wk)
        return g

    def status(self) -> int:
        """0, or the first error of the plan, then of the last call (synchronises)."""
        with torch.cuda.device(self.device):
            return scfa_get_device_status(self.plan_buf) or scfa_get_device_status(self.ws)
