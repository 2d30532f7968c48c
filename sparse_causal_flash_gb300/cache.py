"""Serving steps over the paged 4-bit key/value cache, composed from C-ABI calls.

KVCache4 owns the pages, block tables and workspaces of a fixed number of
request rows; step() plans the new tokens' slots on the GPU, quantises their
keys and values into the pages and attends over what each token sees. Nothing
is read back on the host, so a step can be captured as one CUDA graph and
replayed for as long as its inputs keep their shapes. Tokens whose keys a keep
mask drops take no room: the cache holds the kept ones. The mask is one for all
heads; QK-sparse masks that differ from head to head and hash-sparse attention
have no serving form here.
"""
from __future__ import annotations

import torch

from . import (_rows4, cache4_attn_workspace_size, cache4_page_bytes, cache4_plan_workspace_size, scfa_cache4_append,
               scfa_cache4_attn, scfa_cache4_plan, scfa_cache4_read, scfa_get_device_status, workspace)

# a scale is a normal fp32 number whose product with log2(e) is one too
_SCALES = torch.finfo(torch.float32).tiny, float.fromhex("0x1.62e42ep+127")


class KVCache4:
    """Pages, tables and the launch sequence of serving steps for R request rows."""

    def __init__(self, R: int, n_pages: int, Hq: int, Hkv: int, D: int, max_len: int, max_tokens: int,
                 page_size: int = 64, dtype=torch.bfloat16, device="cuda", rope=None, wq=None, wk=None, eps: float = 1e-6):
        """R request rows share n_pages pages of page_size tokens; a request
        caches at most max_len tokens (rounded up to whole pages), a step
        brings at most max_tokens new ones over all requests. rope: a rope.Rope;
        steps then take their tokens' positions and turn queries and keys by
        them before all else, with wq and wk [D] fp32 behind a root-mean-square
        norm of each head."""
        nbytes = cache4_page_bytes(page_size, D)
        if nbytes == 0:
            raise ValueError(f"KVCache4: head dimension {D} or page size {page_size} is not supported")
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"KVCache4: rows are bf16 or fp16, not {dtype}")
        if min(R, n_pages, max_len, max_tokens) < 1:
            raise ValueError(f"KVCache4: {R} requests, {n_pages} pages, {max_len} tokens a request and {max_tokens} a "
                             "step must be positive")
        if Hkv < 1 or Hq < Hkv or Hq % Hkv != 0:
            raise ValueError(f"KVCache4: {Hq} query heads are no multiple of {Hkv} key heads")
        # with its index: "cuda" is the device that is current now, not the one that is at a later call
        self.device = dev = torch.empty(0, device=device).device
        self.dtype = dtype
        self.R, self.n_pages, self.Hq, self.Hkv, self.D, self.page_size = R, n_pages, Hq, Hkv, D, page_size
        self.max_len, self.max_tokens = max_len, max_tokens
        max_pages = -(-max_len // page_size)
        i32 = dict(dtype=torch.int32, device=dev)
        self.cache = torch.zeros((n_pages, Hkv, nbytes), dtype=torch.uint8, device=dev)
        self.len = torch.zeros(R, **i32)
        self.table = torch.full((R, max_pages), -1, **i32)
        # a stack: page 0 on top
        self.free = torch.arange(n_pages - 1, -1, -1, **i32)
        self.n_free = torch.full((1,), n_pages, **i32)
        self.q_start = torch.zeros(R + 1, **i32)
        self.slot = torch.empty(max_tokens, **i32)
        self.vis = torch.empty(max_tokens, **i32)
        self.o = torch.zeros((max_tokens, Hq, D), dtype=dtype, device=dev)
        self.lse = torch.zeros((max_tokens, Hq), dtype=torch.float32, device=dev)
        self.rope, self.wq, self.wk, self.eps = rope, wq, wk, float(eps)
        self.q_r = self.k_r = None
        if rope is None and (wq is not None or wk is not None):
            raise ValueError("KVCache4: the norm comes with the rotary positions; Rope(0) turns nothing")
        if rope is not None:
            if rope.rot > D or (wq is None) != (wk is None):
                raise ValueError(f"KVCache4: {rope.rot} of {D} channels to turn, or a weight without the other")
            self.q_r = torch.empty((max_tokens, Hq, D), dtype=dtype, device=dev)
            self.k_r = torch.empty((max_tokens, Hkv, D), dtype=dtype, device=dev)
        self.ws_plan = workspace(cache4_plan_workspace_size(max_tokens, R), dev)
        self.ws_attn = workspace(cache4_attn_workspace_size(max_tokens, R, Hq, Hkv, D), dev)
        for ws in (self.ws_plan, self.ws_attn):
            ws[:4].zero_()  # the status word: no step has run yet

    def step(self, q, k, v, new_len, scale, keep=None, stream=None, pos=None):
        """One serving step: new_len [R] int32 new tokens of each request, packed
        request by request in q [N, Hq, D], k, v [N, Hkv, D] (N from 1 to
        max_tokens; the sum of new_len may be smaller), keep [N] uint8 or
        None. Returns views of o [N, Hq, D] and lse [N, Hq], which the next
        step overwrites and whose rows from the sum of new_len on are left as
        they were. A step that does not fit (status()) caches nothing and
        computes nothing. Steps follow one another on one stream, or the
        caller orders them. pos [N] int32, with a rope and only with one: the
        tokens' positions in their texts (dropped tokens count)."""
        N = q.shape[0]
        if N > self.max_tokens:
            raise ValueError(f"KVCache4.step: {N} token rows, room for {self.max_tokens}")
        # all of it before the plan runs: a step that raises must leave the cache as it was
        for key, t, H in (("q", q, self.Hq), ("k", k, self.Hkv), ("v", v, self.Hkv)):
            st, sh = _rows4("KVCache4.step", key, t, N, H, self.D, self.dtype, self.len.get_device())
            if (st | sh) & 7 or t.data_ptr() & 15:
                raise ValueError(f"KVCache4.step: {key} needs strides that are multiples of 8 and a 16-byte aligned "
                                 f"start, got {t.stride()} at {t.data_ptr():#x}")
        if not _SCALES[0] <= scale <= _SCALES[1]:
            raise ValueError(f"KVCache4.step: scale {scale} is not a positive fp32 number of at most {_SCALES[1]:.7g}")
        if (pos is None) != (self.rope is None):
            raise ValueError("KVCache4.step: positions come with a rope, and only with one")
        if self.rope is not None:
            qr, kr = self.q_r[:N], self.k_r[:N]
            self.rope.fwd(q, k, pos, qr, kr, self.wq, self.wk, self.eps, stream=stream)
            q, k = qr, kr
        slot, vis, o, lse = self.slot[:N], self.vis[:N], self.o[:N], self.lse[:N]
        scfa_cache4_plan(self.len, new_len, keep, self.free, self.n_free, self.table, self.page_size, self.n_pages,
                         self.len, self.n_free, self.q_start, slot, vis, self.ws_plan, stream)
        scfa_cache4_append(k, v, slot, self.cache, self.page_size, stream)
        scfa_cache4_attn(q, self.cache, self.page_size, self.table, self.q_start, vis, scale, o, lse, self.ws_attn, 0,
                         stream)
        return o, lse

    def capture(self, q, k, v, new_len, scale, keep=None, pos=None):
        """The step on these input tensors as a CUDA graph; each replay() is
        one more step. They and this object must stay alive and in place; with
        a rope the caller moves pos on between replays.
        Nothing is run: the cache is as before."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.device(self.device), torch.cuda.graph(g):
            self.step(q, k, v, new_len, scale, keep, pos=pos)
        return g

    def rows(self, request: int):
        """(k, v) [tokens, Hkv, D]: the values the cache holds of a request.
        Reads its length back; like release() and status() on the current
        stream, which must be behind the steps."""
        n = int(self.len[request])
        shape = (max(n, 1), self.Hkv, self.D)
        k = torch.empty(shape, dtype=self.dtype, device=self.device)
        v = torch.empty(shape, dtype=self.dtype, device=self.device)
        t = torch.arange(max(n, 1), dtype=torch.int32, device=self.device)
        slot = self.table[request, t // self.page_size] * self.page_size + t % self.page_size
        scfa_cache4_read(self.cache, self.page_size, slot, k, v)
        return k[:n], v[:n]

    def release(self, request: int):
        """Give a request's pages back (reads its length back); its row is free for another."""
        n = -(-int(self.len[request]) // self.page_size)
        have = int(self.n_free)
        self.free[have:have + n] = self.table[request, :n]
        self.n_free += n
        self.len[request] = 0

    def status(self) -> int:
        """Status of the last step that was launched (0 before the first): 0, or the first error of its plan, then of
        its attention (synchronises). Each step, a replayed one too, replaces the status of the one before."""
        with torch.cuda.device(self.device):
            return scfa_get_device_status(self.ws_plan) or scfa_get_device_status(self.ws_attn)
