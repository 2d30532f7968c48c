"""Rotary positions of a model's queries and keys: its frequencies, kept on the GPU, and the calls that turn rows by them.

Steps take a Rope and turn their queries and keys (pipeline.Step at the rows' original positions, packed.PackedStep and
cache.KVCache4 at given ones). Contexts longer than the trained one are reached by changing the frequencies:
  "linear"  every frequency divided by `stretch`;
  "base"    the base raised to base * stretch^(rot / (rot - 2)): the fastest pair keeps its frequency, the slowest is divided
            by `stretch`;
  "parts"   pairs that turn more than `fast` times over the trained length stay, those that turn less than `slow` times are
            divided by `stretch`, those between are blended linearly by their turns; cosines and sines times
            0.1 ln(stretch) + 1. (Some models' code blends by the pair's number instead, between the pairs that turn `fast`
            and `slow` times: their frequencies are passed as inv_freq, with the factor.)
"""
from __future__ import annotations

import math

import torch

from . import rope_table, rope_workspace_size, scfa_rope_bwd, scfa_rope_fwd, workspace


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "", stretch: float = 1.0, trained: int = 0,
                     slow: float = 1.0, fast: float = 32.0):
    """(inv_freq [rot / 2] float64 on the CPU, factor): base^(-2 i / rot), changed by `scaling` ("", "linear", "base" or
    "parts", which takes the trained length)."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rope_frequencies: {rot} channels do not make pairs")
    if scaling not in ("", "linear", "base", "parts") or not stretch >= 1.0 or not base > 0.0:
        raise ValueError(f"rope_frequencies: scaling {scaling!r}, stretch {stretch}, base {base}")
    if scaling == "base" and rot > 2:
        base = base * stretch ** (rot / (rot - 2))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))
    if scaling == "linear":
        return f / stretch, 1.0
    if scaling == "parts":
        if trained < 1 or not 0 <= slow < fast:
            raise ValueError(f"rope_frequencies: trained length {trained}, turns from {slow} to {fast}")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        return f / stretch * (1 - keep) + f * keep, 0.1 * math.log(stretch) + 1.0
    return f, 1.0


class Rope:
    """Frequencies of one model on one GPU. Stateless beyond them: one Rope serves any number of steps and streams."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "", stretch: float = 1.0,
                 trained: int = 0, slow: float = 1.0, fast: float = 32.0, inv_freq=None, factor=None, device="cuda"):
        """The first `rot` channels of each head turn; interleaved: pairs are (2 i, 2 i + 1), else (i, i + rot / 2). Or
        frequencies of one's own: inv_freq [rot / 2], radians per position, and factor (1)."""
        if inv_freq is None:
            inv_freq, f = rope_frequencies(rot, base, scaling, stretch, trained, slow, fast)
        else:
            inv_freq, f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu"), 1.0
            if rot < 0 or rot % 2 or inv_freq.shape != (rot // 2,):
                raise ValueError(f"Rope: {rot} channels to turn need half as many frequencies, got {tuple(inv_freq.shape)}")
        self.rot, self.interleaved = rot, bool(interleaved)
        self.factor = float(f if factor is None else factor)
        self.inv_freq = inv_freq
        self.table = rope_table(inv_freq, device)

    def fwd(self, q, k, pos, q_out, k_out, wq=None, wk=None, eps=1e-6, count=None, stream=None):
        """scfa_rope_fwd with these frequencies."""
        scfa_rope_fwd(q, k, pos, self.table, q_out, k_out, self.interleaved, self.factor, wq, wk, eps, count, stream)

    def bwd(self, dq, dk, pos, dq_out, dk_out, q=None, k=None, wq=None, wk=None, eps=1e-6, dwq=None, dwk=None, ws=None,
            count=None, stream=None):
        """scfa_rope_bwd with these frequencies."""
        scfa_rope_bwd(dq, dk, pos, self.table, dq_out, dk_out, self.interleaved, self.factor, q, k, wq, wk, eps, dwq, dwk, ws,
                      count, stream)

    def workspace(self, N: int, Hq: int, Hkv: int, D: int) -> torch.Tensor:
        """A workspace for bwd() with a norm."""
        return workspace(rope_workspace_size(N, Hq, Hkv, D), self.table.device)
