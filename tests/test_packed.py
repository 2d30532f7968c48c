"""Packed sequences without a GPU: the oracle against torch's autograd in 64 bits and by hand, sizes, and the refusals of
the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import packed as op


@pytest.fixture(scope="module")
def scfa():
    from sparse_causal_flash_gb300 import build
    build.build()
    import sparse_causal_flash_gb300 as s
    return s


# ---------------------------------------------------------------- the oracle
def test_mask_by_hand():
    assert op.mask(2, 4).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert op.mask(3, 2).tolist() == [[0, 0], [1, 0], [1, 1]]  # more queries than keys: the first sees nothing
    assert op.mask(2, 4, 2).tolist() == [[0, 1, 1, 0], [0, 0, 1, 1]]
    assert op.mask(2, 2, 1).tolist() == [[1, 0], [0, 1]]


@pytest.mark.parametrize("n,m,window", [(1, 1, 0), (5, 5, 0), (3, 9, 0), (7, 4, 0), (6, 11, 3), (4, 4, 1), (3, 0, 0)])
def test_oracle_against_autograd(n, m, window):
    g = torch.Generator().manual_seed(n * 100 + m)
    q, k, v, do = (torch.randn(x, 8, generator=g, dtype=torch.float64) for x in (n, m, m, n))
    for t in (q, k, v):
        t.requires_grad_(True)
    ok = torch.as_tensor(op.mask(n, m, window))
    s = torch.where(ok, 0.3 * q @ k.T, -torch.inf)
    some = ok.any(1) if m else torch.zeros(n, dtype=torch.bool)
    p = torch.softmax(torch.where(some[:, None], s, 0.0), 1) * some[:, None] if m else s
    o = p @ v
    got, lse = op.forward(q.detach().numpy(), k.detach().numpy(), v.detach().numpy(), 0.3, window)
    assert np.allclose(got, o.detach().numpy(), atol=1e-14)
    assert np.array_equal(np.isneginf(lse), ~some.numpy())
    if some.any():
        assert np.allclose(lse[some.numpy()], torch.logsumexp(s[some], 1).detach().numpy())
    if m:
        grads = torch.autograd.grad((o * do).sum(), (q, k, v))
        for a, b in zip(op.backward(*(t.detach().numpy() for t in (q, k, v, do)), 0.3, window), grads):
            assert np.allclose(a, b.numpy(), atol=1e-13)


def test_oracle_gradient_against_differences():
    g = np.random.default_rng(3)
    x = [g.standard_normal((a, 6)) for a in (4, 7, 7)]
    do = g.standard_normal((4, 6))
    grads = op.backward(*x, do, 0.4, 5)
    for i in range(3):
        u = g.standard_normal(x[i].shape)
        lo, hi = ([y + s * u if j == i else y for j, y in enumerate(x)] for s in (-1e-6, 1e-6))
        d = ((op.forward(*hi, 0.4, 5)[0] - op.forward(*lo, 0.4, 5)[0]) * do).sum() / 2e-6
        assert abs(d - (grads[i] * u).sum()) < 1e-7


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("N,M,R,Hq,Hkv,ok", [
    (0, 0, 1, 1, 1, True), (1, 1, 1, 128, 1, True), (100, 90, 7, 12, 4, True), (1 << 20, 1 << 20, 3, 8, 1, True),
    (8, 8, 0, 4, 4, False), (8, 8, 1, 4, 3, False), (8, 8, 1, 2, 4, False), (8, 8, 1, 129, 1, False), (-1, 8, 1, 4, 4, False),
    (8, -1, 1, 4, 4, False), (8, 8, 1, 4, 0, False), (2 ** 31 - 1, 8, 1, 128, 1, False)])
def test_sizes(scfa, N, M, R, Hq, Hkv, ok):
    n = scfa.packed_plan_size(N, M, R, Hq, Hkv)
    assert (n > 0) == ok and n % 256 == 0
    for back in (False, True):
        w = scfa.packed_workspace_size(back, N, M, R, Hq, Hkv, 64)
        assert (w > 0) == ok and w % 256 == 0
    assert scfa.packed_workspace_size(True, N, M, R, Hq, Hkv, 80) == 0


# ---------------------------------------------------------------- refusals
FAKE = ctypes.c_void_p(4096)


def plan_args(**kw):
    a = dict(qs=FAKE, ks=FAKE, N=8, M=8, R=2, Hq=4, Hkv=2, window=0, plan=FAKE, nb=1 << 26, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(qs=None), 1), (dict(ks=None), 1), (dict(plan=None), 1), (dict(N=-1), 1), (dict(M=-1), 1), (dict(R=0), 1),
    (dict(window=-1), 1), (dict(Hkv=0), 1), (dict(Hq=3), 1), (dict(Hq=1), 1), (dict(Hq=258), 2), (dict(nb=100), 3),
    (dict(plan=ctypes.c_void_p(4160)), 3), (dict(N=2 ** 31 - 1, Hq=256), 2)])
def test_plan_refusals(scfa, kw, code):
    assert scfa._lib.scfa_packed_plan(*plan_args(**kw)) == code


def rows(name, t=512, h=64):
    return {name: FAKE, name + "t": t, name + "h": h}


def fwd_args(**kw):
    a = dict(**rows("q"), **rows("k"), **rows("v"), plan=FAKE, pb=1 << 20, N=8, M=8, Hq=4, Hkv=2, D=64, scale=0.1, dt=0,
             **rows("o"), lse=FAKE, ws=FAKE, nb=1 << 32, flags=0, st=None)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(**rows("q"), **rows("k"), **rows("v"), **rows("o"), lse=FAKE, **rows("do"), plan=FAKE, pb=1 << 20, N=8, M=8,
             Hq=4, Hkv=2, D=64, scale=0.1, dt=0, **rows("dq"), **rows("dk"), **rows("dv"), ws=FAKE, nb=1 << 32, flags=0,
             st=None)
    a.update(kw)
    return list(a.values())


BOTH = [(dict(plan=None), 1), (dict(ws=None), 1), (dict(N=-1), 1), (dict(M=-1), 1), (dict(Hkv=0), 1), (dict(Hq=5), 1),
        (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=3e38), 1), (dict(D=96), 2),
        (dict(dt=3), 2), (dict(Hq=258), 2), (dict(N=1 << 30), 2), (dict(M=1 << 30), 2), (dict(nb=1000), 3),
        (dict(ws=ctypes.c_void_p(4160)), 3), (dict(plan=ctypes.c_void_p(4160)), 1), (dict(pb=8), 1), (dict(lse=None), 1),
        (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(qt=0), 1), (dict(kt=-512), 1),
        (dict(vh=0), 1), (dict(qh=4), 1), (dict(k=ctypes.c_void_p(4100)), 1)]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(oh=32), 1), (dict(ot=32), 1), (dict(ot=64), 1)])
def test_fwd_refusals(scfa, kw, code):
    assert scfa._lib.scfa_packed_fwd(*fwd_args(**kw)) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(do=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(dqh=32), 1), (dict(dkt=64), 1),
    (dict(dvt=12), 1), (dict(doh=0), 1), (dict(ot=0), 1)])
def test_bwd_refusals(scfa, kw, code):
    assert scfa._lib.scfa_packed_bwd(*bwd_args(**kw)) == code


def test_binding_refuses_before_any_launch(scfa):
    from sparse_causal_flash_gb300.packed import PackedStep
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        scfa.scfa_packed_plan(i, i, 4, 4, 2, 2, 0, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        scfa.scfa_packed_fwd(x, x, x, torch.zeros(256, dtype=torch.uint8), 0.1, x, torch.zeros(4, 2), torch.zeros(256))
    for kw in (dict(Hq=3, Hkv=2), dict(D=96), dict(N=0), dict(R=0), dict(dtype=torch.float32), dict(norm=True)):
        with pytest.raises(ValueError):
            PackedStep(**{**dict(N=8, R=1, Hq=4, Hkv=2, D=64), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(qs=None), 1), (dict(plan=None), 1), (dict(N=-1), 1), (dict(R=0), 1), (dict(window=-1), 1), (dict(Hkv=0), 1),
    (dict(Hq=3), 1), (dict(Hq=258), 2), (dict(nb=100), 3), (dict(plan=ctypes.c_void_p(4160)), 3), (dict(N=2 ** 31 - 1, Hq=256), 2)])
def test_self_plan_refusals(scfa, kw, code):
    a = dict(qs=FAKE, N=8, R=2, Hq=4, Hkv=2, window=0, plan=FAKE, nb=1 << 26, st=None)
    a.update(kw)
    assert scfa._lib.scfa_packed_plan_self(*a.values()) == code


def test_self_plan_binding_refuses_cpu_tensors(scfa):
    with pytest.raises(ValueError, match="CUDA"):
        scfa.scfa_packed_plan_self(torch.zeros(3, dtype=torch.int32), 4, 2, 2, 0, torch.zeros(1 << 20, dtype=torch.uint8))
