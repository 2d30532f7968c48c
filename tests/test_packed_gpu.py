"""Attention over packed sequences with shared key heads on the GPU against the float64 oracle, head by head.

Bounds, u = finfo.eps / 2 of the rows' type (2^-8 bf16, 2^-11 fp16), sums of D or n products in fp32 with at most 2^-23 of
the magnitudes' sum per addition (tensor cores may cut instead of round):
- a score: d = (D 2^-23) scale sum|q k|, and 2^-22 of itself and of its row's largest for the products with scale log2(e);
  a weight P then is off by e_p = 2 d + 2^-20 of itself (the exponential is within 2^-22).
- o: the weights' rounding u once for their product with V, e_p for each and for their sum, the sums n 2^-23, then the
  output's own rounding u.
- lse: d + 2^-20 + 2^-22 |lse|.
- gradients take o and lse as they are stored: |lse| 2^-22 more in e_p (fp32), and delta = rowsum(dO o) is off by
  u sum|dO o|. dP and delta are sums of D products. dS = P (dP - delta) is rounded once (u). Then dq, dk, dv are sums like o.
Below the normal numbers of fp16 a rounding moves by 2^-25: for P and dS that is an absolute error of each term."""
import numpy as np
import pytest
import torch

from oracle import packed as op

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def scfa():
    import sparse_causal_flash_gb300 as s
    s.load()
    return s


def dbl(t):
    return t.detach().double().cpu().numpy()


def rand(seed, shape, dt=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dt).cuda()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def unit(dt):
    return torch.finfo(dt).eps / 2


def half_step(x, dt):
    f = torch.finfo(dt)
    return np.maximum(np.abs(x) * f.eps / 2, f.tiny * f.eps / 2) * (1 + 2.0 ** -8)


def tiny(dt):
    return 2.0 ** -25 if dt == HF else 0.0


def parts(q, k, scale, window, lse_given):
    """(P, lse, relative error of each weight [n, m])"""
    p, lse = op.weights(q, k, scale, window)
    n, m = p.shape
    D = q.shape[1]
    mag = scale * (np.abs(q) @ np.abs(k).T)
    d = D * 2.0 ** -23 * mag + 2.0 ** -22 * mag
    seen = op.mask(n, m, window)
    top = np.where(seen, d, 0.0).max(1, keepdims=True, initial=0.0)
    e = d + top + 2.0 ** -20
    if lse_given:
        e = d + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse))[:, None]
    return p, lse, e, top[:, 0]


def check(name, got, ref, bound):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    assert np.all(err <= bound), f"{name}: {float((err / np.maximum(bound, 1e-300)).max()):.2f} of the bound"


def check_head_fwd(o, lse, q, k, v, scale, window, dt):
    ref, ref_l = op.forward(q, k, v, scale, window)
    p, _, e, top = parts(q, k, scale, window, False)
    n = k.shape[0]
    size = (p * (unit(dt) + 2 * e + n * 2.0 ** -23)) @ np.abs(v) + tiny(dt) * n * np.abs(v).max(0, initial=0.0)
    check("o", o, ref, size * 1.01 + half_step(ref, dt))
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_l))
    ok = ~np.isneginf(ref_l)
    assert np.all(np.abs(lse - np.where(ok, ref_l, 0))[ok] <= (top + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_l))[ok])
    assert not o[~ok].any()


def grad_bounds(q, k, v, do, o, scale, window, dt):
    """Reference gradients of one query head and what they may be off by, before the outputs' rounding (dk, dv are summed
    over a key head's query heads first)."""
    p, _, e, _ = parts(q, k, scale, window, True)
    n, m = p.shape
    D = q.shape[1]
    u = unit(dt)
    dp = do @ v.T
    delta = (p * dp).sum(1, keepdims=True)
    ds = p * (dp - delta)
    e_dp = D * 2.0 ** -23 * (np.abs(do) @ np.abs(v).T)
    e_delta = ((u + D * 2.0 ** -23) * np.abs(do) * np.abs(o)).sum(1, keepdims=True) + \
        (np.abs(do) @ np.abs(v).T * p * (u + 2 * e)).sum(1, keepdims=True)  # o is the forward's
    e_ds = u * np.abs(ds) + e * np.abs(ds) + p * (e_dp + e_delta) + tiny(dt) * (p > 0)
    e_p = p * (u + e) + tiny(dt) * (p > 0)
    acc_k, acc_q = m * 2.0 ** -23, n * 2.0 ** -23
    dq = scale * (ds @ k), scale * ((e_ds + acc_k * np.abs(ds)) @ np.abs(k))
    dk = scale * (ds.T @ q), scale * ((e_ds + acc_q * np.abs(ds)).T @ np.abs(q))
    dv = p.T @ do, (e_p + acc_q * p).T @ np.abs(do)
    return dq, dk, dv


class Problem:
    def __init__(self, scfa, lens, Hq, Hkv, D, dt=BF, window=0, pad=0, seed=0, fused=False, q_scale=1.0, starts=None, junk=None):
        n, m = [a for a, _ in lens], [b for _, b in lens]
        q0, k0 = starts or (0, 0)
        self.qs, self.ks = np.concatenate([[q0], q0 + np.cumsum(n)]), np.concatenate([[k0], k0 + np.cumsum(m)])
        self.N, self.M = int(self.qs[-1]) + pad, int(self.ks[-1]) + pad
        self.Hq, self.Hkv, self.D, self.dt, self.window, self.scfa = Hq, Hkv, D, dt, window, scfa
        self.scale = D ** -0.5
        N, M = self.N, self.M
        if fused and N == M:
            x = rand(seed, (N, Hq + 2 * Hkv, D), dt)
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            self.q.mul_(q_scale)
        else:  # heads outermost
            self.q = rand(seed, (Hq, N, D), dt, q_scale).transpose(0, 1)
            self.k, self.v = (rand(seed + i, (Hkv, M, D), dt).transpose(0, 1) for i in (1, 2))
        self.do = rand(seed + 3, (N, Hq, D), dt)
        if junk is not None:  # rows of nobody
            for t, s in ((self.q, self.qs), (self.do, self.qs), (self.k, self.ks), (self.v, self.ks)):
                t[:int(s[0])] = junk
                t[int(s[-1]):] = junk
        new = dict(dtype=dt, device="cuda")
        self.o, self.lse = torch.full((N, Hq, D), 5.0, **new), torch.full((N, Hq), 5.0, device="cuda")
        self.dq, self.dk, self.dv = (torch.full((a, h, D), 5.0, **new) for a, h in ((N, Hq), (M, Hkv), (M, Hkv)))
        self.plan = scfa.workspace(scfa.packed_plan_size(N, M, len(lens), Hq, Hkv))
        self.ws = scfa.workspace(scfa.packed_workspace_size(True, N, M, len(lens), Hq, Hkv, D))
        self.ws.random_(0, 256)  # whatever was there
        self.plan.random_(0, 256)
        scfa.scfa_packed_plan(i32(self.qs), i32(self.ks), N, M, Hq, Hkv, window, self.plan)

    def forward(self, **kw):
        self.scfa.scfa_packed_fwd(self.q, self.k, self.v, self.plan, self.scale, self.o, self.lse, self.ws, **kw)

    def backward(self, **kw):
        self.scfa.scfa_packed_bwd(self.q, self.k, self.v, self.o, self.lse, self.do, self.plan, self.scale, self.dq, self.dk,
                                  self.dv, self.ws, **kw)

    def status(self):
        return self.scfa.scfa_get_device_status(self.plan) or self.scfa.scfa_get_device_status(self.ws)

    def seqs(self, only=None):
        for r in range(len(self.qs) - 1) if only is None else only:
            yield slice(int(self.qs[r]), int(self.qs[r + 1])), slice(int(self.ks[r]), int(self.ks[r + 1]))

    def check_forward(self, only=None, heads=None):
        G = self.Hq // self.Hkv
        for a, b in self.seqs(only):
            for h in range(self.Hq) if heads is None else heads:
                check_head_fwd(dbl(self.o[a, h]), dbl(self.lse[a, h]), dbl(self.q[a, h]), dbl(self.k[b, h // G]),
                               dbl(self.v[b, h // G]), self.scale, self.window, self.dt)

    def check_backward(self, only=None, key_heads=None):
        G = self.Hq // self.Hkv
        for a, b in self.seqs(only):
            for kh in range(self.Hkv) if key_heads is None else key_heads:
                k, v = dbl(self.k[b, kh]), dbl(self.v[b, kh])
                sums = [np.zeros_like(k) for _ in range(4)]
                for h in range(kh * G, kh * G + G):
                    dq, dk, dv = grad_bounds(dbl(self.q[a, h]), k, v, dbl(self.do[a, h]), dbl(self.o[a, h]), self.scale,
                                             self.window, self.dt)
                    check("dq", dbl(self.dq[a, h]), dq[0], dq[1] * 1.01 + half_step(dq[0], self.dt))
                    for s, x in zip(sums, (*dk, *dv)):
                        s += x
                check("dk", dbl(self.dk[b, kh]), sums[0], sums[1] * 1.01 + half_step(sums[0], self.dt))
                check("dv", dbl(self.dv[b, kh]), sums[2], sums[3] * 1.01 + half_step(sums[2], self.dt))

    def check_untouched(self):
        for t, s in ((self.o, self.qs), (self.lse, self.qs), (self.dq, self.qs), (self.dk, self.ks), (self.dv, self.ks)):
            assert bool((t[:int(s[0])] == 5).all()) and bool((t[int(s[-1]):] == 5).all())

    def all(self):
        self.forward()
        self.backward()
        assert self.status() == 0
        self.check_forward()
        self.check_backward()
        self.check_untouched()


def same(lens):
    return [(n, n) for n in lens]


# (lens, Hq, Hkv, D, window)
CASES = [
    (same([1]), 1, 1, 64, 0), (same([1, 1, 1]), 4, 2, 128, 0), (same([2, 0, 5]), 3, 3, 64, 0), (same([127, 128, 129]), 2, 2, 64, 0),
    (same([256, 255, 257]), 2, 1, 128, 0), (same([15, 16, 17, 31, 33, 0, 0, 64]), 6, 2, 128, 0), (same([400]), 8, 1, 64, 0),
    (same([300, 41]), 5, 1, 128, 0), (same([100, 7]), 12, 1, 64, 0), (same([43, 21]), 48, 1, 64, 0), (same([5, 3]), 128, 1, 128, 0),
    (same([9]), 100, 2, 64, 0), (same([60]), 65, 1, 64, 0), ([(3, 700), (1, 130), (17, 17)], 4, 1, 128, 0),
    ([(1, 1500)], 8, 2, 64, 0), ([(1, 5), (1, 0), (0, 9), (4, 4)], 4, 4, 64, 0), ([(200, 90), (7, 1)], 3, 1, 128, 0),
    ([(130, 1)], 1, 1, 64, 0), (same([300, 200]), 4, 2, 64, 1), (same([300, 200]), 4, 2, 128, 37), (same([500]), 3, 1, 64, 128),
    (same([500]), 2, 2, 128, 200), ([(100, 600), (300, 100)], 6, 2, 64, 129), (same([700]), 1, 1, 128, 100000),
    (same([50, 60]), 4, 1, 64, 2 ** 31 - 1), (same([640]), 7, 7, 128, 0)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("lens,Hq,Hkv,D,window", CASES)
def test_against_the_oracle(scfa, lens, Hq, Hkv, D, window, dt):
    Problem(scfa, lens, Hq, Hkv, D, dt, window, pad=3, seed=len(lens) + Hq, fused=Hq % 2 == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3e4])
def test_rows_of_nobody_stay_out_and_stay(scfa, D, junk):
    """Rows before the first and behind the last sequence: whatever they hold reaches no result, and theirs are not
    written."""
    Problem(scfa, same([70, 13, 200]), 6, 2, D, BF, pad=90, starts=(33, 20), junk=junk, seed=4).all()


@pytest.mark.parametrize("D", [64, 128])
def test_what_is_not_finite_stays_in_its_sequence(scfa, D):
    p = Problem(scfa, same([90, 150, 33, 140]), 6, 2, D, seed=5)
    a, b = slice(90, 240), slice(240, 273)
    p.q[100, 1, 5] = float("nan")
    p.k[150, 0, 3] = float("inf")
    p.v[239, 1, 0] = float("nan")
    p.do[245, 2, 7] = float("-inf")
    p.forward()
    p.backward()
    assert p.status() == 0
    p.check_forward([0, 3])
    p.check_backward([0, 3])
    o, lse = p.o.float(), p.lse
    assert not torch.isfinite(o[100, 1]).any() and not torch.isfinite(lse[100, 1])  # a query row: its own o and lse
    assert torch.isfinite(o[100, 0]).all() and torch.isfinite(o[99, 1]).all()
    assert torch.isnan(o[239, 3:, 0]).all()  # the value's channel in the heads that read it
    p.check_forward([2])
    assert torch.isfinite(p.dq[a].float()).any() and not torch.isfinite(p.dv[b, 0].float()).all()
    # head 1 of the third sequence has another key head's dO
    assert torch.isfinite(p.dv[b, 1].float()).all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("scale_up", [300.0, 30000.0])
def test_scores_far_from_zero(scfa, dt, scale_up):
    """Rows of scores up to 10^5 and more: the largest keeps its weight (a row that sees equal keys averages them)."""
    n, D = 150, 64
    p = Problem(scfa, same([n]), 2, 1, D, dt, seed=6)
    p.q.fill_(1.0)
    p.k.copy_(torch.sign(rand(1, (n, 1, D), dt)))
    p.k[7], p.k[3] = 1.0, 1.0
    p.q.mul_(scale_up / 8)
    p.forward()
    assert p.status() == 0
    o, v = dbl(p.o), dbl(p.v)
    for t in range(10, n):  # keys 3 and 7 have the one largest score, the others lie thousands below
        ref = (v[3, 0] + v[7, 0]) / 2
        assert np.all(np.abs(o[t] - ref) <= half_step(ref, dt) + unit(dt) * (np.abs(v[3, 0]) + np.abs(v[7, 0])))


@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([(3, 9000)], 4, 1, 128), ([(1, 20000), (2, 15000)], 2, 1, 64), ([(40, 6000), (9, 300)], 8, 2, 64), (same([3300]), 2, 1, 128),
    (same([2900]), 1, 1, 64), ([(100, 12000)], 16, 2, 128)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_work_that_is_cut_over_ctas(scfa, lens, Hq, Hkv, D, dt):
    """Few rows over a long axis: their work is cut, left in parts and joined; equal bits on every run."""
    p = Problem(scfa, lens, Hq, Hkv, D, dt, seed=7)
    p.all()
    first = [t.clone() for t in (p.o, p.lse, p.dq, p.dk, p.dv)]
    for _ in range(3):
        p.ws.random_(0, 256)
        p.forward()
        p.backward()
        assert p.status() == 0
        assert all(torch.equal(a, b) for a, b in zip(first, (p.o, p.lse, p.dq, p.dk, p.dv)))


@pytest.mark.parametrize("window", [310, 2 ** 31 - 1])
def test_a_window_wider_than_the_keys_hides_none(scfa, window):
    """Also where the first queries stand before the first key."""
    lens = [(10, 5), (300, 290), (7, 7)]
    p, r = (Problem(scfa, lens, 4, 2, 64, window=w, seed=12) for w in (window, 0))
    for x in (p, r):
        x.forward()
        x.backward()
        assert x.status() == 0
    r.check_forward()
    assert all(torch.equal(getattr(p, key), getattr(r, key)) for key in ("o", "lse", "dq", "dk", "dv"))


@pytest.mark.parametrize("lens", [[(5, 384)], [(5, 385)], [(384, 384)], [(385, 380)], [(1, 100), (2, 284)], [(200, 2000)]])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1)])
def test_on_either_side_of_what_is_never_cut(scfa, lens, Hq, Hkv):
    """Calls on at most three tiles of keys (backward: and of queries) have no join behind them."""
    Problem(scfa, lens, Hq, Hkv, 64, seed=13).all()


def test_many_sequences(scfa):
    """More sequences than the plan has threads, most of them short or empty."""
    g = np.random.default_rng(0)
    lens = [(int(n), int(n) + int(m)) for n, m in zip(g.integers(0, 9, 2500), g.integers(0, 5, 2500))]
    p = Problem(scfa, lens, 4, 2, 64, seed=8)
    p.forward()
    p.backward()
    assert p.status() == 0
    only = [0, 1, 1023, 1024, 1025, 2048, 2498, 2499] + list(range(300, 340))
    p.check_forward(only)
    p.check_backward(only)


def test_results_are_the_same_bits_each_time(scfa):
    p = Problem(scfa, same([1000, 37, 512]), 6, 2, 64, HF, seed=9)
    p.forward()
    p.backward()
    first = [t.clone() for t in (p.o, p.lse, p.dq, p.dk, p.dv)]
    for _ in range(20):
        p.forward()
        p.backward()
        assert all(torch.equal(a, b) for a, b in zip(first, (p.o, p.lse, p.dq, p.dk, p.dv)))


def test_a_group_is_its_heads_with_copies_of_their_keys(scfa):
    """Shared key heads against as many key heads as query heads: o bit by bit, dk and dv summed."""
    lens, D = same([200, 61]), 64
    p = Problem(scfa, lens, 4, 2, D, seed=10)
    p.forward()
    p.backward()
    r = Problem(scfa, lens, 4, 4, D, seed=10)
    r.q.copy_(p.q), r.do.copy_(p.do)
    r.k.copy_(p.k.repeat_interleave(2, 1)), r.v.copy_(p.v.repeat_interleave(2, 1))
    r.forward()
    r.backward()
    assert p.status() == 0 and r.status() == 0
    p.check_forward()
    r.check_forward()
    p.check_backward()
    r.check_backward()


# ---------------------------------------------------------------- plans, workspaces, streams, graphs
@pytest.mark.parametrize("qs,ks", [([0, 5, 4], [0, 5, 5]), ([0, 5, 11], [0, 5, 5]), ([-1, 5, 6], [0, 5, 5]), ([0, 5, 6], [0, 9, 5]),
                                   ([0, 5, 6], [0, 5, 11]), ([0, 5, 6], [-3, 0, 0]), ([0, 2 ** 31 - 1, 2 ** 31 - 1], [0, 5, 5])])
def test_bad_starts_compute_nothing(scfa, qs, ks):
    p = Problem(scfa, same([5, 5]), 2, 1, 64)
    assert (p.N, p.M) == (10, 10)
    scfa.scfa_packed_plan(i32(qs), i32(ks), 10, 10, 2, 1, 0, p.plan)
    assert scfa.scfa_get_device_status(p.plan) == 1
    p.forward()
    assert scfa.scfa_get_device_status(p.ws) == 1
    p.backward()
    assert scfa.scfa_get_device_status(p.ws) == 1
    assert all(bool((t == 5).all()) for t in (p.o, p.lse, p.dq, p.dk, p.dv))
    scfa.scfa_packed_plan(i32(p.qs), i32(p.ks), 10, 10, 2, 1, 0, p.plan)  # and a good plan works again
    p.all()


def test_a_plan_for_other_tensors_is_refused(scfa):
    p = Problem(scfa, same([5, 5]), 2, 1, 64)
    r = Problem(scfa, same([5, 6]), 2, 1, 64)
    h = Problem(scfa, same([5, 5]), 2, 2, 64)
    for plan in (r.plan, h.plan, torch.zeros_like(p.plan), p.plan[:256]):
        scfa.scfa_packed_fwd(p.q, p.k, p.v, plan, p.scale, p.o, p.lse, p.ws)
        assert scfa.scfa_get_device_status(p.ws) == 1
        scfa.scfa_packed_bwd(p.q, p.k, p.v, p.o, p.lse, p.do, plan, p.scale, p.dq, p.dk, p.dv, p.ws)
        assert scfa.scfa_get_device_status(p.ws) == 1
    assert all(bool((t == 5).all()) for t in (p.o, p.lse, p.dq, p.dk, p.dv))
    # a workspace of fewer sequences has no room for the rows' statistics
    many = Problem(scfa, same([1] * 64), 2, 1, 64)
    many.forward()
    small = scfa.workspace(scfa.packed_workspace_size(True, many.N, many.M, 1, 2, 1, 64))
    if small.numel() < many.ws.numel():
        scfa.scfa_packed_bwd(many.q, many.k, many.v, many.o, many.lse, many.do, many.plan, many.scale, many.dq, many.dk,
                             many.dv, small)
        assert scfa.scfa_get_device_status(small) == 3
    p.all()


def test_empty_batches(scfa):
    for lens, pad in ((same([0, 0]), 0), (same([0]), 4), ([(0, 6)], 0), ([(6, 0)], 0)):
        p = Problem(scfa, lens, 2, 1, 64, pad=pad)
        p.forward()
        p.backward()
        assert p.status() == 0
        p.check_untouched()
        a, b = (slice(int(s[0]), int(s[-1])) for s in (p.qs, p.ks))
        assert not p.o[a].any() and bool(torch.isneginf(p.lse[a]).all())
        assert not p.dq[a].any() and not p.dk[b].any() and not p.dv[b].any()


def test_two_calls_at_once_share_a_plan(scfa):
    """Two layers on two streams with one plan and a workspace each."""
    lens = same([700, 300]) + [(5, 3000)]
    a, b = Problem(scfa, lens, 4, 1, 64, seed=11), Problem(scfa, lens, 4, 1, 64, seed=12)
    b.plan = a.plan
    ref = []
    for p in (a, b):
        p.forward()
        p.backward()
        ref.append([t.clone() for t in (p.o, p.lse, p.dq, p.dk, p.dv)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for p, s in zip((a, b), streams):
            p.forward(stream=s)
            p.backward(stream=s)
    torch.cuda.synchronize()
    for p, r in zip((a, b), ref):
        assert p.status() == 0
        assert all(torch.equal(x, y) for x, y in zip(r, (p.o, p.lse, p.dq, p.dk, p.dv)))


def test_captured_steps_share_a_workspace(scfa):
    """Two graphs on one workspace, replayed in turn; a plan between replays."""
    a, b = Problem(scfa, [(4, 3000), (60, 60)], 4, 1, 64, seed=13), Problem(scfa, same([64, 3]), 4, 1, 64, seed=14)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for p in (a, b):
        p.ws = ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.forward()
            p.backward()
        graphs.append(g)
    for _ in range(2):
        for p, g in zip((a, b), graphs):
            g.replay()
            assert p.status() == 0
            p.check_forward()
            p.check_backward()
    # other sequences on the same rows
    b.qs = b.ks = np.array([0, 10, 67])
    scfa.scfa_packed_plan(i32(b.qs), i32(b.ks), b.N, b.M, 4, 1, 0, b.plan)
    graphs[1].replay()
    assert b.status() == 0
    b.check_forward()
    b.check_backward()


def test_a_stalled_pipeline_ends_with_a_status(scfa):
    """The producer withholds its loads: every wait gives up after its limit, and the device works on."""
    p = Problem(scfa, same([300, 20]), 4, 2, 64)
    p.forward(flags=scfa.FLAG_DEBUG_STALL)
    assert scfa.scfa_get_device_status(p.ws) == 5
    p.forward()
    p.backward(flags=scfa.FLAG_DEBUG_STALL)
    assert scfa.scfa_get_device_status(p.ws) == 5
    p.all()


def test_offsets_past_32_bits(scfa):
    """Rows whose offsets pass 2^31 elements, and values in a wide projection."""
    N, Hq, Hkv, D = 70000, 256, 4, 128
    lens = same([N - 300, 300])
    p = Problem.__new__(Problem)
    p.qs = p.ks = np.array([0, N - 300, N])
    p.N = p.M = N
    p.Hq, p.Hkv, p.D, p.dt, p.window, p.scfa, p.scale = Hq, Hkv, D, BF, 40, scfa, D ** -0.5
    new = dict(dtype=BF, device="cuda")
    qkv = torch.zeros((N, Hq + 2 * Hkv, D), **new)
    qkv[-600:] = rand(1, (600, Hq + 2 * Hkv, D))
    p.q, p.k, p.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    p.do = torch.zeros((N, Hq, D), **new)
    p.do[-600:] = rand(2, (600, Hq, D))
    p.o, p.lse = torch.empty((N, Hq, D), **new), torch.empty((N, Hq), device="cuda")
    grads = torch.empty_like(qkv)
    p.dq, p.dk, p.dv = grads[:, :Hq], grads[:, Hq:Hq + Hkv], grads[:, Hq + Hkv:]
    p.plan = scfa.workspace(scfa.packed_plan_size(N, N, len(lens), Hq, Hkv))
    p.ws = scfa.workspace(scfa.packed_workspace_size(True, N, N, len(lens), Hq, Hkv, D))
    scfa.scfa_packed_plan(i32(p.qs), i32(p.ks), N, N, Hq, Hkv, 40, p.plan)
    p.forward()
    p.backward()
    assert p.status() == 0
    p.check_forward([1], [0, 100, 255])
    p.check_backward([1], [3])


# ---------------------------------------------------------------- whole steps
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dt", [BF, HF])
def test_step_runs_all_of_it(scfa, norm, dt):
    """Norm, rotary positions, attention and all gradients of a layer, against the oracles one after another: each operator
    is held to its own bound on the rows that the one before it gave."""
    from oracle import rope as orope
    from sparse_causal_flash_gb300.packed import PackedStep
    from sparse_causal_flash_gb300.rope import Rope
    N, Hq, Hkv, D, lens = 260, 6, 2, 64, [100, 1, 0, 130]
    rope = Rope(32, interleaved=True)
    st = PackedStep(N, len(lens), Hq, Hkv, D, window=90, rope=rope, norm=norm, dtype=dt)
    starts = i32(np.concatenate([[0], np.cumsum(lens)]))
    st.plan(starts)
    x = rand(1, (N, Hq + 2 * Hkv, D), dt)
    x[231:] = float("nan")  # rows of nobody
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    do = rand(2, (N, Hq, D), dt)
    do[231:] = float("nan")
    pos = i32(np.concatenate([np.arange(n) for n in lens] + [np.zeros(29)]))
    w = [1 + 0.3 * rand(3 + i, (D,), torch.float32) for i in range(2)] if norm else [None, None]
    st.run(q, k, v, do, 0.125, pos, *w)
    assert st.status() == 0
    p = Problem.__new__(Problem)
    p.qs = p.ks = starts.cpu().numpy()
    p.Hq, p.Hkv, p.D, p.dt, p.window, p.scale = Hq, Hkv, D, dt, 90, 0.125
    p.q, p.k, p.v, p.o, p.lse, p.do = st.q_r, st.k_r, v, st.o, st.lse, do
    p.check_forward()
    # the turned rows
    n = 231
    f = rope.inv_freq.numpy()
    for got, rows, i in ((st.q_r, q, 0), (st.k_r, k, 1)):
        ref = orope.forward(dbl(rows[:n]), pos[:n].cpu().numpy(), f, True, 1.0, None if w[i] is None else dbl(w[i]), 1e-6)
        assert np.all(np.abs(dbl(got[:n]) - ref) <= half_step(ref, dt) + 2.0 ** -16 * np.abs(ref).max())
    # the attention's gradients before they were turned back: the same call again
    dq, dk, dv = (torch.zeros_like(t) for t in (st.q_r, st.k_r, st.k_r))
    ws = scfa.workspace(scfa.packed_workspace_size(True, N, N, len(lens), Hq, Hkv, D))
    scfa.scfa_packed_bwd(st.q_r, st.k_r, v, st.o, st.lse, do, st.plan_buf, 0.125, dq, dk, dv, ws)
    p.dq, p.dk, p.dv = dq, dk, dv
    p.check_backward()
    assert torch.equal(dv[:n], st.dv[:n]) and not st.dqkv[n:].any()
    for got, g, rows, i, dw in ((st.dq, dq, q, 0, st.dwq), (st.dk, dk, k, 1, st.dwk)):
        ref, ref_w = orope.backward(dbl(g[:n]), pos[:n].cpu().numpy(), f, True, 1.0, dbl(rows[:n]) if norm else None,
                                    None if w[i] is None else dbl(w[i]), 1e-6)
        assert np.all(np.abs(dbl(got[:n]) - ref) <= half_step(ref, dt) + 2.0 ** -15 * np.abs(ref).max())
        if norm:
            assert np.all(np.abs(dbl(dw) - ref_w) <= 2.0 ** -14 * np.abs(dbl(g[:n])).sum((0, 1)) * 3)
    # captured, and with another batch planned between replays
    first = st.dqkv.clone()
    graph = st.capture(q, k, v, do, 0.125, pos, *w)
    st.dqkv.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert st.status() == 0 and torch.equal(first[:n], st.dqkv[:n])


def test_step_gradient_against_differences(scfa):
    """The loss's change along directions against the gradients, through the whole step in fp16."""
    from sparse_causal_flash_gb300.packed import PackedStep
    from sparse_causal_flash_gb300.rope import Rope
    N, Hq, Hkv, D = 64, 4, 2, 64
    st = PackedStep(N, 2, Hq, Hkv, D, rope=Rope(64), norm=True, eps=1e-5, dtype=HF)
    st.plan(i32([0, 40, 64]))
    x = rand(1, (N, Hq + 2 * Hkv, D), HF)
    do = rand(2, (N, Hq, D), HF)
    pos = i32(np.concatenate([np.arange(40), np.arange(24)]))
    w = [1 + 0.3 * rand(3 + i, (D,), torch.float32) for i in range(2)]

    def loss(x, w):
        """In 64 bits, by the oracles."""
        from oracle import rope as orope
        f, ps = st.rope.inv_freq.numpy(), pos.cpu().numpy()
        q = orope.forward(x[:, :Hq], ps, f, w=w[0], eps=1e-5)
        k = orope.forward(x[:, Hq:Hq + Hkv], ps, f, w=w[1], eps=1e-5)
        total = 0.0
        for a, b in ((0, 40), (40, 64)):
            for h in range(Hq):
                total += (op.forward(q[a:b, h], k[a:b, h // 2], x[a:b, Hq + Hkv + h // 2], 0.125)[0] * dbl(do[a:b, h])).sum()
        return total

    st.run(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], do, 0.125, pos, *w)
    assert st.status() == 0
    x64, w64, g = dbl(x), [dbl(t) for t in w], np.random.default_rng(0)
    grads = [dbl(st.dqkv), dbl(st.dwq), dbl(st.dwk)]
    size = np.sqrt(sum((t * t).sum() for t in grads))
    for _ in range(6):
        u = [g.standard_normal(t.shape) for t in (x64, *w64)]
        h = 1e-5
        d = (loss(x64 + h * u[0], [w64[0] + h * u[1], w64[1] + h * u[2]]) -
             loss(x64 - h * u[0], [w64[0] - h * u[1], w64[1] - h * u[2]])) / (2 * h)
        # every rounding of a row on the way is at most 2^-11 of it; some forty meet in a gradient, along a random direction
        assert abs(d - sum((a * b).sum() for a, b in zip(u, grads))) <= 40 * 2.0 ** -11 * size


def test_step_refuses_what_does_not_fit(scfa):
    from sparse_causal_flash_gb300.packed import PackedStep
    from sparse_causal_flash_gb300.rope import Rope
    plain, turned = PackedStep(8, 1, 2, 1, 64), PackedStep(8, 1, 2, 1, 64, rope=Rope(0), norm=True)
    x, pos, w = rand(1, (8, 4, 64)), i32(np.arange(8)), torch.ones(64, device="cuda")
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    for st, kw in ((plain, dict(pos=pos)), (plain, dict(wq=w, wk=w)), (turned, dict()), (turned, dict(pos=pos)),
                   (turned, dict(pos=pos, wq=w))):
        with pytest.raises(ValueError):
            st.forward(q, k, v, 0.1, **kw)
    with pytest.raises(ValueError):
        plain.plan(i32([0, 4, 8]))
    with pytest.raises(ValueError):
        plain.forward(q[:4], k, v, 0.1)
    with pytest.raises(ValueError):
        PackedStep(8, 1, 2, 1, 64, rope=Rope(128))
    bad = x.transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match="channels"):
        plain.forward(bad[:, :2], k, v, 0.1)
    expanded = x[:1, :2].expand(8, 2, 64)  # rows that are one row: strides of zero
    with pytest.raises(scfa.ScfaError):
        plain.forward(expanded, k, v, 0.1)



@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size,v_up,scale", [(4e3, 8.0, 0.5), (1e-3, 1.0, 8.0), (1e-4, 1.0, 8.0), (1e-3, 0.01, 8.0)])
@pytest.mark.parametrize("lens,Hq,Hkv,window", [([(1500, 1500), (3, 3)], 2, 1, 0), ([(5, 9000)], 4, 1, 0),
                                                ([(700, 700)], 3, 3, 300)])
def test_fp16_gradients_of_any_size(scfa, monkeypatch, lens, Hq, Hkv, window, D, size, v_up, scale):
    """Flat rows over many keys: weights times (dP - delta) lie far below fp16's smallest number, or with a large dO above
    its largest, where the gradients themselves do not. P is held times 2^10 and dS times 2^k with 2^k |dO| |V| >= 2^10.5 for
    the longest rows of a piece of work: a rounding below the normal numbers moves P by at most 2^-35 and dS by at most
    2^-25 / 2^k <= 2^-35.5 |dO| |V|."""
    p = Problem(scfa, lens, Hq, Hkv, D, HF, window, seed=22, q_scale=0.1)
    p.k.mul_(0.1)
    p.v.mul_(v_up)
    p.do.copy_((p.do.float() * size).to(HF))
    p.scale = scale
    p.forward()
    p.backward()
    assert p.status() == 0
    norms = [float(torch.linalg.vector_norm(t.double(), dim=-1).max()) for t in (p.do, p.v)]
    monkeypatch.setitem(globals(), "tiny", lambda dt: 2.0 ** -35 + 2.0 ** -35.5 * norms[0] * norms[1])
    p.check_backward()


def test_fp16_gradients_beside_rows_that_are_not_finite(scfa):
    """A row of dO or v that is not finite leaves other sequences' bits alone, and the scale of its own as it is."""
    p, r = (Problem(scfa, same([90, 150, 33]), 4, 2, 64, HF, seed=23) for _ in range(2))
    for x in (p, r):
        x.do.mul_(1e-3)
        x.forward()
    r.do[100, 1, 5], r.do[200, 3, 0] = float("inf"), float("nan")
    for x in (p, r):
        x.backward()
        assert x.status() == 0
    for a, b in ((slice(0, 90), slice(0, 90)), (slice(240, 273), slice(240, 273))):
        assert all(torch.equal(getattr(p, key)[a], getattr(r, key)[a]) for key in ("dq", "dk", "dv"))
    for t, h in ((100, 1), (200, 3)):
        assert not torch.isfinite(r.dq[t, h]).any()
    ok = torch.ones(150, dtype=torch.bool, device="cuda")
    ok[[10, 110]] = False
    assert torch.isfinite(r.dq[90:240][ok]).all()
    assert float((p.dq[90:240][ok].double() - r.dq[90:240][ok].double()).abs().max()) <= float(p.dq.abs().max()) * 2.0 ** -9


# ---------------------------------------------------------------- steps: batches that are refused, plans that are shared
def packed_step(N=40, R=2, Hq=4, Hkv=2, D=64, **kw):
    from sparse_causal_flash_gb300.packed import PackedStep
    from sparse_causal_flash_gb300.rope import Rope
    st = PackedStep(N, R, Hq, Hkv, D, rope=Rope(D), norm=True, **kw)
    x = rand(1, (N, Hq + 2 * Hkv, D))
    args = (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], rand(2, (N, Hq, D)), 0.125, i32(np.arange(N)),
            torch.ones(D, device="cuda"), torch.ones(D, device="cuda"))
    return st, args


@pytest.mark.parametrize("starts", [[0, 30, 20], [0, 30, 41], [-1, 20, 40], [3, 20, 40], [40, 40, 40], [2 ** 31 - 1] * 3])
def test_step_leaves_gradients_of_a_refused_batch_alone(scfa, starts):
    """Starts that fall or leave the rows, or do not begin at 0: the status says so, and no row is written or turned."""
    st, args = packed_step()
    st.plan(i32([0, 20, 40]))
    st.run(*args)
    assert st.status() == 0
    first = st.dqkv.clone(), st.o.clone(), st.lse.clone()
    st.plan(i32(starts))
    for _ in range(2):
        st.run(*args)
        assert st.status() == 1
        assert all(torch.equal(a, b) for a, b in zip(first, (st.dqkv, st.o, st.lse)))
        assert not st.dwq.any() and not st.dwk.any()  # sums over no rows
    st.plan(i32([0, 20, 40]))
    st.run(*args)
    assert st.status() == 0
    assert all(torch.equal(a, b) for a, b in zip(first, (st.dqkv, st.o, st.lse)))


def test_layers_share_a_plan(scfa):
    """Forwards of all layers, then their backwards, on one plan: the bits of steps with plans of their own; and the next
    batch by one plan() for both."""
    (a, args), (alone, _) = packed_step(), packed_step()
    b, _ = packed_step(plan_of=a)
    other = (*(t.flip(0) for t in args[:4]), *args[4:])
    for starts in ([0, 20, 40], [0, 3, 37]):
        a.plan(i32(starts))
        a.forward(*args[:3], *args[4:])
        b.forward(*other[:3], *other[4:])
        b.backward(*other)
        a.backward(*args)
        assert a.status() == 0 and b.status() == 0
        alone.plan(i32(starts))
        for st, x in ((a, args), (b, other)):
            alone.run(*x)
            n = starts[-1]
            assert all(torch.equal(getattr(st, key)[:n], getattr(alone, key)[:n]) for key in ("o", "lse", "dqkv"))
            assert torch.equal(st.dwq, alone.dwq) and torch.equal(st.dwk, alone.dwk)
    b.plan(i32([0, 41, 40]))
    assert a.status() == 1
    for kw in (dict(N=41), dict(R=3), dict(Hq=2), dict(window=7)):
        with pytest.raises(ValueError, match="plan"):
            packed_step(plan_of=a, **kw)


def test_step_before_its_plan_computes_nothing(scfa, monkeypatch):
    """Also on memory that holds the plan of a step that is gone."""
    from sparse_causal_flash_gb300 import packed
    st, _ = packed_step()
    st.plan(i32([0, 20, 40]))
    plan = st.plan_buf
    monkeypatch.setattr(packed, "workspace", lambda n, dev: plan.clone() if n == plan.numel() else scfa.workspace(n, dev))
    st, args = packed_step()
    assert st.status() == 0
    for _ in range(2):
        st.run(*args)
        assert st.status() == 1
        assert not st.o.any() and not st.lse.any() and not st.dqkv.any() and not st.dwq.any()
    st.plan(i32([0, 20, 40]))
    st.run(*args)
    assert st.status() == 0 and bool(st.o.any())


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hq,Hkv", [([(200, 90), (40, 40)], 3, 1), ([(150, 7), (129, 128)], 4, 2), ([(300, 20)], 1, 1),
                                         ([(20, 3)], 8, 1)])
def test_queries_that_see_nothing_pass_no_gradient(scfa, lens, Hq, Hkv, D, dt):
    """Also where their rows of q and dO are not finite."""
    p = Problem(scfa, lens, Hq, Hkv, D, dt, seed=21)
    bad = []
    for (n, m), (a, _) in zip(lens, p.seqs()):
        bad.append(slice(a.start, a.start + max(0, n - m)))
        p.q[bad[-1]], p.do[bad[-1]] = float("nan"), float("inf")
    p.forward()
    p.backward()
    assert p.status() == 0
    for b in bad:
        assert not p.o[b].any() and bool(torch.isneginf(p.lse[b]).all()) and not p.dq[b].any()
        p.q[b] = p.do[b] = 0.0  # what the oracle may multiply by its zeros
    p.check_forward()
    p.check_backward()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("scale_up", [300.0, 30000.0])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_scores_far_from_zero(scfa, monkeypatch, dt, scale_up, D):
    """The forward's test of far scores, backward. The scores are exact here (one q, keys of +-1). A weight is recomputed from
    the stored lse: four roundings (lse from log2 units, its storage, log2(e), the way back) of at most 2^-24 |lse| each
    are 2^-22 |lse| of the weight."""
    n = 150
    p = Problem(scfa, same([n]), 2, 1, D, dt, seed=6)
    p.q.fill_(1.0)
    p.k.copy_(torch.sign(rand(1, (n, 1, D), dt)))
    p.k[7], p.k[3] = 1.0, 1.0
    p.q.mul_(scale_up / 8)
    p.forward()
    p.backward()
    assert p.status() == 0
    whole = parts

    def exact_scores(q, k, scale, window, lse_given):
        w, lse, _, top = whole(q, k, scale, window, lse_given)
        return w, lse, np.broadcast_to(2.0 ** -20 + 2.0 ** -22 * np.abs(lse)[:, None], w.shape), top

    monkeypatch.setitem(globals(), "parts", exact_scores)
    p.check_backward()


@pytest.mark.parametrize("D", [64, 128])
def test_shared_key_heads_are_copies_of_theirs(scfa, D):
    """o and lse bit by bit: a row's products, maxima and sums run over the same key tiles in the same order, whatever rows
    stand beside it (keys of tiles that it does not see add zeros). dk and dv of a shared head are the sums over its
    query heads: each side rounds once (u), the sums differ in order by n G 2^-23 of the magnitudes."""
    lens = same([200, 61])
    p, r = Problem(scfa, lens, 4, 2, D, seed=10), Problem(scfa, lens, 4, 4, D, seed=10)
    r.q.copy_(p.q), r.do.copy_(p.do)
    r.k.copy_(p.k.repeat_interleave(2, 1)), r.v.copy_(p.v.repeat_interleave(2, 1))
    for x in (p, r):
        x.forward()
        x.backward()
        assert x.status() == 0
    assert torch.equal(p.o, r.o) and torch.equal(p.lse, r.lse) and torch.equal(p.dq, r.dq)
    for key in ("dk", "dv"):
        one, two = dbl(getattr(p, key)), dbl(getattr(r, key))
        heads = two.reshape(*two.shape[:1], 2, 2, D)
        mags = np.zeros_like(one)
        for a, b in p.seqs():
            for h in range(4):
                q, k, v, do, o = (dbl(x) for x in (p.q[a, h], p.k[b, h // 2], p.v[b, h // 2], p.do[a, h], p.o[a, h]))
                w, _ = op.weights(q, k, p.scale)
                ds = np.abs(w * (do @ v.T - (do * o).sum(1, keepdims=True)))
                mags[b, h // 2] += w.T @ np.abs(do) if key == "dv" else p.scale * (ds.T @ np.abs(q))
        bound = half_step(one, BF) + half_step(heads[:, :, 0], BF) + half_step(heads[:, :, 1], BF) + 1.01 * 400 * 2.0 ** -23 * mags
        assert np.all(np.abs(one - heads.sum(2)) <= bound)


@pytest.mark.parametrize("D", [64, 128])
def test_a_stalled_pipeline_ends_with_a_status_in_fp16(scfa, D):
    """The warps that prepare dS's scale give up as the others do."""
    p = Problem(scfa, same([300, 20]) + [(2, 5000)], 4, 2, D, HF)
    p.forward()
    p.backward(flags=scfa.FLAG_DEBUG_STALL)
    assert scfa.scfa_get_device_status(p.ws) == 5
    p.all()


@pytest.mark.parametrize("D", [64, 128])
def test_fp16_query_gradients_beside_far_larger_ones(scfa, monkeypatch, D):
    """Rows of dO that are 2^20 apart, token by token and head by head, over flat rows: each row of dQ is held to its own
    size. Its dS moves by at most 2^-25 / 2^k <= 2^-37 |dO| |V| below the normal numbers, with the row's own |dO|."""
    p = Problem(scfa, same([1200, 5]), 4, 2, D, HF, seed=24, q_scale=0.1)
    p.k.mul_(0.1)
    p.scale = 8.0
    big = torch.arange(p.N, device="cuda")[:, None] * 3 + torch.arange(4, device="cuda") * 5
    p.do.copy_((p.do.float() * torch.where(big % 7 < 3, 1000.0, 1000.0 * 2.0 ** -20)[..., None]).to(HF))
    p.forward()
    p.backward()
    assert p.status() == 0
    v_long = float(torch.linalg.vector_norm(p.v.double(), dim=-1).max())
    monkeypatch.setitem(globals(), "tiny", lambda dt: 0.0)
    for a, b in p.seqs():
        for h in range(4):
            k, v, do = dbl(p.k[b, h // 2]), dbl(p.v[b, h // 2]), dbl(p.do[a, h])
            (ref, size), _, _ = grad_bounds(dbl(p.q[a, h]), k, v, do, dbl(p.o[a, h]), p.scale, 0, HF)
            low = 2.0 ** -37 * v_long * np.linalg.norm(do, axis=1)[:, None] * p.scale * (op.mask(len(do), len(k)) @ np.abs(k))
            check("dq", dbl(p.dq[a, h]), ref, (size + low) * 1.01 + half_step(ref, HF))
