"""Parity of the paged 4-bit cache on the GPU against the float64 oracle."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import cache4 as oc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
ROOT = pathlib.Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def scfa():
    import sparse_causal_flash_gb300 as s
    s.load()
    return s


def i32(x, dev="cuda"):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev)


def dbl(t):
    return t.detach().double().cpu().numpy()


def rand(seed, shape, dt=BF, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(dt)


def noise_cache(seed, P, H, D, ps):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (P, H, ps * (D + D // 16)), generator=g, dtype=torch.uint8).cuda()


# ---------------------------------------------------------------- plan
def run_plan(scfa, length, new, keep, free, n_free, table, N, ps, P, in_place=False):
    R = len(length)
    ln, nf, tb = i32(length), i32([n_free]), i32(table)
    fr = i32(list(free) + [-1] * (P - len(free)))
    lo, fo = (ln, nf) if in_place else (torch.full_like(ln, -7), torch.full_like(nf, -7))
    qs, slot, vis = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (R + 1, N, N))
    ws = scfa.workspace(scfa.cache4_plan_workspace_size(N, R))
    kp = None if keep is None else torch.as_tensor(np.asarray(keep), dtype=torch.uint8).cuda()
    scfa.scfa_cache4_plan(ln, i32(new), kp, fr, nf, tb, ps, P, lo, fo, qs, slot, vis, ws)
    st = scfa.scfa_get_device_status(ws)
    return st, dict(table=tb, len=lo, n_free=fo, q_start=qs, slot=slot, vis=vis)


def plan_problem(seed, R, lo, hi, n_hi, ps, slack=4):
    g = np.random.default_rng(seed)
    length, new = g.integers(lo, hi + 1, R), g.integers(0, n_hi + 1, R)
    mp = max(1, -(-(hi + n_hi) // ps))
    P = int(sum(-(-(int(a) + n_hi) // ps) for a in length)) + slack
    order = g.permutation(P)
    table, at = np.full((R, mp), -1), 0
    for r in range(R):
        n = -(-int(length[r]) // ps)
        table[r, :n] = order[at:at + n]
        at += n
    return length, new, order[at:].tolist(), table, P


@pytest.mark.parametrize("R,lo,hi,n_hi,ps,pad,drop", [
    (1, 0, 0, 1, 16, 0, None), (1, 15, 15, 1, 16, 3, None), (5, 0, 40, 9, 16, 2, 0.5), (33, 0, 300, 1, 64, 7, None),
    (64, 1, 5000, 1, 32, 0, None), (7, 0, 100, 200, 16, 5, 0.3), (3, 0, 10, 3000, 256, 1, 0.8), (2, 5, 9, 2600, 16, 0, None),
    (1500, 0, 50, 2, 16, 9, 0.7), (1100, 0, 20, 9, 16, 40, 0.5), (40, 0, 64, 0, 16, 1, None), (12, 0, 64, 30, 16, 0, 0.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_oracle(scfa, R, lo, hi, n_hi, ps, pad, drop, in_place):
    length, new, free, table, P = plan_problem(R * 7 + hi, R, lo, hi, n_hi, ps)
    N = int(new.sum()) + pad or 1
    keep = None if drop is None else (np.random.default_rng(3).random(N) < drop).astype(np.uint8) * 5
    ref = oc.plan(length, new, keep, free, len(free), table, N, ps, P)
    st, got = run_plan(scfa, length, new, keep, free, len(free), table, N, ps, P, in_place)
    assert st == 0
    for key, v in ref.items():
        assert np.array_equal(got[key].cpu().numpy().reshape(np.shape(v)), v), key


@pytest.mark.parametrize("length,new,n_free,N,code", [
    ([3, -1], [1, 1], 4, 4, 1), ([3, 3], [1, -2], 4, 4, 1), ([3, 3], [3, 2], 4, 4, 1), ([31, 3], [2, 1], 4, 4, 1),
    ([3, 40], [1, 1], 4, 4, 1), ([16, 16], [1, 1], 1, 4, 3), ([3, 3], [1, 1], -1, 4, 1), ([3, 3], [1, 1], 9, 4, 1),
    ([2 ** 31 - 1, 3], [1, 1], 4, 4, 1), ([3, 3], [2 ** 31 - 1, 2 ** 31 - 1], 4, 4, 1)])
@pytest.mark.parametrize("mask", [False, True])
def test_plan_that_does_not_fit_changes_nothing(scfa, length, new, n_free, N, code, mask):
    table = [[0, -1], [1, -1]]
    keep = [1] * N if mask else None
    st, got = run_plan(scfa, length, new, keep, [5, 4, 3, 2], n_free, table, N, 16, 8)
    assert st == code
    assert got["table"].tolist() == table and got["len"].tolist() == length and got["n_free"].tolist() == [n_free]
    assert got["q_start"].tolist() == [0, 0, 0] and got["slot"].tolist() == [-1] * N and got["vis"].tolist() == [0] * N


def test_plan_reports_page_ids_out_of_range(scfa):
    st, got = run_plan(scfa, [3, 16], [1, 1], None, [1, 800], 2, [[-1, -1], [0, -1]], 2, 16, 8)
    assert st == 1 and got["slot"].tolist() == [-1, -1] and got["vis"].tolist() == [4, 17]


# ---------------------------------------------------------------- append / read
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,H,ps,strided", [(1, 1, 16, False), (3, 5, 16, True), (37, 2, 64, False), (129, 3, 256, True)])
def test_append_then_read_matches_the_oracle(scfa, dt, D, N, H, ps, strided):
    P = -(-N // ps) + 3
    cache = noise_cache(N, P, H, D, ps)
    before = cache.clone()
    g = np.random.default_rng(N)
    slot = g.permutation(P * ps)[:N]
    if N > 3:
        slot[1], slot[2] = -1, P * ps  # a dropped row and one outside the cache
    kv = rand(N, (N, 2 * H + 3, D), dt, 2.0).cuda()
    k, v = kv[:, 1:1 + H], kv[:, 2 + H:2 + 2 * H]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    scfa.scfa_cache4_append(k, v, i32(slot), cache, ps)
    out = torch.full((N, 2 * H, D), 3.0, dtype=dt, device="cuda")
    ko, vo = (out[:, :H], out[:, H:]) if strided else (torch.full((N, H, D), 3.0, dtype=dt, device="cuda") for _ in "kv")
    scfa.scfa_cache4_read(cache, ps, i32(slot), ko, vo)
    live = ((slot >= 0) & (slot < P * ps))[:, None, None]
    assert np.array_equal(dbl(ko), oc.values(dbl(k)) * live)
    assert np.array_equal(dbl(vo), oc.values(dbl(v)) * live)
    # the bytes are where the format puts them, and nothing else was written
    flat, changed = cache.view(-1).cpu().numpy(), set()
    for n in np.flatnonzero(live[:, 0, 0])[:4]:
        for h in (0, H - 1):
            assert np.array_equal(oc.row(flat, int(slot[n]), h, H, D, ps, False), oc.values(dbl(k[n, h])))
            assert np.array_equal(oc.row(flat, int(slot[n]), h, H, D, ps, True), oc.values(dbl(v[n, h])))
    for n in np.flatnonzero(live[:, 0, 0]):
        for h in range(H):
            for ch in range(D):
                for is_v in (False, True):
                    at, _, sc = oc.addresses(int(slot[n]), h, ch, H, D, ps, is_v)
                    changed |= {at, sc}
    rest = np.ones(flat.size, bool)
    rest[list(changed)] = False
    assert np.array_equal(flat[rest], before.view(-1).cpu().numpy()[rest])


@pytest.mark.parametrize("dt", [BF, HF])
def test_append_at_the_borders(scfa, dt):
    """Ties of scale and code, zeros, the smallest and largest numbers, NaN and infinities."""
    D, H, ps = 64, 1, 16
    top = 3e38 if dt is BF else 65504.0
    rows = []
    for m in range(128, 256):  # every significand of the largest magnitude, ties of the scale among them
        rows.append([m / 16.0] + [(i + 0.5) * m / 112.0 for i in range(31)])
    for s in (1.0, 1.125, 1.25, 1.875, 2.0 ** -15, 1.5 * 2.0 ** -10):  # ties of the code
        rows.append([7 * s] + [(i / 2.0 - 7.5) * s for i in range(31)])
    rows += [[0.0] * 32, [-0.0] * 32, [float("nan")] * 32, [float("inf"), 1.0, float("nan")] + [-3.0] * 29,
             [-float("inf")] + [64512.0] * 31, [top] + [-top] * 31, [1e-6] * 32, [1.4e-5, 1.6e-5, -4e-5] + [0.0] * 29,
             [5.9e-8] * 32, [64512.0, -65000.0] + [60000.0] * 30, [float("nan"), 7.0] + [0.5] * 30]
    if len(rows) % 2:
        rows.append([1.0] * 32)
    x = torch.tensor(rows).to(dt).view(-1, 1, D).cuda()
    N = x.shape[0]
    cache = noise_cache(5, -(-N // ps), H, D, ps)
    slot = torch.arange(N, dtype=torch.int32, device="cuda")
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    scfa.scfa_cache4_append(x, x.flip(0), slot, cache, ps)
    scfa.scfa_cache4_read(cache, ps, slot, ko, vo)
    assert np.array_equal(dbl(ko), oc.values(dbl(x)))
    assert np.array_equal(dbl(vo), oc.values(dbl(x.flip(0))))


def test_append_and_read_past_32_bit_offsets(scfa):
    """A cache of more than 2^32 bytes: rows at its far end."""
    D, H, ps = 128, 8, 64
    P = (1 << 32) // (H * ps * (D + D // 16)) + 9
    cache = torch.zeros((P, H, ps * (D + D // 16)), dtype=torch.uint8, device="cuda")
    slot = np.array([5, P * ps - 1, P * ps - 70, (P // 2) * ps + 3])
    k, v = rand(1, (4, H, D)).cuda(), rand(2, (4, H, D)).cuda()
    scfa.scfa_cache4_append(k, v, i32(slot), cache, ps)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    scfa.scfa_cache4_read(cache, ps, i32(slot), ko, vo)
    assert np.array_equal(dbl(ko), oc.values(dbl(k))) and np.array_equal(dbl(vo), oc.values(dbl(v)))
    # and attended over
    table, qs, vis = i32([[P - 1, P - 2]]), i32([0, 1]), i32([ps + 1])
    q, o, lse = rand(3, (1, H, D)).cuda(), torch.empty((1, H, D), dtype=BF, device="cuda"), torch.empty((1, H), device="cuda")
    ws = scfa.workspace(scfa.cache4_attn_workspace_size(1, 1, H, H, D))
    scfa.scfa_cache4_attn(q, cache, ps, table, qs, vis, 0.09, o, lse, ws)
    assert scfa.scfa_get_device_status(ws) == 0
    slots = np.concatenate([np.arange(ps) + (P - 1) * ps, [(P - 2) * ps]])
    kk = torch.empty((ps + 1, H, D), dtype=BF, device="cuda")
    vv = torch.empty_like(kk)
    scfa.scfa_cache4_read(cache, ps, i32(slots), kk, vv)
    check_rows(dbl(q), dbl(kk), dbl(vv), [ps + 1], 0.09, o, lse, BF)


# ---------------------------------------------------------------- attention
def check_rows(q, k, v, vis, scale, o, lse, dt):
    """Rows q [n, Hq, D] over k, v [L, Hkv, D] (the exact values the cache holds).

    Bounds. uo is half a step of the output type. A weight p is rounded to
    fp16 (half a step: 2^-11) before it meets V: at most 2^-11 sum(p |v|) in O,
    and weights below 2^-21 of the largest lose up to 2^-32 of it: 2^-32 n
    max|v|. A score is, per group, a sum of 32 products q (c + 8) <= 15 |q| in
    fp32, each of its D / 8 + 4 additions off by at most 2^-23 of 15 sum |q|, and
    q itself by 2^-25 of its row's largest: e = (D / 8 + 4) 2^-23 15 scale
    sum_g s_g sum |q_g| + 2^-20 |score| for the products with the scales and
    the change of base. Weights are then off by 2 e relative (numerator and
    denominator), LSE by e; exp2 and the fp32 sums add 2^-18."""
    uo, up = (2.0 ** -8 if dt is BF else 2.0 ** -11), 2.0 ** -11
    o, lse = dbl(o), dbl(lse)
    G, D = q.shape[1] // k.shape[1], q.shape[2]
    for t in range(q.shape[0]):
        for h in range(q.shape[1]):
            n, hk = int(vis[t]), h // G
            kk, vv = k[:n, hk], v[:n, hk]
            ro, rl = oc.attention(q[t, h], kk, vv, scale)
            if n == 0:
                assert not o[t, h].any() and lse[t, h] == -np.inf
                continue
            # a group's scale is at most its largest value (the code of that is 7, or 0 in a zero group)
            sg = np.abs(kk).reshape(n, -1, 32).max(-1) / 6 + 2.0 ** -15
            qg = np.abs(q[t, h]).reshape(-1, 32).sum(-1)
            s = np.abs(kk @ q[t, h] * scale).max()
            e = (D / 8 + 4) * 2.0 ** -23 * 15 * scale * (sg @ qg).max() + 2.0 ** -20 * s
            p = np.exp(kk @ q[t, h] * scale - rl)
            a = p @ np.abs(vv)
            assert abs(lse[t, h] - rl) <= e + 2.0 ** -18 * max(1.0, abs(rl)), (t, h, lse[t, h], rl)
            err = np.abs(o[t, h] - ro)
            tol = uo * np.abs(ro) + (up + 2 * e + 2.0 ** -18) * a + 2.0 ** -32 * n * np.abs(vv).max() + 2.0 ** -24
            assert np.all(err <= tol), (t, h, n, float((err / tol).max()))


def attn_problem(scfa, seed, lens, news, Hq, Hkv, D, ps, dt, extra=0, spread=0.3):
    """Rows cached through append, their exact values, and everything attn takes."""
    R = len(lens)
    g = np.random.default_rng(seed)
    have = [-(-n // ps) for n in lens]
    P, mp = sum(have) + 4, max(1, max(have)) + 1
    order = g.permutation(P)
    table, at = np.full((R, mp), -1), 0
    for r in range(R):
        table[r, :have[r]] = order[at:at + have[r]]
        at += have[r]
    cache = noise_cache(seed, P, Hkv, D, ps)
    rows = []
    for r in range(R):
        n = max(1, lens[r])
        k, v = rand(seed + 2 * r, (n, Hkv, D), dt, spread).cuda(), rand(seed + 2 * r + 1, (n, Hkv, D), dt, spread).cuda()
        if lens[r]:
            pos = np.arange(n)
            scfa.scfa_cache4_append(k, v, i32(table[r, pos // ps] * ps + pos % ps), cache, ps)
        rows.append((oc.values(dbl(k))[:lens[r]], oc.values(dbl(v))[:lens[r]]))
    q_start = np.concatenate([[0], np.cumsum(news)])
    N = int(q_start[-1]) + extra
    vis = np.full(max(N, 1), 10 ** 6)
    for r in range(R):
        vis[q_start[r]:q_start[r + 1]] = np.maximum(0, lens[r] - news[r] + 1 + np.arange(news[r]))
    q = rand(seed + 999, (max(N, 1), Hq, D), dt).cuda()
    return dict(q=q, cache=cache, ps=ps, table=i32(table), q_start=i32(q_start), vis=i32(vis), rows=rows, news=news,
                scale=D ** -0.5, dt=dt)


def run_attn(scfa, p, o=None, lse=None, stream=None):
    N, Hq, D = p["q"].shape
    o = torch.full((N, Hq, D), 77.0, dtype=p["dt"], device="cuda") if o is None else o
    lse = torch.full((N, Hq), 77.0, device="cuda") if lse is None else lse
    ws = scfa.workspace(scfa.cache4_attn_workspace_size(N, p["table"].shape[0], Hq, p["cache"].shape[1], D))
    scfa.scfa_cache4_attn(p["q"], p["cache"], p["ps"], p["table"], p["q_start"], p["vis"], p["scale"], o, lse, ws, 0,
                          stream)
    return o, lse, ws


def check_attn(scfa, p):
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    qs, vis = p["q_start"].tolist(), p["vis"].cpu().numpy()
    for r, (k, v) in enumerate(p["rows"]):
        a, b = qs[r], qs[r + 1]
        check_rows(dbl(p["q"][a:b]), k, v, vis[a:b], p["scale"], o[a:b], lse[a:b], p["dt"])
    assert torch.all(o[qs[-1]:] == 77.0) and torch.all(lse[qs[-1]:] == 77.0)  # rows behind the last request
    return o, lse


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (12, 1), (20, 1), (40, 1)])
def test_attn_single_tokens(scfa, dt, D, Hq, Hkv):
    check_attn(scfa, attn_problem(scfa, Hq + D, [1, 0, 17, 64, 65, 300], [1] * 6, Hq, Hkv, D, 64, dt))


@pytest.mark.parametrize("ps", [16, 32, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_attn_page_sizes_and_ragged_tokens(scfa, ps, D):
    check_attn(scfa, attn_problem(scfa, ps, [5, 0, 16, 255, 257, 40, 1], [5, 0, 3, 0, 9, 1, 1], 4, 2, D, ps, BF, extra=3))


@pytest.mark.parametrize("lens,news,Hq,Hkv,D,dt", [
    ([3001], [1], 8, 1, 128, BF), ([2049, 3, 700], [1, 1, 1], 16, 2, 64, HF), ([1500], [130], 4, 2, 128, BF),
    ([70, 333, 64], [70, 65, 64], 6, 2, 64, BF), ([900, 33], [37, 33], 5, 1, 128, HF), ([0, 0], [3, 1], 4, 2, 64, BF),
    ([130] * 70, [1] * 70, 8, 8, 64, BF), ([20] * 9, [16] * 9, 2, 1, 128, BF), ([4, 4], [9, 2], 2, 2, 64, BF),
    ([700, 2100], [12, 9], 4, 1, 64, BF), ([2100, 5], [12, 5], 5, 1, 128, HF), ([1000] * 20, [7] * 20, 8, 2, 128, BF),
    ([1000, 40, 3, 600], [9, 1, 2, 7], 12, 2, 64, HF), ([129] * 3, [1] * 3, 48, 1, 128, BF), ([300], [257], 3, 3, 128, HF),
    ([0, 7, 0], [40, 7, 1], 4, 4, 64, BF), ([64] * 4, [33, 1, 64, 2], 2, 1, 128, BF), ([33] * 50, [17] * 50, 2, 2, 64, BF)])
def test_attn_shapes(scfa, lens, news, Hq, Hkv, D, dt):
    check_attn(scfa, attn_problem(scfa, sum(lens), lens, news, Hq, Hkv, D, 16, dt))


def test_attn_without_any_token(scfa):
    p = attn_problem(scfa, 1, [5, 9], [0, 0], 4, 2, 64, 16, BF, extra=3)
    check_attn(scfa, p)


@pytest.mark.parametrize("news", [[1, 3], [9, 7], [90, 25]])
@pytest.mark.parametrize("dt", [BF, HF])
def test_attn_far_scores(scfa, dt, news):
    """Scores far from zero, of both signs: the running maximum grows and the first keys hold next to nothing."""
    p = attn_problem(scfa, 8, [400, 90], news, 4, 2, 64, 32, dt, spread=1.5)
    p["scale"] = 0.9
    p["q"] *= torch.linspace(-6, 6, p["q"].shape[0] * 4, device="cuda").view(-1, 4, 1).to(dt)
    check_attn(scfa, p)


def test_attn_strides_and_equal_bits(scfa):
    p = attn_problem(scfa, 3, [100, 900, 33], [2, 1, 4], 8, 2, 128, 64, BF)
    o, lse = check_attn(scfa, p)
    wide = torch.zeros((7, 8 + 4, 128), dtype=BF, device="cuda")
    wide[:, 2:10] = p["q"]
    out = torch.full((7, 3, 8, 128), 5.0, dtype=BF, device="cuda")
    o2, l2, _ = run_attn(scfa, {**p, "q": wide[:, 2:10]}, o=out[:, 1])
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert torch.all(out[:, 0] == 5.0) and torch.all(out[:, 2] == 5.0)
    heads_first = torch.empty((8, 7, 128), dtype=BF, device="cuda").transpose(0, 1)
    o3, _, _ = run_attn(scfa, {**p, "q": heads_first.copy_(p["q"])}, o=torch.empty_like(heads_first))
    assert torch.equal(o, o3)


def test_attn_on_a_side_stream_and_in_a_graph(scfa):
    p = attn_problem(scfa, 4, [100, 900, 33, 2], [1] * 4, 8, 2, 64, 64, BF)
    o, lse, _ = run_attn(scfa, p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2, _ = run_attn(scfa, p, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    ws = scfa.workspace(scfa.cache4_attn_workspace_size(4, 4, 8, 2, 64))
    outs = [(torch.zeros_like(o), torch.zeros_like(lse)) for _ in range(2)]
    graphs = []
    for a, b in outs:  # two graphs on one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            scfa.scfa_cache4_attn(p["q"], p["cache"], p["ps"], p["table"], p["q_start"], p["vis"], p["scale"], a, b, ws)
        graphs.append(g)
    for i in (0, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(o, a) and torch.equal(lse, b)
    # longer answers on the same graph
    p["vis"].sub_(1)
    graphs[0].replay()
    o3, l3, _ = run_attn(scfa, p)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], o3) and torch.equal(outs[0][1], l3)


@pytest.mark.parametrize("news", [[1, 2], [20, 30]])
def test_attn_page_ids_out_of_range_are_masked_and_reported(scfa, news):
    p = attn_problem(scfa, 5, [200, 90], news, 4, 2, 64, 16, BF)
    P = p["cache"].shape[0]
    p["table"][0, 3], p["table"][1, 0], p["table"][1, 5] = -5, P, 2 ** 30
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 1
    for r, gone in ((0, {3}), (1, {0, 5})):
        k, v = p["rows"][r]
        sel = [i for i in range(len(k)) if i // 16 not in gone]
        a, b = p["q_start"][r:r + 2].tolist()
        for t in range(a, b):
            n = sum(i < int(p["vis"][t]) for i in sel)
            check_rows(dbl(p["q"][t:t + 1]), k[sel], v[sel], [n], p["scale"], o[t:t + 1], lse[t:t + 1], BF)
    p["table"][0, 3] = p["table"][0, 2]
    p["table"][1, 0] = p["table"][1, 5] = p["table"][1, 1]
    _, _, ws2 = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws2) == 0


@pytest.mark.parametrize("new", [1, 10])
def test_attn_page_id_out_of_range_for_all_keys(scfa, new):
    p = attn_problem(scfa, 6, [10], [new], 2, 1, 64, 16, BF)
    p["table"].fill_(-1)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 1
    assert not o.any() and torch.all(lse == -torch.inf)


def test_attn_wild_row_bounds(scfa):
    """q_start and vis outside their ranges read and write nothing out of bounds."""
    p = attn_problem(scfa, 7, [30, 30], [2, 2], 2, 1, 64, 16, BF)
    p["vis"][3] = 2 ** 31 - 1  # more than the table has pages for: its pages past the end are -1
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 1
    p["q_start"].copy_(i32([0, 2, 400]))
    o, lse, ws = run_attn(scfa, p)
    torch.cuda.synchronize()
    p["q_start"].copy_(i32([-3, 2, 1]))
    run_attn(scfa, p)
    torch.cuda.synchronize()


@pytest.mark.parametrize("news", [[1, 1], [20, 3]])
def test_attn_stalled_pipeline_reports_a_timeout(scfa, news):
    p = attn_problem(scfa, 9, [300, 20], news, 8, 2, 64, 16, BF)
    N, Hq, D = p["q"].shape
    o, lse = torch.empty_like(p["q"]), torch.empty((N, Hq), device="cuda")
    ws = scfa.workspace(scfa.cache4_attn_workspace_size(N, 2, Hq, 2, D))
    scfa.scfa_cache4_attn(p["q"], p["cache"], 16, p["table"], p["q_start"], p["vis"], 0.125, o, lse, ws,
                          scfa.FLAG_DEBUG_STALL)
    assert scfa.scfa_get_device_status(ws) == 5
    check_attn(scfa, p)  # the device stays usable


# ---------------------------------------------------------------- steps
@pytest.mark.parametrize("dt,D,Hq,Hkv,ps", [(BF, 64, 12, 12, 64), (HF, 128, 8, 2, 16)])
@pytest.mark.parametrize("drop", [None, 0.6])
def test_steps_together(scfa, dt, D, Hq, Hkv, ps, drop):
    """Prompts, then single tokens, a release and a new request, against a dense replay of everything cached."""
    from sparse_causal_flash_gb300.cache import KVCache4
    R, scale = 3, D ** -0.5
    c = KVCache4(R, 24, Hq, Hkv, D, max_len=160, max_tokens=160, page_size=ps, dtype=dt)
    held = [(np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))) for _ in range(R)]
    g = np.random.default_rng(1)
    for i, new in enumerate([[40, 0, 75], [1, 0, 1], [1, 33, 1], "release", [1, 1, 20], [4, 4, 0], [0, 0, 0]]):
        if new == "release":
            c.release(2)
            held[2] = tuple(np.zeros((0, Hkv, D)) for _ in "kv")
            assert sorted(c.free[:int(c.n_free)].tolist() + c.table[0, :-(-int(c.len[0]) // ps)].tolist()
                          + c.table[1, :-(-int(c.len[1]) // ps)].tolist()) == list(range(24))
            continue
        N = sum(new) + 2
        q = rand(50 + i, (N, Hq, D), dt).cuda()
        kv = rand(90 + i, (N, 2 * Hkv, D), dt).cuda()
        keep = None if drop is None else (g.random(N) < drop).astype(np.uint8)
        o, lse = c.step(q, kv[:, :Hkv], kv[:, Hkv:], i32(new), scale,
                        None if keep is None else torch.as_tensor(keep).cuda())
        assert c.status() == 0
        at = 0
        for r in range(R):
            k, v = held[r]
            for t in range(at, at + new[r]):
                if keep is None or keep[t]:
                    k = np.concatenate([k, oc.values(dbl(kv[t:t + 1, :Hkv]))])
                    v = np.concatenate([v, oc.values(dbl(kv[t:t + 1, Hkv:]))])
                check_rows(dbl(q[t:t + 1]), k, v, [len(k)], scale, o[t:t + 1], lse[t:t + 1], dt)
            held[r], at = (k, v), at + new[r]
        assert c.len.tolist() == [len(k) for k, _ in held]
    for r in range(R):
        k, v = c.rows(r)
        assert np.array_equal(dbl(k), held[r][0]) and np.array_equal(dbl(v), held[r][1])


def test_captured_steps_equal_eager_ones(scfa):
    from sparse_causal_flash_gb300.cache import KVCache4
    R, Hq, Hkv, D = 5, 8, 2, 64
    a, b = (KVCache4(R, 60, Hq, Hkv, D, max_len=96, max_tokens=300, page_size=16) for _ in "ab")
    prompt = i32([30, 1, 50, 0, 17])
    q, kv = rand(1, (98, Hq, D)).cuda(), rand(2, (98, 2 * Hkv, D)).cuda()
    for c in (a, b):
        c.step(q, kv[:, :Hkv], kv[:, Hkv:], prompt, 0.125)
    q1, kv1, ones = torch.empty_like(q[:R]), torch.empty_like(kv[:R]), i32([1] * R)
    g = b.capture(q1, kv1[:, :Hkv], kv1[:, Hkv:], ones, 0.125)
    assert b.len.tolist() == a.len.tolist()
    for i in range(20):
        q1.copy_(rand(100 + i, (R, Hq, D)))
        kv1.copy_(rand(200 + i, (R, 2 * Hkv, D)))
        o, lse = a.step(q1, kv1[:, :Hkv], kv1[:, Hkv:], ones, 0.125)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, b.o[:R]) and torch.equal(lse, b.lse[:R])
    assert a.len.tolist() == b.len.tolist() == [50, 21, 70, 20, 37]
    assert torch.equal(a.cache, b.cache) and torch.equal(a.table, b.table)
    assert a.status() == 0 and b.status() == 0


def test_step_without_room_computes_nothing(scfa):
    from sparse_causal_flash_gb300.cache import KVCache4
    c = KVCache4(2, 3, 4, 2, 64, max_len=64, max_tokens=64, page_size=16)
    q, kv = rand(1, (60, 4, 64)).cuda(), rand(2, (60, 4, 64)).cuda()
    c.step(q[:40], kv[:40, :2], kv[:40, 2:], i32([20, 20]), 0.125)
    assert c.status() == 3 and c.len.tolist() == [0, 0] and int(c.n_free) == 3
    assert not c.o.any() and not c.cache.any()
    c.step(q[:40], kv[:40, :2], kv[:40, 2:], i32([32, 8]), 0.125)
    assert c.status() == 0 and c.len.tolist() == [32, 8] and int(c.n_free) == 0


@pytest.mark.parametrize("Hq", [8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 200])
def test_attn_query_heads_per_key_head(scfa, Hq):
    """Single tokens on both sides of every change of the row block."""
    check_attn(scfa, attn_problem(scfa, Hq, [1, 130, 700], [1] * 3, Hq, 1, 64, 32, BF))


@pytest.mark.parametrize("R,per", [(161, 1), (400, 1), (737, 9), (900, 12)])
def test_attn_more_requests_than_threads(scfa, R, per):
    """The requests of a CTA's piece are found in several rounds; some bring nothing."""
    news = [0 if r % 7 == 3 else per + (r % 3 if per > 1 else 0) for r in range(R)]
    lens = [n + (r * 37) % 150 for r, n in enumerate(news)]
    check_attn(scfa, attn_problem(scfa, R, lens, news, 2, 1, 64, 32, BF, extra=2))


@pytest.mark.parametrize("news", [[1, 1], [1, 3], [9, 7], [90, 25]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attn_a_query_that_is_not_finite_spoils_its_row_only(scfa, news, bad):
    p = attn_problem(scfa, 12, [1400, 90], news, 4, 2, 128, 32, BF)
    p["q"][1, 2, 5] = bad
    o, lse, _ = run_attn(scfa, p)
    assert torch.isnan(lse[1, 2]) and torch.isnan(o[1, 2]).all()
    qs, vis = p["q_start"].tolist(), p["vis"].tolist()
    for r, (k, v) in enumerate(p["rows"]):
        for t in range(qs[r], qs[r + 1]):
            for h in (h for h in range(4) if (t, h) != (1, 2)):
                check_rows(dbl(p["q"][t:t + 1, h:h + 1]), k[:, h // 2:h // 2 + 1], v[:, h // 2:h // 2 + 1], [vis[t]],
                           p["scale"], o[t:t + 1, h:h + 1], lse[t:t + 1, h:h + 1], BF)


@pytest.mark.parametrize("news", [[1, 3], [9, 7], [90, 25]])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("k_by,v_by,q_by", [(2.0 ** -14, 2.0 ** -13, 2.0 ** 10), (2.0 ** 12, 2.0 ** 13, 2.0 ** -13)])
def test_attn_small_and_large_rows(scfa, news, dt, k_by, v_by, q_by):
    """Scales at both ends of the format, queries that undo those of the keys."""
    p = attn_problem(scfa, 14, [200, 90], news, 4, 2, 64, 32, dt)
    ps, rows = p["ps"], []
    for r, n in enumerate([200, 90]):
        k, v = rand(50 + r, (n, 2, 64), dt).cuda() * k_by, rand(60 + r, (n, 2, 64), dt).cuda() * v_by
        pos = torch.arange(n, device="cuda")
        scfa.scfa_cache4_append(k, v, (p["table"][r, pos // ps] * ps + pos % ps).int(), p["cache"], ps)
        rows.append((oc.values(dbl(k)), oc.values(dbl(v))))
    check_attn(scfa, {**p, "rows": rows, "q": p["q"] * q_by})


@pytest.mark.parametrize("news", [[1, 1], [9, 7], [90, 25]])
@pytest.mark.parametrize("by", [2.0 ** -108, 2.0 ** 100])
def test_attn_scale_undoes_the_queries(scfa, news, by):
    """A power of two moved from the queries to the scale changes no bit."""
    p = attn_problem(scfa, 16, [700, 90], news, 4, 2, 128, 32, BF)
    o, lse, _ = run_attn(scfa, p)
    o2, lse2, _ = run_attn(scfa, {**p, "q": p["q"] * by, "scale": p["scale"] / by})
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_streams_with_workspaces_of_their_own(scfa):
    ps = [attn_problem(scfa, 20 + i, [900, 5000, 33], news, 8, 2, 64, 64, BF)
          for i, news in enumerate([[1] * 3, [40, 9, 20]])]
    ref = [run_attn(scfa, p)[:2] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(20):
        got = [run_attn(scfa, p, stream=s)[:2] + (s,) for p, s in zip(ps, streams)]
        torch.cuda.synchronize()
        for (o, lse), (a, b, _) in zip(ref, got):
            assert torch.equal(o, a) and torch.equal(lse, b)


@pytest.mark.parametrize("N,R", [(5, 2), (40, 3), (4097, 2), (20011, 3), (70000, 1200)])
@pytest.mark.parametrize("ko,vo", [(0, 0), (3, 0), (0, 1)])
def test_plan_masks_at_any_address(scfa, N, R, ko, vo):
    """The keep mask is read 16 tokens at a time where it and vis are aligned, one by one elsewhere."""
    g = np.random.default_rng(N + ko)
    cut = np.sort(g.integers(0, N + 1, R - 1))
    new = np.diff(np.concatenate([[0], cut, [N - N // 5]]).clip(max=N - N // 5))
    length = g.integers(0, 50, R)
    mp = int(-(-(length + new).max() // 16))
    table, at = np.full((R, mp), -1), 0
    for r in range(R):
        n = -(-int(length[r]) // 16)
        table[r, :n] = np.arange(at, at + n)
        at += n
    P = at + int((-(-(length + new) // 16)).sum())
    keep = (g.random(N) < 0.5).astype(np.uint8)
    ref = oc.plan(length, new, keep, list(range(at, P)), P - at, table, N, 16, P)
    kp, vis = torch.zeros(N + 16, dtype=torch.uint8, device="cuda")[ko:ko + N], i32([-9] * (N + 4))[vo:vo + N]
    kp.copy_(torch.as_tensor(keep))
    ln, nf, tb, fr = i32(length), i32([P - at]), i32(table), i32(list(range(at, P)) + [-1] * at)
    qs, slot = i32([-9] * (R + 1)), i32([-9] * N)
    ws = scfa.workspace(scfa.cache4_plan_workspace_size(N, R))
    scfa.scfa_cache4_plan(ln, i32(new), kp, fr, nf, tb, 16, P, ln, nf, qs, slot, vis, ws)
    assert scfa.scfa_get_device_status(ws) == 0
    for key, got in dict(table=tb, len=ln, n_free=nf, q_start=qs, slot=slot, vis=vis).items():
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref[key])), ref[key]), key


def test_steps_on_another_stream(scfa):
    from sparse_causal_flash_gb300.cache import KVCache4
    R, Hq, Hkv, D = 2, 4, 2, 128
    a, b, c = (KVCache4(R, 20, Hq, Hkv, D, max_len=96, max_tokens=100, page_size=32) for _ in "abc")
    side = torch.cuda.Stream()
    for i, new in enumerate([[50, 0], [1, 30], [1, 1]]):
        q, kv, n = rand(i, (sum(new), Hq, D)).cuda(), rand(9 + i, (sum(new), 2 * Hkv, D)).cuda(), i32(new)
        torch.cuda.synchronize()
        o, lse = a.step(q, kv[:, :Hkv], kv[:, Hkv:], n, 0.1)
        ob, lb = b.step(q, kv[:, :Hkv], kv[:, Hkv:], n, 0.1, stream=side)
        with torch.cuda.stream(side):
            oc_, lc = c.step(q, kv[:, :Hkv], kv[:, Hkv:], n, 0.1)
        torch.cuda.synchronize()
        for x, y in ((ob, lb), (oc_, lc)):
            assert torch.equal(o, x) and torch.equal(lse, y)
    assert a.status() == b.status() == c.status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attn_past_32_bit_offsets(scfa, new):
    """The same rows in the first and in the last pages of a cache of more than 2^32 bytes: the same bits."""
    H, D, ps, L = 8, 128, 256, 700
    P = 2 ** 32 // (H * ps * (D + D // 16)) + 8
    cache = torch.empty((P, H, ps * (D + D // 16)), dtype=torch.uint8, device="cuda")
    k, v, q = rand(1, (L, H, D)).cuda(), rand(2, (L, H, D)).cuda(), rand(3, (new, 16, D)).cuda()
    t, got = torch.arange(L, device="cuda"), []
    for pages in ([0, 1, 2], [P - 1, P - 3, P - 2]):
        table = i32([pages])
        scfa.scfa_cache4_append(k, v, (table[0, t // ps] * ps + t % ps).int(), cache, ps)
        p = dict(q=q, cache=cache, ps=ps, table=table, q_start=i32([0, new]), vis=i32(range(L - new + 1, L + 1)),
                 scale=D ** -0.5, dt=BF)
        got.append(run_attn(scfa, p)[:2])
        cache[pages].fill_(0)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][1]).all()


def test_a_first_call_may_be_captured(scfa):
    """In a process that has run no kernel of the library yet."""
    code = """if 1:
        import torch
        from sparse_causal_flash_gb300.cache import KVCache4
        for new in (1, 40):
            q, kv = torch.randn(2 * new, 4, 64).cuda().bfloat16(), torch.randn(2 * new, 4, 64).cuda().bfloat16()
            n = torch.full((2,), new, dtype=torch.int32, device="cuda")
            a, b = (KVCache4(2, 20, 4, 2, 64, max_len=128, max_tokens=80, page_size=16) for _ in "ab")
            g = a.capture(q, kv[:, :2], kv[:, 2:], n, 0.125)
            g.replay()
            o, lse = b.step(q, kv[:, :2], kv[:, 2:], n, 0.125)
            torch.cuda.synchronize()
            assert a.status() == 0 and torch.equal(a.o[:2 * new], o) and torch.equal(a.lse[:2 * new], lse) and o.any()
    """
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_a_refused_step_leaves_the_cache_as_it_was(scfa):
    from sparse_causal_flash_gb300.cache import KVCache4
    c = KVCache4(2, 8, 4, 2, 64, max_len=64, max_tokens=16, page_size=16)
    q, kv, new = rand(1, (9, 4, 64)).cuda(), rand(2, (9, 4, 64)).cuda(), i32([5, 4])
    k, v = kv[:, :2], kv[:, 2:]
    odd = torch.zeros(9 * 4 * 64 + 8, dtype=BF, device="cuda")
    for bad in (dict(k=k.float()), dict(v=v[:8]), dict(v=kv), dict(q=q.cpu()), dict(q=q[:, :, :32]), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=1e-50), dict(scale=1e39),
                dict(q=odd[4:4 + q.numel()].view(q.shape)), dict(new_len=new.long()),
                dict(k=odd[:9 * 132].as_strided((9, 2, 64), (132, 64, 1))), dict(keep=torch.ones(9, device="cuda") > 0)):
        with pytest.raises(ValueError):
            c.step(**{**dict(q=q, k=k, v=v, new_len=new, scale=0.125), **bad})
    assert c.len.tolist() == [0, 0] and int(c.n_free) == 8 and not c.cache.any()
    c.step(q, k, v, new, 0.125)
    assert c.status() == 0 and c.len.tolist() == [5, 4]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [3, 12, 25])
def test_attn_many_short_items_keep_their_queries(scfa, D, new):
    """Blocks of 32, 64 and 128 rows, a dozen items of one unit in every CTA: each takes the place of the queries of the
    item before last, whose scores have to be done."""
    R = 1000
    p = attn_problem(scfa, 31, [new + r % 60 for r in range(R)], [new] * R, 8, 2, D, 32, BF)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    for _ in range(10):
        o2, lse2, _ = run_attn(scfa, p)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    vis = p["vis"].cpu().numpy()
    for r in range(0, R, 37):
        a, b = r * new, r * new + new
        check_rows(dbl(p["q"][a:b]), *p["rows"][r], vis[a:b], p["scale"], o[a:b], lse[a:b], BF)


@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 128), (HF, 64), (HF, 128)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("new,Hq", [(1, 2), (1, 12), (4, 2), (10, 2), (20, 2), (70, 2)])
def test_attn_an_infinite_query_over_keys_of_one_sign(scfa, dt, D, bad, new, Hq):
    """Blocks of 8 to 128 rows, each row with a query channel that is not finite and up to three keys whose codes in it have
    one sign: NaN in o and lse, and finite rows beside it."""
    for sign in (1.0, -1.0):
        p = attn_problem(scfa, 17, [0] * 4, [new] * 4, Hq, 1, D, 16, dt)
        p["vis"].copy_(i32([min(3, t + r) for r in range(4) for t in range(new)]))
        P = p["cache"].shape[0]
        p["table"][:, 0] = i32(np.arange(4) % P)
        k, v = rand(3, (P * 16, 1, D), dt).cuda(), rand(4, (P * 16, 1, D), dt).cuda()
        k[..., 7] = sign * (1 + k[..., 7].abs())
        scfa.scfa_cache4_append(k, v, torch.arange(P * 16, dtype=torch.int32, device="cuda"), p["cache"], 16)
        p["q"][::2, 0, 7] = bad
        o, lse, ws = run_attn(scfa, p)
        assert scfa.scfa_get_device_status(ws) == 0
        spoilt = torch.zeros_like(lse, dtype=torch.bool)
        spoilt[::2, 0] = True
        none = (p["vis"] == 0)[:, None].expand_as(lse)  # a row that sees no key has nothing to spoil
        assert torch.equal(torch.isnan(lse), spoilt & ~none)
        assert torch.equal(torch.isnan(o), (spoilt & ~none)[..., None].expand_as(o))
        assert torch.all(lse[none] == -torch.inf) and not o[none].any()
        assert torch.isfinite(lse[~none & ~spoilt]).all() and torch.isfinite(o).all(-1)[~none & ~spoilt].all()


def _far_problem(scfa, news, dt, D, by, far_keys):
    """Scores of about +-by: one key of each request is nearest to the queries, the others a quarter of its score or more away."""
    p = attn_problem(scfa, 19, [0] * len(news), news, 4, 2, D, 16, dt)
    n = 40
    p["table"] = i32(np.arange(3 * len(news)).reshape(len(news), 3))
    cache = noise_cache(5, 3 * len(news), 2, D, 16)
    g = np.random.default_rng(int(sum(news)))
    u = rand(6, (1, 2, D), torch.float32).cuda()
    w = torch.tensor(g.uniform(0.3, 0.74, (len(news), 48)), device="cuda", dtype=torch.float32)
    best = g.integers(0, n, len(news))
    for r, b in enumerate(best):
        w[r, b] = 1.0
    if far_keys:  # all scores are far below zero, the nearest key's the least so
        w = -1.3 + w
    rows = []
    for r in range(len(news)):
        k = (w[r, :, None, None] * u).to(dt)
        v = rand(40 + r, (48, 2, D), dt).cuda()
        scfa.scfa_cache4_append(k, v, i32(np.arange(48) + 48 * r), cache, 16)
        rows.append((oc.values(dbl(k))[:n], oc.values(dbl(v))[:n]))
    p["q"] = (u.repeat_interleave(2, 1) * 0.37).to(dt).expand(sum(news), -1, -1).contiguous()
    p["vis"].fill_(n)
    top = float(np.abs(rows[0][0][best[0], 0] @ dbl(p["q"])[0, 0]))
    return {**p, "cache": cache, "rows": rows, "scale": by / top}, best


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [9, 7], [20, 16], [90, 25]])
@pytest.mark.parametrize("dt,D", [(BF, 64), (HF, 128)])
@pytest.mark.parametrize("by", [2.0 ** 22, 2.0 ** 30, 2.0 ** 60, 2.0 ** 95])
@pytest.mark.parametrize("far_keys", [False, True])
def test_attn_scores_that_fp32_can_hardly_tell_apart(scfa, news, dt, D, by, far_keys):
    """Scores past 2^24 in either direction: steps of fp32 there are whole softmax widths, but the nearest key, whose score
    is a fifth apart, has all the weight: lse is its score, within the error of a score that check_rows derives, and o its
    value, but for the rounding of one weight to fp16 (2^-11), exp2 and the sums (2^-18) and that of o."""
    p, best = _far_problem(scfa, news, dt, D, by, far_keys)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    at, uo = 0, 2.0 ** -8 if dt is BF else 2.0 ** -11
    for r, new in enumerate(news):
        k, v = (np.repeat(x, 2, 1) for x in p["rows"][r])
        q = dbl(p["q"][at:at + new])
        s = np.einsum("thd,lhd->thl", q, k) * p["scale"]
        order = np.sort(s, -1)
        assert np.all(s.argmax(-1) == best[r]) and np.all(order[..., -1] - order[..., -2] > 0.15 * np.abs(order[..., -1]))
        sg, qg = np.abs(k).reshape(len(k), 4, -1, 32).max(-1) / 6, np.abs(q).reshape(new, 4, -1, 32).sum(-1)
        e = (D / 8 + 4) * 2.0 ** -23 * 15 * p["scale"] * np.einsum("thg,lhg->thl", qg, sg).max(-1) + 2.0 ** -20 * np.abs(s).max(-1)
        assert np.all(np.abs(dbl(lse[at:at + new]) - s.max(-1)) <= e + 2.0 ** -18 * np.abs(s.max(-1)))
        want = v[best[r]]
        assert np.all(np.abs(dbl(o[at:at + new]) - want) <= (uo + 2.0 ** -11 + 2.0 ** -18) * np.abs(want))
        at += new


def test_status_before_the_first_step(scfa):
    """Of a new cache, of one whose step is only captured, and of one whose first step was refused: 0, in memory that held something else."""
    from sparse_causal_flash_gb300.cache import KVCache4
    size = dict(R=2, n_pages=8, Hq=4, Hkv=2, D=64, max_len=64, max_tokens=16, page_size=16)
    q, kv, new = rand(1, (9, 4, 64)).cuda(), rand(2, (9, 4, 64)).cuda(), i32([5, 4])
    c = KVCache4(**size)
    for ws in (c.ws_plan, c.ws_attn):
        ws.fill_(7)
    torch.cuda.synchronize()
    del c, ws  # the allocator gives the next one the same memory
    c = KVCache4(**size)
    assert c.status() == 0
    g = c.capture(q, kv[:, :2], kv[:, 2:], new, 0.125)
    assert c.status() == 0
    with pytest.raises(ValueError):
        c.step(q.float(), kv[:, :2], kv[:, 2:], new, 0.125)
    assert c.status() == 0
    g.replay()
    assert c.status() == 0 and c.len.tolist() == [5, 4]


@pytest.mark.parametrize("new", [1, 20])
def test_attn_the_longest_request(scfa, new):
    """2^31 - 256 positions, all but the last pages one page of zero keys: the last visible key outweighs them (e^60 to
    2^31), those behind it would outweigh it."""
    D, ps, L = 64, 16, 2 ** 31 - 256
    k = torch.zeros((64, 1, D), dtype=BF)
    v = rand(2, (64, 1, D))
    q = rand(3, (1, 2, D)).repeat(new, 1, 1)
    q[:, 1] = q[:, 0]
    scale = 0.125
    one = (60 / scale / (q[0, 0].double() @ q[0, 0].double()) * q[0, 0].double()).to(BF)  # a score of about 60
    k[48 + 10, 0], k[48 + 11:, 0] = one, 2 * one
    cache = noise_cache(1, 4, 1, D, ps)
    scfa.scfa_cache4_append(k.cuda(), v.cuda(), torch.arange(64, dtype=torch.int32, device="cuda"), cache, ps)
    table = torch.zeros((1, L // ps), dtype=torch.int32, device="cuda")
    table[0, -1] = 3
    p = dict(q=q.cuda().contiguous(), cache=cache, ps=ps, table=table, q_start=i32([0, new]), vis=i32([L - 5] * new),
             scale=scale, dt=BF)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    kk, vv = oc.values(dbl(k))[48:59], oc.values(dbl(v))[48:59]
    assert np.all(np.abs(kk[10, 0] @ dbl(q[0, 0]) * scale - 60) < 10)
    check_rows(dbl(p["q"]), kk, vv, [11] * new, scale, o, lse, BF)


def test_expanded_rows_are_read_but_not_written(scfa):
    """Inputs may repeat a row by a stride of 0; outputs may not."""
    N, H, D, ps = 20, 2, 64, 16
    row, cache = rand(1, (1, H, D)).cuda(), noise_cache(2, 2, H, D, ps)
    k, v, slot = row.expand(N, -1, -1), row[:, :1].expand(N, H, -1), torch.arange(N, dtype=torch.int32, device="cuda")
    scfa.scfa_cache4_append(k, v, slot, cache, ps)
    ko, vo = (torch.full((N, H, D), 3.0, dtype=BF, device="cuda") for _ in "kv")
    scfa.scfa_cache4_read(cache, ps, slot, ko, vo)
    assert np.array_equal(dbl(ko), oc.values(dbl(k))) and np.array_equal(dbl(vo), oc.values(dbl(v)))
    for bad in (dict(k_out=ko[:1].expand(N, -1, -1)), dict(v_out=vo[:, :1].expand(-1, H, -1))):
        with pytest.raises(scfa.ScfaError):
            scfa.scfa_cache4_read(cache, ps, slot, **{**dict(k_out=ko, v_out=vo), **bad})
    q = rand(3, (1, 2 * H, D)).cuda().expand(N, -1, -1)
    p = dict(q=q, cache=cache, ps=ps, table=i32([[0, 1]]), q_start=i32([0, N]), vis=i32(range(1, N + 1)), scale=0.125, dt=BF)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    check_rows(dbl(q), dbl(ko), dbl(vo), list(range(1, N + 1)), 0.125, o, lse, BF)
    with pytest.raises(scfa.ScfaError):
        run_attn(scfa, p, o=o[:1].expand(N, -1, -1))


def test_a_cache_keeps_the_index_of_its_device(scfa):
    """"cuda" names the current device at every call; the cache stays where it was made."""
    from sparse_causal_flash_gb300.cache import KVCache4
    for device in ("cuda", torch.device("cuda"), torch.device("cuda", 0)):
        c = KVCache4(2, 4, 4, 2, 64, max_len=32, max_tokens=4, device=device)
        assert c.device == c.cache.device == torch.device("cuda", 0)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 2], [40, 9, 20]])
def test_attn_in_place_of_its_queries(scfa, news):
    """o may be q itself: a row's queries have been read by all that need them when its o is written."""
    p = attn_problem(scfa, 23, [900, 5000, 40], news, 8, 2, 64, 64, BF)
    o, lse, _ = run_attn(scfa, p)
    for _ in range(5):
        q = p["q"].clone()
        o2, lse2, _ = run_attn(scfa, {**p, "q": q}, o=q)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [1, 4, 20, 70])
@pytest.mark.parametrize("by", [2.0 ** 30, -2.0 ** 95])
def test_attn_far_scores_of_requests_that_are_cut(scfa, new, by):
    """The same over so many keys that every request's parts are joined: pages of one row each, one page nearest."""
    D, L, ps, Hq = 64, 40000, 16, 2
    u = rand(6, (1, 1, D), torch.float32)
    near = 777 if by > 0 else 1234  # its page
    w = torch.full((2, ps, 1, 1), 0.5 if by > 0 else 1.0)
    w[1] = 1.0 if by > 0 else 0.5
    k, v = (w * u).to(BF).flatten(0, 1), rand(7, (2, 1, 1, D)).expand(2, ps, 1, D).flatten(0, 1)
    cache = noise_cache(1, 2, 1, D, ps)
    scfa.scfa_cache4_append(k.cuda(), v.cuda(), torch.arange(2 * ps, dtype=torch.int32, device="cuda"), cache, ps)
    table = torch.zeros((3, L // ps), dtype=torch.int32, device="cuda")
    table[:, near] = 1
    q = (u * 0.37 * np.sign(by)).to(BF).expand(3 * new, Hq, D).contiguous().cuda()
    kk, vv = oc.values(dbl(k))[::ps], oc.values(dbl(v))[::ps]
    scale = abs(by) / abs(float(kk[1, 0] @ dbl(q)[0, 0]))
    p = dict(q=q, cache=cache, ps=ps, table=table, q_start=i32(np.arange(4) * new), vis=i32([L] * 3 * new), scale=scale, dt=BF)
    o, lse, ws = run_attn(scfa, p)
    assert scfa.scfa_get_device_status(ws) == 0
    s = kk[:, 0] @ dbl(q)[0, 0] * scale
    assert s[1] - s[0] > 0.3 * abs(s[1])
    sg, qg = np.abs(kk[:, 0]).reshape(2, -1, 32).max(-1) / 6, np.abs(dbl(q)[0, 0]).reshape(-1, 32).sum(-1)
    e = (D / 8 + 4) * 2.0 ** -23 * 15 * scale * (sg @ qg).max() + 2.0 ** -20 * np.abs(s).max()  # as check_rows derives it
    assert np.all(np.abs(dbl(lse) - s[1]) <= e + 2.0 ** -18 * abs(s[1]) + np.log(ps))
    # sixteen equal weights, each rounded to fp16 once
    assert np.all(np.abs(dbl(o) - vv[1]) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.abs(vv[1]))


def test_a_request_that_is_released_twice_gives_its_pages_back_once(scfa):
    from sparse_causal_flash_gb300.cache import KVCache4
    c = KVCache4(2, 6, 4, 2, 64, max_len=64, max_tokens=60, page_size=16)
    q, kv = rand(1, (50, 4, 64)).cuda(), rand(2, (50, 4, 64)).cuda()
    c.step(q, kv[:, :2], kv[:, 2:], i32([33, 17]), 0.125)
    assert c.status() == 0 and int(c.n_free) == 1
    for _ in range(2):
        c.release(0)
        assert int(c.n_free) == 4 and c.len.tolist() == [0, 17]
    held = c.table[1, :2].tolist()
    assert sorted(c.free[:4].tolist() + held) == list(range(6))
    with pytest.raises(IndexError):
        c.release(2)
    k, v = c.rows(0)
    assert k.shape == v.shape == (0, 2, 64)
