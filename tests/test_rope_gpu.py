"""Rotary positions, their norm and their gradients on the GPU against the float64 oracle, and the steps that use them.

Bounds, u = finfo.eps / 2 of the rows' type (2^-8 bf16, 2^-11 fp16), e = 2^-24:
- a row's norm: sixteen squares a thread and three shuffles, so the sum of squares is off by 19 e of itself, its root's
  reciprocal by half of that and 2^-22 of its own; with two products less than 2^-19 of a value.
- an angle is exact up to its rounding to fp32 (2^-25 of half a turn, 2^-23 radians); the hardware's sine and cosine are
  within 2^-20 over half a turn. A turned value a cos - b sin is then within 2^-19 (|a| + |b|) factor, with the fp32
  products and their sum, and the norm's share as much again: 2^-18 in all, then the output's rounding u.
- a gradient with a norm adds a mean over the row: products within 2^-18 of their magnitudes, so an element is within
  2^-17 r (|g w| + |n| mean|g w n|) of magnitudes taken after the turn (each at most |a| + |b| of its pair).
- a weight's gradient sums |g n| over all rows: 2^-17 of the magnitudes, and at most rows / 2 additions in a row's
  thread, each rounding by e of a partial sum."""
import numpy as np
import pytest
import torch

from oracle import rope as orope

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module")
def scfa():
    import sparse_causal_flash_gb300 as s
    s.load()
    return s


def dbl(t):
    return t.detach().double().cpu().numpy()


def rand(seed, shape, dt, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp(spread * torch.randn(shape[-1:], generator=g))
    return x.to(dt).cuda()


def half_step(x, dt):
    """What rounding to dt moves a value by: u of it, and below the normal numbers half the smallest number."""
    f = torch.finfo(dt)
    return np.maximum(np.abs(x) * f.eps / 2, f.tiny * f.eps / 2)


def pair_sum(x, rot, interleaved):
    """|a| + |b| at both channels of each pair, |x| elsewhere."""
    y = np.abs(x)
    a, b = orope.pairs(rot, interleaved)
    s = y[..., a] + y[..., b]
    y[..., a] = y[..., b] = s
    return y


def check_fwd(got, x, pos, freq, interleaved, factor, w, dt):
    ref = orope.forward(x, pos, freq, interleaved, factor, w, EPS)
    n = x if w is None else orope.norm(x, w, EPS)
    bound = half_step(ref, dt) * (1 + 2.0 ** -10) + 2.0 ** -18 * max(1.0, abs(factor)) * pair_sum(n, 2 * freq.size, interleaved)
    err = np.abs(dbl(got) - ref)
    assert np.all(err <= bound), float((err / bound).max())


def check_bwd(got, dw, dy, x, pos, freq, interleaved, factor, w, dt):
    ref, ref_w = orope.backward(dy, pos, freq, interleaved, factor, x, w, EPS)
    g = pair_sum(dy, 2 * freq.size, interleaved) * max(1.0, abs(factor))  # at least |g|
    if w is None:
        bound = 2.0 ** -18 * g
    else:
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        n = np.abs(x * r)
        gw = g * np.abs(w)
        bound = 2.0 ** -17 * r * (gw + n * np.mean(gw * n, -1, keepdims=True))
        rows = x.shape[0] * x.shape[1]
        limit = (2.0 ** -17 + rows / 2 * 2.0 ** -24) * (g * n).sum((0, 1))
        assert np.all(np.abs(dbl(dw) - ref_w) <= limit)
    bound = bound + half_step(ref, dt) * (1 + 2.0 ** -10)
    err = np.abs(dbl(got) - ref)
    assert np.all(err <= bound), float((err / bound).max())


def freqs(rot):
    return 10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


# (N, Hq, Hkv, D, rot, interleaved, norm, factor)
CASES = [(1, 1, 0, 64, 64, False, False, 1.0), (1, 1, 1, 128, 128, False, True, 1.0), (3, 5, 1, 64, 64, True, True, 1.2),
         (7, 8, 2, 128, 2, False, True, 1.0), (5, 3, 3, 64, 62, False, True, 1.0), (5, 3, 3, 128, 126, False, False, 0.5),
         (33, 4, 4, 128, 96, False, True, 1.0), (64, 12, 4, 64, 48, True, False, -1.0), (257, 6, 2, 64, 32, False, True, 1.0),
         (130, 32, 8, 128, 128, False, True, 1.3), (19, 7, 1, 128, 22, True, True, 1.0), (11, 2, 2, 64, 0, False, True, 1.0),
         (2500, 12, 4, 64, 64, False, True, 1.0), (1700, 16, 4, 128, 64, True, False, 1.0), (9000, 1, 0, 64, 20, False, True, 1.0)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,il,norm,factor", CASES)
def test_rows_and_gradients(scfa, N, Hq, Hkv, D, rot, il, norm, factor, dt):
    f = freqs(rot)
    table = scfa.rope_table(f)
    pos = torch.as_tensor(np.random.default_rng(N).integers(-50, 300000, N), dtype=torch.int32).cuda()
    pos[0] = 2 ** 31 - 1
    pos[-1] = -2 ** 31 if N > 1 else 0
    # a fused projection's views in, gradients of one out
    qkv = rand(N + D, (N, Hq + 2 * Hkv, D), dt, 0.7)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv] if Hkv else None
    w = [1 + 0.3 * rand(5 + i, (D,), torch.float32) if norm and (i == 0 or Hkv) else None for i in range(2)]
    out = torch.full_like(qkv, 9.0)
    qo, ko = out[:, :Hq], out[:, Hq:Hq + Hkv] if Hkv else None
    scfa.scfa_rope_fwd(q, k, pos, table, qo, ko, il, factor, *w, EPS)
    p = pos.cpu().numpy().astype(np.float64)
    wn = [None if x is None else dbl(x) for x in w]
    check_fwd(qo, dbl(q), p, f, il, factor, wn[0], dt)
    if Hkv:
        check_fwd(ko, dbl(k), p, f, il, factor, wn[1], dt)
        assert bool((out[:, Hq + Hkv:] == 9).all())
    dy = rand(N + 3, (N, Hq + Hkv, D), dt)
    dq, dk = dy[:, :Hq], dy[:, Hq:] if Hkv else None
    grad = torch.full_like(qkv, 9.0)
    gq, gk = grad[:, :Hq], grad[:, Hq:Hq + Hkv] if Hkv else None
    kw, dw = {}, [None, None]
    if norm:
        dw = [torch.empty(D, device="cuda"), torch.empty(D, device="cuda") if Hkv else None]
        kw = dict(q=q, k=k, wq=w[0], wk=w[1], eps=EPS, dwq=dw[0], dwk=dw[1],
                  ws=scfa.workspace(scfa.rope_workspace_size(N, Hq, Hkv, D)))
    scfa.scfa_rope_bwd(dq, dk, pos, table, gq, gk, il, factor, **kw)
    check_bwd(gq, dw[0], dbl(dq), dbl(q), p, f, il, factor, wn[0], dt)
    if Hkv:
        check_bwd(gk, dw[1], dbl(dk), dbl(k), p, f, il, factor, wn[1], dt)
        assert bool((grad[:, Hq + Hkv:] == 9).all())
    if norm:  # the same bits again
        first = grad.clone(), [None if x is None else x.clone() for x in dw]
        scfa.scfa_rope_bwd(dq, dk, pos, table, gq, gk, il, factor, **kw)
        assert torch.equal(first[0], grad)
        assert all(a is None or torch.equal(a, b) for a, b in zip(first[1], dw))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot,il", [(128, False), (96, True), (40, False)])
def test_more_rows_than_run_at_once(scfa, rot, il, norm):
    """Units of four heads, the last with one; in place; the tokens end inside; a gradient without a norm as well."""
    N, n, Hq, Hkv, D = 15013, 14990, 5, 1, 128
    x, k = rand(1, (N, Hq, D), BF, 0.7), rand(2, (N, Hkv, D), BF, 0.7)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 7 - 5000
    w = [1 + 0.3 * rand(5 + i, (D,), torch.float32) if norm else None for i in range(2)]
    f, p, table = freqs(rot), pos[:n].cpu().numpy().astype(np.float64), scfa.rope_table(freqs(rot))
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    y, z = x.clone(), k.clone()
    scfa.scfa_rope_fwd(y, z, pos, table, y, z, il, 1.2, *w, EPS, count)
    for got, was, wi in ((y, x, w[0]), (z, k, w[1])):
        check_fwd(got[:n], dbl(was[:n]), p, f, il, 1.2, None if wi is None else dbl(wi), BF)
        assert torch.equal(got[n:], was[n:])
    if not norm:
        scfa.scfa_rope_bwd(y.copy_(x), None, pos, table, y, None, il, 1.2, count=count)
        check_bwd(y[:n], None, dbl(x[:n]), None, p, f, il, 1.2, None, BF)
        assert torch.equal(y[n:], x[n:])


@pytest.mark.parametrize("rot,il", [(128, False), (128, True), (40, False)])
def test_gradients_of_more_rows_than_run_at_once(scfa, rot, il):
    """A CTA takes several units of two heads; the last head stands alone; the tokens end inside a unit's row."""
    N, n, Hq, Hkv, D = 20011, 19990, 5, 1, 128
    x, dy = rand(1, (N, Hq, D), BF, 0.7), rand(2, (N, Hq, D), BF)
    k, dk = rand(3, (N, Hkv, D), BF, 0.7), rand(4, (N, Hkv, D), BF)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 3 - 5000
    w = [1 + 0.3 * rand(5 + i, (D,), torch.float32) for i in range(2)]
    f, p = freqs(rot), pos[:n].cpu().numpy().astype(np.float64)
    gq, gk, dw = torch.full_like(dy, 9.0), torch.full_like(dk, 9.0), torch.empty(2, D, device="cuda")
    scfa.scfa_rope_bwd(dy, dk, pos, scfa.rope_table(f), gq, gk, il, q=x, k=k, wq=w[0], wk=w[1], eps=EPS, dwq=dw[0], dwk=dw[1],
                       ws=scfa.workspace(scfa.rope_workspace_size(N, Hq, Hkv, D)),
                       count=torch.tensor([n], dtype=torch.int32, device="cuda"))
    check_bwd(gq[:n], dw[0], dbl(dy[:n]), dbl(x[:n]), p, f, il, 1.0, dbl(w[0]), BF)
    check_bwd(gk[:n], dw[1], dbl(dk[:n]), dbl(k[:n]), p, f, il, 1.0, dbl(w[1]), BF)
    assert bool((gq[n:] == 9).all()) and bool((gk[n:] == 9).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot", [64, 38])
def test_in_place_and_other_strides(scfa, rot, norm):
    """[B][H][T][D] rows as T tokens of B H heads, turned in place; positions that are shared by all heads."""
    B, H, T, D = 2, 3, 37, 64
    f = freqs(rot)
    x = rand(1, (B, H, T, D), BF)
    rows = x.view(B * H, T, D).transpose(0, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w = 1 + 0.3 * rand(5, (D,), torch.float32) if norm else None
    before = dbl(rows)
    scfa.scfa_rope_fwd(rows, None, pos, scfa.rope_table(f), rows, None, wq=w, eps=EPS)
    check_fwd(rows, before, np.arange(T), f, False, 1.0, None if w is None else dbl(w), BF)
    dy = rand(2, (B, H, T, D), BF)
    g = dy.view(B * H, T, D).transpose(0, 1)
    before_g, x0 = dbl(g), torch.as_tensor(before).to(BF).cuda()
    kw, dw = {}, None
    if norm:
        dw = torch.empty(D, device="cuda")
        kw = dict(q=x0, wq=w, eps=EPS, dwq=dw, ws=scfa.workspace(scfa.rope_workspace_size(T, B * H, 0, D)))
    scfa.scfa_rope_bwd(g, None, pos, scfa.rope_table(f), g, None, **kw)
    check_bwd(g, dw, before_g, before, np.arange(T), f, False, 1.0, None if w is None else dbl(w), BF)


def test_a_turn_there_and_back(scfa):
    x = rand(1, (50, 4, 128), HF)
    pos = torch.arange(0, 50 * 7919, 7919, dtype=torch.int32, device="cuda")
    table, y = scfa.rope_table(freqs(128)), torch.empty_like(x)
    scfa.scfa_rope_fwd(x, None, pos, table, y, None)
    scfa.scfa_rope_bwd(y, None, pos, table, y, None)
    # two roundings of values of at most |a| + |b|, which the second turn may mix, and the two turns' own errors
    bound = pair_sum(dbl(x), 128, False) * (2 * 2.0 ** -11 + 2.0 ** -17) + 2.0 ** -24
    assert np.all(np.abs(dbl(y) - dbl(x)) <= bound * 1.01)


def test_count_keeps_the_rows_behind(scfa):
    N, Hq, Hkv, D = 70, 4, 2, 64
    f, table = freqs(D), scfa.rope_table(freqs(D))
    x = rand(1, (N, Hq + Hkv, D), BF)
    x[40:] = float("nan")
    dy = rand(2, (N, Hq + Hkv, D), BF)
    dy[40:] = float("nan")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    w = [1 + 0.3 * rand(5 + i, (D,), torch.float32) for i in range(2)]
    count = torch.tensor([40], dtype=torch.int32, device="cuda")
    for n, c in ((40, count), (0, torch.zeros_like(count)), (0, torch.full_like(count, -5))):
        out = torch.full_like(x, 7.0)
        scfa.scfa_rope_fwd(x[:, :Hq], x[:, Hq:], pos, table, out[:, :Hq], out[:, Hq:], wq=w[0], wk=w[1], eps=EPS, count=c)
        assert bool((out[n:] == 7).all())
        check_fwd(out[:n, :Hq], dbl(x[:n, :Hq]), np.arange(n), f, False, 1.0, dbl(w[0]), BF)
        dw = [torch.empty(D, device="cuda") for _ in range(2)]
        g = torch.full_like(x, 7.0)
        scfa.scfa_rope_bwd(dy[:, :Hq], dy[:, Hq:], pos, table, g[:, :Hq], g[:, Hq:], q=x[:, :Hq], k=x[:, Hq:], wq=w[0], wk=w[1],
                           eps=EPS, dwq=dw[0], dwk=dw[1], count=c, ws=scfa.workspace(scfa.rope_workspace_size(N, Hq, Hkv, D)))
        assert bool((g[n:] == 7).all())
        for i, sl in enumerate((slice(0, Hq), slice(Hq, None))):
            check_bwd(g[:n, sl], dw[i], dbl(dy[:n, sl]), dbl(x[:n, sl]), np.arange(n), f, False, 1.0, dbl(w[i]), BF)
    big = torch.full_like(count, 1 << 30)  # clamped to N
    out = torch.zeros_like(x)
    scfa.scfa_rope_fwd(x[:40], None, pos[:40], table, out[:40], None, count=big)
    check_fwd(out[:40], dbl(x[:40]), np.arange(40), f, False, 1.0, None, BF)


def test_values_that_are_not_finite_stay_in_their_rows(scfa):
    x = rand(1, (9, 2, 64), BF)
    x[4, 1, 3] = float("inf")
    y = torch.empty_like(x)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    scfa.scfa_rope_fwd(x, None, pos, scfa.rope_table(freqs(64)), y, None, wq=w)
    ok = torch.isfinite(y).all(-1)
    assert not ok[4, 1] and int(ok.sum()) == 17
    z = torch.zeros_like(x)  # rows of zeros: the norm's eps keeps them
    scfa.scfa_rope_fwd(z, None, pos, scfa.rope_table(freqs(64)), y, None, wq=w)
    assert not y.any()


def test_keys_and_their_output_come_together(scfa):
    x, pos, table = rand(1, (3, 2, 64), BF), torch.zeros(3, dtype=torch.int32, device="cuda"), scfa.rope_table(freqs(64))
    for f in (scfa.scfa_rope_fwd, scfa.scfa_rope_bwd):
        with pytest.raises(ValueError, match="together"):
            f(x, x, pos, table, torch.empty_like(x), None)
        with pytest.raises(ValueError, match="together"):
            f(x, None, pos, table, torch.empty_like(x), torch.empty_like(x))


def test_no_tokens(scfa):
    e = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    p = torch.empty(0, dtype=torch.int32, device="cuda")
    table, w, dw = scfa.rope_table(freqs(64)), torch.ones(64, device="cuda"), torch.full((64,), 5.0, device="cuda")
    scfa.scfa_rope_fwd(e, None, p, table, e, None)
    scfa.scfa_rope_bwd(e, None, p, table, e, None, q=e, wq=w, dwq=dw, ws=scfa.workspace(scfa.rope_workspace_size(0, 4, 0, 64)))
    assert not dw.any()


def test_offsets_past_32_bits(scfa):
    """The last rows of 2.4 billion elements."""
    N, H, D = 300000, 64, 128
    x = torch.zeros((N, H, D), dtype=BF, device="cuda")
    tail = rand(1, (3, H, D), BF)
    x[-3:] = tail
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    f = freqs(D)
    scfa.scfa_rope_fwd(x, None, pos, scfa.rope_table(f), x, None)
    check_fwd(x[-3:], dbl(tail), np.arange(N - 3, N), f, False, 1.0, None, BF)
    assert not x[:-3].any()


def test_another_stream_and_a_graph(scfa):
    N, H, D = 40, 4, 64
    x, y = rand(1, (N, H, D), BF), torch.zeros((N, H, D), dtype=BF, device="cuda")
    pos, f = torch.arange(N, dtype=torch.int32, device="cuda"), freqs(D)
    table, w, dw = scfa.rope_table(f), torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    ws = scfa.workspace(scfa.rope_workspace_size(N, H, 0, D))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    scfa.scfa_rope_fwd(x, None, pos, table, y, None, wq=w, eps=EPS, stream=st)
    st.synchronize()
    check_fwd(y, dbl(x), np.arange(N), f, False, 1.0, np.ones(D), BF)
    dy, g = rand(2, (N, H, D), BF), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scfa.scfa_rope_bwd(dy, None, pos, table, g, None, q=x, wq=w, eps=EPS, dwq=dw, ws=ws)
    for seed in (2, 3):
        dy.copy_(rand(seed, (N, H, D), BF))
        graph.replay()
        torch.cuda.synchronize()
        check_bwd(g, dw, dbl(dy), dbl(x), np.arange(N), f, False, 1.0, np.ones(D), BF)


# ---------------------------------------------------------------- the steps that turn their rows
@pytest.mark.parametrize("mode", ["dense", "qk", "hash"])
def test_step_with_rope(scfa, mode):
    """A step with a rope is the step on turned rows, its gradients turned back: bit for bit where the step's are."""
    from sparse_causal_flash_gb300.pipeline import Step
    from sparse_causal_flash_gb300.rope import Rope
    B, H, T, D = 1, 2, 300, 64
    q, k, v, do = (rand(i, (B, H, T, D), BF) for i in range(4))
    rope, kw, ctor = Rope(48, interleaved=True), {}, {}
    m = {"dense": scfa.MODE_DENSE, "qk": scfa.MODE_QK, "hash": scfa.MODE_HASH}[mode]
    q_pos = k_pos = torch.arange(T).expand(B, H, T)
    if mode == "qk":
        g = torch.Generator().manual_seed(0)
        q_pos, k_pos = (torch.stack([torch.sort(torch.randperm(2 * T, generator=g)[:T])[0] for _ in range(H)])[None].to(torch.int32)
                        for _ in range(2))
        q_pos[0, 1, -5:] = -1
        k_pos[0, 0, -9:] = 2 ** 31 - 1
        kw = dict(q_idx=q_pos.cuda(), k_idx=k_pos.cuda())
    if mode == "hash":
        ctor, kw = dict(n_buckets=4), dict(R=rand(9, (D, 2), BF))
    a = Step(m, B, H, T, T, D, rope=rope, **ctor).run(q, k, v, do, 0.125, **kw)
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    for x, y, p in ((q, qr, q_pos), (k, kr, k_pos)):
        rope.fwd(x.view(-1, 1, D), None, p.reshape(-1).to(torch.int32).cuda(), y.view(-1, 1, D), None)
    b = Step(m, B, H, T, T, D, **ctor).run(qr, kr, v, do, 0.125, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse) and torch.equal(a.dv, b.dv)
    for x, y, p in ((b.dq, a.dq, q_pos), (b.dk, a.dk, k_pos)):
        ref = torch.empty_like(x)
        rope.bwd(x.view(-1, 1, D), None, p.reshape(-1).to(torch.int32).cuda(), ref.view(-1, 1, D), None)
        # dq sums key tiles in the order they come: a rounding of dq before the turn and one behind it
        assert float((ref.double() - y.double()).abs().max()) <= (0 if y is a.dk else 4 * 2.0 ** -8 * float(ref.abs().max()))


def test_host_pipeline_with_rope(scfa):
    from sparse_causal_flash_gb300.pipeline import HostPipeline, Step
    from sparse_causal_flash_gb300.rope import Rope
    B, H, T, D = 1, 2, 200, 64
    rope = Rope(64)
    hp = HostPipeline(scfa.MODE_DENSE, B, H, T, T, D, rope=rope)
    st = Step(scfa.MODE_DENSE, B, H, T, T, D, rope=rope)
    for i in range(5):
        ins = {n: rand(10 * i + j, (B, H, T, D), BF).cpu().pin_memory() for j, n in enumerate(("q", "k", "v", "do"))}
        outs = [torch.empty((B, H, T, D), dtype=BF).pin_memory(), torch.empty((B, H, T)).pin_memory()] + \
            [torch.empty((B, H, T, D), dtype=BF).pin_memory() for _ in range(3)]
        hp.submit(ins, outs, 0.125)
        hp.synchronize()
        st.run(*(ins[n].cuda() for n in ("q", "k", "v", "do")), 0.125)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], st.o.cpu()) and torch.equal(outs[1], st.lse.cpu()) and torch.equal(outs[3], st.dk.cpu())


def test_cache_steps_with_rope_and_norm(scfa):
    """Serving steps that turn their rows are the steps on turned rows."""
    from sparse_causal_flash_gb300.cache import KVCache4
    from sparse_causal_flash_gb300.rope import Rope
    Hq, Hkv, D = 4, 2, 64
    rope, w = Rope(64, scaling="parts", stretch=4.0, trained=2048), [1 + 0.2 * rand(i, (D,), torch.float32) for i in range(2)]
    args = (2, 16, Hq, Hkv, D, 96, 80)
    a = KVCache4(*args, page_size=16, rope=rope, wq=w[0], wk=w[1])
    b = KVCache4(*args, page_size=16)
    base = torch.tensor([5000, 90000], device="cuda")
    done = torch.zeros(2, dtype=torch.int64, device="cuda")
    for i, new in enumerate(([50, 30], [1, 1], [3, 0])):
        x = rand(20 + i, (sum(new), Hq + 2 * Hkv, D), BF)
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        pos = torch.cat([base[r] + done[r] + torch.arange(new[r], device="cuda") for r in range(2)]).to(torch.int32)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        o, lse = a.step(q, k, v, n, 0.125, pos=pos)
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        rope.fwd(q, k, pos, qr, kr, *w)
        o2, lse2 = b.step(qr, kr, v, n, 0.125)
        assert a.status() == 0 and b.status() == 0
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        done += n
    assert all(torch.equal(x, y) for x, y in zip(a.rows(1), b.rows(1)))
    with pytest.raises(ValueError, match="positions"):
        a.step(q, k, v, n, 0.125)
    with pytest.raises(ValueError, match="positions"):
        b.step(q, k, v, n, 0.125, pos=pos)
    assert torch.equal(a.len, b.len)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("N,H", [(6, 3), (9000, 5)])
@pytest.mark.parametrize("D,rot,il", [(64, 0, False), (64, 32, False), (128, 96, False), (64, 20, False), (128, 126, False),
                                      (64, 0, True), (64, 32, True), (128, 22, True)])
def test_channels_that_do_not_turn_pass_as_they_are(scfa, D, rot, il, N, H, dt):
    """Bit for bit, whatever stands in the channels beside them: infinities, NaN, zeros with a sign."""
    x = rand(rot + H, (N, H, D), dt)
    x[..., rot:] = torch.tensor([float("inf"), 1.5, -0.0, float("nan"), -2.0, 0.0, float("-inf"), 3.0], dtype=dt,
                                device="cuda").repeat(D // 8)[rot:]
    x[1::2, :, rot:] = x[1::2, :, rot:].flip(-1)
    x[-1, :, rot:] = torch.roll(x[0, :, rot:], 1, -1)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 3 + 1
    f, table = freqs(rot), scfa.rope_table(freqs(rot))
    for call, sign in ((scfa.scfa_rope_fwd, 1), (scfa.scfa_rope_bwd, -1)):
        y = torch.zeros_like(x)
        call(x, None, pos, table, y, None, il, 1.3)
        was, got = x[..., rot:], y[..., rot:]
        assert torch.equal(torch.isnan(was), torch.isnan(got))
        same = ~torch.isnan(was)
        assert torch.equal(was.view(torch.int16)[same], got.view(torch.int16)[same])
        if rot:
            check_fwd(y[..., :rot], dbl(x[..., :rot]), sign * pos.cpu().numpy().astype(np.float64), f, il, 1.3, None, dt)


@pytest.mark.parametrize("D,rot,il", [(64, 32, False), (128, 126, False), (64, 22, True)])
def test_a_channel_that_does_not_turn_spoils_no_other_weight(scfa, D, rot, il):
    """An infinite gradient in a channel behind `rot`: that channel's dw is not finite, every other is."""
    N, H = 70, 3
    x, dy = rand(1, (N, H, D), BF), rand(2, (N, H, D), BF)
    dy[11, 2, D - 2] = float("inf")
    pos, dw = torch.arange(N, dtype=torch.int32, device="cuda"), torch.empty(D, device="cuda")
    scfa.scfa_rope_bwd(dy, None, pos, scfa.rope_table(freqs(rot)), torch.empty_like(x), None, il, q=x,
                       wq=torch.ones(D, device="cuda"), eps=EPS, dwq=dw, ws=scfa.workspace(scfa.rope_workspace_size(N, H, 0, D)))
    assert torch.isfinite(dw).tolist() == [c != D - 2 for c in range(D)]
