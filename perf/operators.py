"""Cases of the paged 4-bit key/value cache: page planning, append, read and attention.

`own = False` computes each operator in plain torch; `own = True` calls
sparse_causal_flash_gb300. Both work on the same cache bytes.

The cache is a uint8 tensor [pages, kv heads, page_size * (D + D / 16)]. A
page of one head is a run of 16-token tiles. With G = D / 32 groups of 32
channels, a tile holds, in this order,
  K codes   [16 tokens][4 j][G g][4 bytes]        (channels 32 g + 8 j + 0..7)
  V codes   [2 u][8 r][4 w][2 b][G g][2 bytes]    (token 8 u + 2 w + b, channels 32 g + 4 r + 0..3)
  K scales  [16 tokens][G], V scales [16 tokens][G]   (one byte each)
A code is 4 bits, c + 8 with c in -7..7; the low half of a byte comes first.
The eight codes of a K word stand for its channels 0 2 4 6 1 3 5 7, the four
of a V piece for its channels 0 1 2 3. A scale byte b is
(1 + (b & 7) / 8) * 2^((b >> 3) - 15). A value is its code times its scale.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's page bookkeeping for a mid-size batch: latency only
        dict(name="plan decode 48", op="plan", R=48, lo=1, hi=8191, n_lo=1, n_hi=1, ps=64, keep=0.0),
        # admission of prompts whose keys are thinned to 70% (the drop rate of the QK-sparse workloads)
        dict(name="plan prompts 24k keep", op="plan", R=97, lo=0, hi=300, n_lo=1, n_hi=506, ps=16, keep=0.7),
        # one new token of each of 64 requests, K and V as views of a fused projection
        dict(name="append decode 64", op="append", N=64, Hq=32, Hkv=8, D=128, ps=64, dt="bf16", drop=0.0),
        # a prompt chunk of a large prefill
        dict(name="append prompt 16384", op="append", N=16384, Hq=32, Hkv=8, D=128, ps=64, dt="bf16", drop=0.0),
        # 12 heads of 64 channels (the 122M-parameter model's attention), fp16, odd count, dropped keys
        dict(name="append 5003 h12 d64 f16", op="append", N=5003, Hq=12, Hkv=12, D=64, ps=16, dt="f16", drop=0.3),
        # rows brought back for a dense pass over a cached prefix
        dict(name="read 32768", op="read", N=32768, Hkv=8, D=128, ps=64, dt="bf16"),
        dict(name="read 1501 h12 d64 f16", op="read", N=1501, Hkv=12, D=64, ps=32, dt="f16"),
        # single tokens over short answers: latency and the split of little work
        dict(name="attn 8 x 512", op="attn", R=8, lo=1, hi=512, n_lo=1, n_hi=1, Hq=32, Hkv=8, D=128, ps=64, dt="bf16"),
        # one request with a very long context: the long axis is all there is to split
        dict(name="attn 1 x 131072", op="attn", R=1, lo=131072, hi=131072, n_lo=1, n_hi=1, Hq=32, Hkv=8, D=128, ps=128,
             dt="bf16"),
        # a ragged decode batch with as many key heads as query heads (12 heads of 64 channels)
        dict(name="attn 61 ragged h12 d64", op="attn", R=61, lo=0, hi=16384, n_lo=1, n_hi=1, Hq=12, Hkv=12, D=64, ps=64,
             dt="bf16"),
        # a few drafted tokens of each request checked at once, fp16
        dict(name="attn 32 drafts f16", op="attn", R=32, lo=700, hi=15000, n_lo=1, n_hi=7, Hq=32, Hkv=8, D=128, ps=32,
             dt="f16"),
        # two prompt chunks over what is cached of them
        dict(name="attn chunks 500", op="attn", R=2, lo=4000, hi=8000, n_lo=477, n_hi=523, Hq=32, Hkv=8, D=128, ps=64,
             dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "read", "attn", "attn", "attn"))
    ps = rng.choice((16, 32, 64, 128, 256))
    if op == "plan":
        if rng.random() < 0.5:
            return dict(op=op, R=_log(rng, 1, 400), lo=rng.randint(0, 64), hi=_log(rng, 65, 30000), n_lo=1, n_hi=1, ps=ps,
                        keep=0.0)
        R, hi = _log(rng, 1, 96), _log(rng, 2, 506)
        return dict(op=op, R=R, lo=0, hi=_log(rng, 1, 4000), n_lo=rng.randint(0, 1), n_hi=hi, ps=ps,
                    keep=rng.choice((0.0, 0.3, 0.7, 0.8)))
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8, 12 if D == 64 else 8))
    G = rng.choice((1, 1, 2, 4, 5, 8))
    dt = rng.choice(("bf16", "bf16", "f16"))
    if op == "append":
        return dict(op=op, N=_log(rng, 1, 16000), Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, dt=dt, drop=rng.choice((0.0, 0.0, 0.3)))
    if op == "read":
        return dict(op=op, N=_log(rng, 1, 32000), Hkv=Hkv, D=D, ps=ps, dt=dt)
    kind = rng.random()
    if kind < 0.6:  # decode: no more cached bytes than the largest listed case has
        R = _log(rng, 1, 96)
        hi = _log(rng, 30, min(130000, 400000000 // (R * Hkv * (D + D // 16))))
        return dict(op=op, R=R, lo=rng.randint(0, hi), hi=hi, n_lo=1, n_hi=1, Hq=Hkv * G, Hkv=Hkv, D=D, ps=ps, dt=dt)
    if kind < 0.8:  # drafts
        R = _log(rng, 1, 32)
        hi = _log(rng, 30, 15000)
        return dict(op=op, R=R, lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(0, 2), n_hi=rng.randint(2, 8), Hq=Hkv * G,
                    Hkv=Hkv, D=D, ps=ps, dt=dt)
    R = rng.randint(1, 2)  # prompt chunks
    hi = _log(rng, 10, 7000)
    return dict(op=op, R=R, lo=rng.randint(0, hi), hi=hi, n_lo=rng.randint(8, 400), n_hi=rng.randint(400, 500),
                Hq=Hkv * min(G, 4), Hkv=Hkv, D=D, ps=ps, dt=dt)


def _ramp(R, lo, hi):
    """R whole numbers from lo to hi in even steps: their sum is the case's, whatever the seed."""
    return [lo + (hi - lo) * i // max(1, R - 1) for i in range(R)] if R > 1 else [hi]


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the format, in plain torch
def _scale_bits(amax):
    """Scale byte of a group's largest magnitude (in 64 bits: quotients fall on the borders between codes)."""
    t = torch.clamp(amax / torch.full_like(amax, 7.0), 2.0 ** -15, 9216.0)  # a true quotient, not amax * (1 / 7)
    m, e = torch.frexp(t)  # t = m 2^e, 0.5 <= m < 1
    q = torch.round(m * 16.0)  # ties to even; 8..16
    e = torch.where(q == 16, e + 1, e)
    q = torch.where(q == 16, 8, q)
    return ((e.to(torch.int32) + 14) * 8 + q.to(torch.int32) - 8).to(torch.uint8)


def _scale_of(b):
    return ((b.to(torch.int32) << 20) + (112 << 23)).view(torch.float32)


def _quantise(x):
    """[..., D] -> codes 0..15 uint8 [..., G, 32] and scale bytes [..., G]."""
    x = x.double().unflatten(-1, (-1, 32))
    x = torch.where(torch.isnan(x), 0.0, x)
    b = _scale_bits(x.abs().amax(-1))
    c = torch.clamp(torch.round(x / _scale_of(b).double()[..., None]), -7, 7)
    return (c + 8).to(torch.uint8), b


def _pack_k(c):
    """codes [N, H, G, 32] -> bytes [N, H, 4, G, 4]"""
    c = c.unflatten(-1, (4, 4, 2)).transpose(-1, -2).flatten(-2)  # [N,H,G,j,8 positions]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(2, 3)


def _pack_v(c):
    """codes [N, H, G, 32] -> bytes [N, H, 8, G, 2]"""
    c = c.unflatten(-1, (8, 4))  # [N,H,G,r,4]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(2, 3)


def _places(slot, H, D, ps, device):
    """Byte positions in the flat cache of the K codes [N,H,4,G,4], V codes [N,H,8,G,2] and scales [N,H,G] of slots."""
    G = D // 32
    tile = 16 * (D + D // 16)
    ar = lambda n: torch.arange(n, device=device)  # noqa: E731
    page, at = slot // ps, slot % ps
    t = at % 16
    base = ((page[:, None] * H + ar(H)) * (ps // 16) + (at // 16)[:, None]) * tile  # [N,H]
    k = base[..., None] + (t * (D // 2))[:, None, None] + ar(D // 2)
    u, w, b = t // 8, t // 2 % 4, t % 2
    v0 = base + (8 * D + u * 4 * D + w * 4 * G + b * 2 * G)[:, None]
    v = v0[:, :, None, None] + (ar(8) * 16 * G)[:, None] + ar(2 * G)
    ks = base[..., None] + (16 * D + t * G)[:, None, None] + ar(G)
    return k.unflatten(-1, (4, G, 4)), v.unflatten(-1, (G, 2)), ks, ks + 16 * G


def _store(cache, ps, slot, k, v):
    """Rows [N,H,D] into the cache at slots >= 0."""
    H, D = k.shape[1], k.shape[2]
    flat = cache.view(-1)
    kept = slot >= 0
    # a dropped row goes where the first kept one goes, with that one's bytes
    first = torch.argmax(kept.to(torch.int32))
    src = torch.where(kept, torch.arange(slot.numel(), device=slot.device), first)
    at = _places(slot.long()[src], H, D, ps, cache.device)
    (kc, kb), (vc, vb) = _quantise(k[src]), _quantise(v[src])
    flat[at[0]] = _pack_k(kc)
    flat[at[1]] = _pack_v(vc)
    flat[at[2]] = kb
    flat[at[3]] = vb


def _load(cache, ps, slot, H, D):
    """fp32 rows [..., H, D] of K and V at slots; zero rows where a slot is negative."""
    shape = slot.shape
    s = slot.reshape(-1).long()
    flat = cache.view(-1)
    at = _places(s.clamp(min=0), H, D, ps, cache.device)
    kb, vb = flat[at[0]], flat[at[1]]
    kc = torch.stack((kb & 15, kb >> 4), -1).flatten(-2)  # [n,H,4,G,8]
    kc = kc.transpose(2, 3).unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)  # [n,H,G,32]
    vc = torch.stack((vb & 15, vb >> 4), -1).flatten(-2).transpose(2, 3).flatten(-2)
    live = (s >= 0).float()[:, None, None, None]
    k = (kc.float() - 8.0) * _scale_of(flat[at[2]])[..., None] * live
    v = (vc.float() - 8.0) * _scale_of(flat[at[3]])[..., None] * live
    return k.flatten(-2).view(*shape, H, D), v.flatten(-2).view(*shape, H, D)


# ------------------------------------------------------------------ inputs
def _rows(g, N, H, D, dt, dev):
    """Rows as a projection gives them: a few channels of every head are larger than the rest."""
    x = torch.randn((N, H, D), generator=g, device=dev)
    wide = torch.exp(0.8 * torch.randn((1, H, D), generator=g, device=dev))
    return (x * wide).to(dt)


def _new_cache(g, pages, H, D, ps, dev):
    """Pages with whatever an earlier request left in them."""
    return torch.randint(0, 256, (pages, H, ps * (D + D // 16)), generator=g, device=dev, dtype=torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, ps = case, case["ps"]
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(c)
    if c["op"] == "plan":
        R = c["R"]
        perm = torch.randperm(R, generator=g, device=dev)
        ln = torch.tensor(_ramp(R, c["lo"], c["hi"]), **i32)[perm]
        new = torch.tensor(_ramp(R, c["n_lo"], c["n_hi"]), **i32)[torch.randperm(R, generator=g, device=dev)]
        N = sum(_ramp(R, c["n_lo"], c["n_hi"]))
        most = _cdiv(c["hi"] + c["n_hi"], ps)
        need = sum(_cdiv(n, ps) for n in _ramp(R, c["lo"], c["hi"]))
        pages = need + R * (1 + _cdiv(c["n_hi"], ps)) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        have = (ln + ps - 1) // ps
        col = torch.arange(most, device=dev)
        at = (torch.cumsum(have, 0) - have)[:, None] + col
        table = torch.where(col < have[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32)
        free = torch.full((pages,), -1, **i32)
        free[:pages - need] = order[need:]
        s.update(len=ln, new=new, N=max(1, N), pages=pages, table=table, free=free,
                 n_free=torch.tensor([pages - need], **i32),
                 keep=(torch.rand(max(1, N), generator=g, device=dev) < c["keep"]).to(torch.uint8) if c["keep"] else None,
                 out_len=torch.empty(R, **i32), out_free=torch.empty(1, **i32), q_start=torch.empty(R + 1, **i32),
                 slot=torch.empty(max(1, N), **i32), vis=torch.empty(max(1, N), **i32))
        return s
    H, D, dt = c["Hkv"], c["D"], _DT[c["dt"]]
    if c["op"] == "append":
        N = c["N"]
        pages = _cdiv(N, ps) + 7
        wide = (c["Hq"] + 2 * H) * D
        qkv = torch.empty((N, wide), dtype=dt, device=dev)
        qkv.view(N, -1, D)[:, c["Hq"]:] = _rows(g, N, 2 * H, D, dt, dev)
        # consecutive tokens in pages of their own, as a plan gives them
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(N, device=dev)
        slot = (order[t // ps] * ps + t % ps).to(torch.int32)
        if c["drop"]:
            slot = torch.where(torch.rand(N, generator=g, device=dev) < c["drop"], -1, slot)
            slot[0] = order[0] * ps
        new = dict(dtype=dt, device=dev)
        s.update(k=qkv.view(N, -1, D)[:, c["Hq"]:c["Hq"] + H], v=qkv.view(N, -1, D)[:, c["Hq"] + H:], slot=slot,
                 cache=_new_cache(g, pages, H, D, ps, dev), k_out=torch.empty((N, H, D), **new),
                 v_out=torch.empty((N, H, D), **new))
        return s
    if c["op"] == "read":
        N = c["N"]
        pages = _cdiv(N, ps) + 7
        cache = _new_cache(g, pages, H, D, ps, dev)
        order = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(N, device=dev)
        slot = (order[t // ps] * ps + t % ps).to(torch.int32)
        _store(cache, ps, slot, _rows(g, N, H, D, dt, dev), _rows(g, N, H, D, dt, dev))
        s.update(cache=cache, slot=slot, k_out=torch.empty((N, H, D), dtype=dt, device=dev),
                 v_out=torch.empty((N, H, D), dtype=dt, device=dev))
        return s
    R, Hq = c["R"], c["Hq"]
    lens = torch.tensor(_ramp(R, c["lo"], c["hi"]))[torch.randperm(R, generator=torch.Generator().manual_seed(seed))]
    new = torch.tensor(_ramp(R, c["n_lo"], c["n_hi"]))
    lens, new = lens.tolist(), [int(n) for n in new]
    lens = [max(ln, n) if ln > 0 else 0 for ln, n in zip(lens, new)]  # the new tokens are cached already
    N = max(1, sum(new))
    have = [_cdiv(n, ps) for n in lens]
    most, pages = max(1, max(have)), sum(have) + 5
    cache = _new_cache(g, pages, H, D, ps, dev)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((R, most), -1, **i32)
    done = 0
    for r in range(R):
        table[r, :have[r]] = order[done:done + have[r]]
        done += have[r]
    wide = _rows(g, 1, 2 * H, D, torch.float32, dev)
    for r in range(R):
        for a in range(0, lens[r], 16384):
            t = torch.arange(a, min(lens[r], a + 16384), device=dev)
            kv = (torch.randn((t.numel(), 2 * H, D), generator=g, device=dev) * (0.4 + wide.abs())).to(dt)
            _store(cache, ps, table[r, t // ps] * ps + (t % ps).to(torch.int32), kv[:, :H], kv[:, H:])
    q = (torch.randn((N, Hq, D), generator=g, device=dev) * 1.2).to(dt)
    vis = torch.zeros(N, dtype=torch.int32)
    q_start, at = [0], 0
    for r in range(R):
        if lens[r]:
            vis[at:at + new[r]] = torch.arange(lens[r] - new[r] + 1, lens[r] + 1, dtype=torch.int32)
        at += new[r]
        q_start.append(at)
    s.update(q=q, cache=cache, table=table, vis=vis.to(dev), q_start=torch.tensor(q_start, **i32), N=N, total=at,
             most_len=max(1, max(lens)), most_new=max(1, max(new)), scale=D ** -0.5,
             o=torch.zeros((N, Hq, D), dtype=dt, device=dev), lse=torch.zeros((N, Hq), device=dev))
    return s


# ------------------------------------------------------------------ one pass
def _plan(s):
    R, N, ps = s["R"], s["N"], s["ps"]
    ln, new, dev = s["len"], s["new"], s["len"].device
    end = torch.cumsum(new, 0)
    q_start = torch.cat((end.new_zeros(1), end))
    t = torch.arange(N, device=dev)
    r = torch.searchsorted(end, t, right=True).clamp(max=R - 1)
    live = t < end[-1]
    keep = live if s["keep"] is None else (s["keep"] != 0) & live
    upto = torch.cat((q_start.new_zeros(1), torch.cumsum(keep, 0)))  # kept before token t
    first = upto[q_start[:-1]]
    kept = upto[q_start[1:]] - first
    have, then = (ln + ps - 1) // ps, (ln + kept + ps - 1) // ps
    taken = torch.cumsum(then - have, 0)
    before = taken - (then - have)
    pos = ln[r] + upto[:-1] - first[r]
    page = pos // ps
    fresh = s["free"][(s["n_free"] - 1 - (before[r] + page - have[r])).clamp(min=0)]
    old = s["table"][r, page.clamp(max=s["table"].shape[1] - 1)]
    slot = torch.where(keep, torch.where(page < have[r], old, fresh) * ps + pos % ps, -1)
    col = torch.arange(s["table"].shape[1], device=dev)
    grown = s["free"][(s["n_free"] - 1 - (before[:, None] + col - have[:, None])).clamp(0, s["pages"] - 1)]
    table = torch.where((col >= have[:, None]) & (col < then[:, None]), grown, s["table"])
    i = torch.int32
    return dict(table=table, len=(ln + kept).to(i), n_free=(s["n_free"] - taken[-1]).to(i), q_start=q_start.to(i),
                slot=slot.to(i), vis=torch.where(live, pos + keep, 0).to(i))


def _attn(s):
    R, ps, H, D, N = s["R"], s["ps"], s["Hkv"], s["D"], s["N"]
    L, n, dev = s["most_len"], s["most_new"], s["q"].device
    G = s["Hq"] // H
    pos = torch.arange(L, device=dev)
    slot = s["table"][:, pos // ps] * ps + pos % ps
    k, v = _load(s["cache"], ps, slot, H, D)  # [R, L, H, D]
    row = s["q_start"][:-1, None] + torch.arange(n, device=dev)  # [R, n]
    live = row < s["q_start"][1:, None]
    row = torch.where(live, row, N).long()
    q = torch.cat((s["q"], s["q"].new_zeros(1, s["Hq"], D)))[row].float().view(R, n, H, G, D)
    vis = torch.cat((s["vis"], s["vis"].new_zeros(1)))[row]  # [R, n]
    a = torch.matmul(q.permute(0, 2, 3, 1, 4).flatten(2, 3), k.permute(0, 2, 3, 1)) * s["scale"]  # [R, H, G n, L]
    a = a.view(R, H, G, n, L).masked_fill_(pos >= vis[:, None, None, :, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    p = torch.exp_(a.sub_(torch.where(m == -math.inf, 0.0, m)))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).view(R, H, G, n, D)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(R, n, s["Hq"], D)
    lse = (m + torch.log(z)).squeeze(-1).permute(0, 3, 1, 2).reshape(R, n, s["Hq"])
    out, out_l = s["o"].new_zeros((N + 1, s["Hq"], D)), s["lse"].new_zeros((N + 1, s["Hq"]))
    out[row.flatten()] = o.flatten(0, 1).to(out.dtype)
    out_l[row.flatten()] = lse.flatten(0, 1)
    return dict(o=out[:N], lse=out_l[:N])


def _call(s):
    """The framework's operators."""
    import sparse_causal_flash_gb300 as scfa

    op = s["op"]
    if op == "plan":
        if "ws" not in s:
            s["ws"] = scfa.workspace(scfa.cache4_plan_workspace_size(s["N"], s["R"]))
        scfa.scfa_cache4_plan(s["len"], s["new"], s["keep"], s["free"], s["n_free"], s["table"], s["ps"], s["pages"],
                              s["out_len"], s["out_free"], s["q_start"], s["slot"], s["vis"], s["ws"])
        return dict(table=s["table"], len=s["out_len"], n_free=s["out_free"], q_start=s["q_start"], slot=s["slot"],
                    vis=s["vis"])
    if op == "attn":
        if "ws" not in s:
            s["ws"] = scfa.workspace(scfa.cache4_attn_workspace_size(s["N"], s["R"], s["Hq"], s["Hkv"], s["D"]))
        scfa.scfa_cache4_attn(s["q"], s["cache"], s["ps"], s["table"], s["q_start"], s["vis"], s["scale"], s["o"],
                              s["lse"], s["ws"])
        return dict(o=s["o"], lse=s["lse"])
    if op == "append":
        scfa.scfa_cache4_append(s["k"], s["v"], s["slot"], s["cache"], s["ps"])
    scfa.scfa_cache4_read(s["cache"], s["ps"], s["slot"], s["k_out"], s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def run(s):
    if own:
        return _call(s)
    op = s["op"]
    if op == "plan":
        return _plan(s)
    if op == "attn":
        return _attn(s)
    if op == "append":  # what the cache now holds of the rows comes back as values
        _store(s["cache"], s["ps"], s["slot"], s["k"], s["v"])
    k, v = _load(s["cache"], s["ps"], s["slot"], s["Hkv"], s["D"])
    return dict(k=k.to(s["k_out"].dtype), v=v.to(s["v_out"].dtype))


def work(case):
    c = case
    if c["op"] == "plan":
        n = sum(_ramp(c["R"], c["n_lo"], c["n_hi"]))
        return dict(bytes=8 * n + (n if c["keep"] else 0) + 20 * c["R"] + 8, flops=0)
    D, H = c["D"], c["Hkv"]
    row = H * (D + D // 16)  # bytes of one token's K and V in the cache
    if c["op"] == "append":
        n = c["N"] * (1 - c["drop"])
        # rows in, codes out; then codes in, values out (the codes just written are read again)
        return dict(bytes=n * (4 * H * D + 2 * row) + c["N"] * (4 * H * D + 8), flops=0)
    if c["op"] == "read":
        return dict(bytes=c["N"] * (row + 4 * H * D + 4), flops=0)
    new = _ramp(c["R"], c["n_lo"], c["n_hi"])
    # the seed pairs lengths with new tokens; the sums are near enough the same for every pairing
    lens = [max(ln, n) if ln > 0 else 0 for ln, n in zip(_ramp(c["R"], c["lo"], c["hi"]), new)]
    seen = sum(n * ln - n * (n - 1) // 2 for ln, n in zip(lens, new) if ln)
    n = sum(new)
    return dict(bytes=sum(lens) * row + n * c["Hq"] * (4 * D + 4) + 4 * n + sum(4 * _cdiv(x, c["ps"]) for x in lens),
                flops=4 * D * c["Hq"] * seen)


# ------------------------------------------------------------------ the definition in 64 bits
def _pow2(e):
    """2^e exactly, e a float64 tensor of whole numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(cache, ps, slot, head, D, is_v):
    """float64 values [n, D] of one head's rows: every channel's byte looked up by its own address."""
    H, G = cache.shape[1], D // 32
    dev = cache.device
    ch = torch.arange(D, device=dev)
    slot = slot.long()
    t, tile = slot % ps % 16, 16 * (D + D // 16)
    base = (slot // ps * H + head) * ps * (D + D // 16) + slot % ps // 16 * tile
    g, in32 = ch // 32, ch % 32
    if not is_v:
        j, c8 = in32 // 8, in32 % 8
        place = c8 // 2 + 4 * (c8 % 2)
        at = (base + t * (D // 2))[:, None] + (j * 4 * G + g * 4 + place // 2)
        high = place % 2
        scale_at = (base + 16 * D + t * G)[:, None] + g
    else:
        r, i = in32 // 4, in32 % 4
        at = (base + 8 * D + (t // 8) * 4 * D + (t // 2 % 4) * 4 * G + (t % 2) * 2 * G)[:, None] + (r * 16 * G + g * 2 + i // 2)
        high = i % 2
        scale_at = (base + 16 * D + 16 * G + t * G)[:, None] + g
    flat = cache.view(-1)
    code = (flat[at].long() >> (4 * high)) % 16 - 8
    b = flat[scale_at].double()
    e = torch.floor(b / 8)
    return code.double() * (8 + (b - 8 * e)) * _pow2(e - 18)


def _exact_round(x):
    """[N, H, D] -> the float64 values that the format holds for them."""
    x = x.double().view(*x.shape[:-1], -1, 32)
    x = torch.where(x != x, torch.zeros_like(x), x)
    a = x.abs().max(-1, keepdim=True).values
    a = (a / torch.full_like(a, 7)).clamp(2.0 ** -15, 9216.0)
    e = torch.floor(torch.log2(a))
    e = torch.where(_pow2(e) > a, e - 1, e)
    e = torch.where(_pow2(e + 1) <= a, e + 1, e)
    step = _pow2(e - 3)
    s = torch.round(a / step) * step
    return (torch.round(x / s).clamp(-7, 7) * s).flatten(-2)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    H, D, ps = s["Hkv"], s["D"], s["ps"]
    if case["op"] == "append":
        kept = (s["slot"] >= 0)[:, None, None]
        return {"k": _exact_round(s["k"]) * kept, "v": _exact_round(s["v"]) * kept}
    if case["op"] == "read":
        return {x: torch.stack([_exact_values(s["cache"], ps, s["slot"], h, D, x == "v") for h in range(H)], 1)
                for x in "kv"}
    G, dev = s["Hq"] // H, s["q"].device
    o = torch.zeros((s["N"], s["Hq"], D), dtype=torch.float64, device=dev)
    lse = torch.zeros((s["N"], s["Hq"]), dtype=torch.float64, device=dev)
    starts = s["q_start"].tolist()
    for r in range(s["R"]):
        a, b = starts[r], starts[r + 1]
        if a == b:
            continue
        vis = s["vis"][a:b].long()
        n = int(vis.max())
        lse[a:b] = -math.inf
        if n == 0:
            continue
        pos = torch.arange(n, device=dev)
        slot = s["table"][r].long()[pos // ps] * ps + pos % ps
        for h in range(H):
            k = _exact_values(s["cache"], ps, slot, h, D, False)
            v = _exact_values(s["cache"], ps, slot, h, D, True)
            x = torch.einsum("ngd,ld->ngl", s["q"][a:b, h * G:(h + 1) * G].double(), k) / math.sqrt(D)
            x = torch.where(pos < vis[:, None, None], x, -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            w = torch.where(z > -math.inf, torch.exp(x - z), 0.0)
            o[a:b, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", w, v)
            lse[a:b, h * G:(h + 1) * G] = z[..., 0]
    return {"o": o, "lse": lse}
