"""Cases of what stands around and inside a training step on packed sequences: rotary positions of queries and keys
with their norm, and attention over packed sequences whose query heads share key heads, each with its gradients.

`own = False` computes each operator in plain torch; `own = True` calls sparse_causal_flash_gb300.

Rotary: a row x [D] at position p. With a norm, x is first divided by sqrt(mean(x^2) + eps) and multiplied by w, channel
by channel. Of the first `rot` channels, pair i (channels i and i + rot / 2, or 2 i and 2 i + 1 when interleaved) turns by
p f[i] radians and is multiplied by `factor`; the other channels stay.

Attention: sequence r has the query rows q_start[r] .. q_start[r + 1] and the key rows k_start[r] .. k_start[r + 1], the
last query aligned with the last key. With n queries and m keys, query t sees the keys j <= t + m - n, and with a window w
only those with j > t + m - n - w; query head h reads key head h / (Hq / Hkv). A query that sees nothing gives o = 0 and
lse = -inf. Rows behind the last sequence belong to nobody and are left as they were (zero here).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of each of 61 requests, far into contexts that the frequencies were stretched for
        dict(name="rope 61 tokens", op="rope", N=61, Hq=32, Hkv=8, D=128, rot=128, il=False, norm=True, stretch=8.0,
             far=250000, dt="bf16"),
        # queries and keys of a training batch, views of a fused projection
        dict(name="rope 8192 tokens norm", op="rope", N=8192, Hq=32, Hkv=8, D=128, rot=128, il=False, norm=True, stretch=1.0,
             far=8192, dt="bf16"),
        # the kept query rows of a QK-sparse step (4 x 12 heads of 8192 tokens, 30% dropped): every row has its own position
        dict(name="rope 275280 kept rows d64", op="rope", N=275280, Hq=1, Hkv=0, D=64, rot=64, il=True, norm=False,
             stretch=1.0, far=8192, dt="bf16"),
        # the gradients of the second case
        dict(name="rope_bwd 8192 tokens norm", op="rope_bwd", N=8192, Hq=32, Hkv=8, D=128, rot=128, il=False, norm=True,
             stretch=1.0, far=8192, dt="bf16"),
        # 12 heads of 64 channels over 4 key heads, half of each head turned, fp16, an odd count
        dict(name="rope_bwd 5003 h12 d64 f16", op="rope_bwd", N=5003, Hq=12, Hkv=4, D=64, rot=32, il=True, norm=True,
             stretch=4.0, far=32768, dt="f16"),
        # a handful of short texts: latency
        dict(name="fwd 7 short h12 d64", op="fwd", R=7, n_lo=1, n_hi=61, m_more=0, window=0, Hq=12, Hkv=12, D=64, pad=3,
             dt="bf16"),
        # one long training sequence, four query heads to a key head
        dict(name="fwd 8192 h32/8 d128", op="fwd", R=1, n_lo=8192, n_hi=8192, m_more=0, window=0, Hq=32, Hkv=8, D=128, pad=0,
             dt="bf16"),
        # prompt chunks over the keys of what came before: few rows over a long axis
        dict(name="fwd 3 chunks over 12000 f16", op="fwd", R=3, n_lo=33, n_hi=97, m_more=12000, window=0, Hq=32, Hkv=8, D=128,
             pad=0, dt="f16"),
        # a sliding window over a long sequence, three query heads to a key head
        dict(name="fwd 16384 window 2000 h12/4 d64", op="fwd", R=1, n_lo=16384, n_hi=16384, m_more=0, window=2000, Hq=12,
             Hkv=4, D=64, pad=0, dt="bf16"),
        # gradients of the handful of short texts
        dict(name="bwd 7 short h12 d64", op="bwd", R=7, n_lo=1, n_hi=61, m_more=0, window=0, Hq=12, Hkv=12, D=64, pad=3,
             dt="bf16"),
        # gradients of the long training sequence
        dict(name="bwd 8192 h32/8 d128", op="bwd", R=1, n_lo=8192, n_hi=8192, m_more=0, window=0, Hq=32, Hkv=8, D=128, pad=0,
             dt="bf16"),
        # gradients of a batch of texts of very unlike lengths, packed without padding, fp16
        dict(name="bwd 9 ragged h12/4 d64 f16", op="bwd", R=9, n_lo=101, n_hi=3501, m_more=0, window=0, Hq=12, Hkv=4, D=64,
             pad=0, dt="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST_ROWS = 8192 * 40  # query and key rows of 128 channels of a drawn rotary case
_MOST_CELLS = 8192 * 8192 * 32 * 128  # score cells x channels of a drawn attention case, masked ones too


def draw(rng):
    op = rng.choice(("rope", "rope_bwd", "fwd", "fwd", "bwd", "bwd"))
    D = rng.choice((64, 128))
    dt = rng.choice(("bf16", "bf16", "f16"))
    if op.startswith("rope"):
        norm = rng.random() < 0.6
        stretch = rng.choice((1.0, 1.0, 4.0, 8.0, 32.0))
        rot = rng.choice((D, D, D // 2, D // 4, D - 16, 2 * rng.randint(1, D // 2)))
        if rng.random() < 0.25:  # rows with positions of their own
            Hq, Hkv = 1, 0
        else:
            Hkv = rng.choice((1, 2, 3, 4, 8, 12))
            Hq = Hkv * rng.choice((1, 1, 2, 3, 4, 5, 8))
        N = _log(rng, 1, _MOST_ROWS * 128 // (D * (Hq + Hkv)))
        return dict(op=op, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot, il=rng.random() < 0.4, norm=norm, stretch=stretch,
                    far=_log(rng, 64, 1000000), dt=dt)
    Hkv = rng.choice((1, 2, 3, 4, 8))
    Hq = Hkv * rng.choice((1, 1, 2, 3, 4, 5, 6, 8))
    R = _log(rng, 1, 64)
    # a gradient that is zero in every row says nothing: more than one key to a query there
    least = 8 if op == "bwd" else 1
    window = rng.choice((0, 0, 0, _log(rng, least, 4096)))
    kind = rng.random()
    if kind < 0.6:  # packed texts
        m_more, most = 0, math.isqrt(_MOST_CELLS // (R * Hq * D))
        n_hi = _log(rng, least, min(16384, most))
    elif kind < 0.85:  # chunks over a prefix
        n_hi = _log(rng, 1, 300)
        m_more = _log(rng, 1, max(2, min(40000, _MOST_CELLS // (R * Hq * D * n_hi) - n_hi)))
    else:  # more queries than keys: the first see nothing
        n_hi = _log(rng, 2 * least, min(2000, math.isqrt(_MOST_CELLS // (R * Hq * D))))
        m_more = -rng.randint(1, n_hi if op == "fwd" else n_hi // 2)
    return dict(op=op, R=R, n_lo=rng.randint(0, n_hi), n_hi=n_hi, m_more=m_more, window=window, Hq=Hq, Hkv=Hkv, D=D,
                pad=rng.choice((0, 0, 5)), dt=dt)


def _lengths(c):
    """(queries, keys) of each sequence: their sum is the case's, whatever the seed."""
    R, lo, hi = c["R"], c["n_lo"], c["n_hi"]
    n = [lo + (hi - lo) * i // (R - 1) for i in range(R)] if R > 1 else [hi]
    return [(x, max(0, x + (c["m_more"] if i % 3 != 2 else c["m_more"] // 2))) for i, x in enumerate(n)]


def _seen(n, m, window):
    """Pairs of a query and a key that it sees."""
    total = 0
    for t in range(max(0, n - m), n):
        k = t + m - n + 1
        total += min(k, window) if window else k
    return total


# ------------------------------------------------------------------ inputs
def _frequencies(rot, stretch):
    """Radians per position of each pair, and the factor. Stretched, pairs that turned less than once over the 8192
    positions of the training turn `stretch` times slower, those that turned more than 32 times stay, and in between
    both are blended."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if stretch == 1.0:
        return f, 1.0
    keep = ((8192 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f / stretch * (1 - keep) + f * keep, 0.1 * math.log(stretch) + 1


def _rows(g, N, H, D, dt, dev):
    """Rows as a projection gives them: a few channels of every head are larger than the rest."""
    x = torch.randn((N, H, D), generator=g, device=dev)
    return (x * torch.exp(0.7 * torch.randn((1, H, D), generator=g, device=dev))).to(dt)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _DT[case["dt"]]
    if case["op"].startswith("rope"):
        N = case["N"]
        f, s["factor"] = _frequencies(case["rot"], case["stretch"])
        s["freq"] = f.to(dev)
        # texts packed one after another: positions that start anew, far ones among them
        start = torch.randint(0, max(1, case["far"] - 500), (N // 500 + 1,), generator=g, device=dev)
        t = torch.arange(N, device=dev)
        s["pos"] = (start[t // 500] + t % 500).clamp(max=case["far"]).to(torch.int32)
        # queries and keys of a fused projection; a head of values behind each key head
        qkv = _rows(g, N, Hq + 2 * Hkv, D, dt, dev)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv] if Hkv else None
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev)
            s["wk"] = 1 + 0.2 * torch.randn(D, generator=g, device=dev) if Hkv else None
        s["eps"] = 1e-6
        new = dict(dtype=dt, device=dev)
        if case["op"] == "rope":
            s["q_out"], s["k_out"] = torch.empty((N, Hq, D), **new), torch.empty((N, Hkv, D), **new) if Hkv else None
        else:
            s["dq"] = torch.randn((N, Hq, D), generator=g, device=dev).to(dt)
            s["dk"] = torch.randn((N, Hkv, D), generator=g, device=dev).to(dt) if Hkv else None
            dqkv = torch.zeros((N, Hq + 2 * Hkv, D), **new)
            s["dq_out"], s["dk_out"] = dqkv[:, :Hq], dqkv[:, Hq:Hq + Hkv] if Hkv else None
            s["dwq"] = torch.empty(D, device=dev) if case["norm"] else None
            s["dwk"] = torch.empty(D, device=dev) if case["norm"] and Hkv else None
        if own:
            _handles(s)
        return s
    lens = _lengths(case)
    order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()
    lens = [lens[i] for i in order]
    s["qs"], s["ks"] = [0], [0]
    for n, m in lens:
        s["qs"].append(s["qs"][-1] + n)
        s["ks"].append(s["ks"][-1] + m)
    s["N"] = N = max(1, s["qs"][-1] + case["pad"])
    s["M"] = M = max(1, s["ks"][-1] + case["pad"])
    s["q_start"] = torch.tensor(s["qs"], dtype=torch.int32, device=dev)
    s["k_start"] = torch.tensor(s["ks"], dtype=torch.int32, device=dev)
    # queries and keys behind their norm, values a view of the projection
    s["q"] = (1.2 * torch.randn((N, Hq, D), generator=g, device=dev)).to(dt)
    s["k"] = (1.2 * torch.randn((M, Hkv, D), generator=g, device=dev)).to(dt)
    s["v"] = _rows(g, M, 2 * Hkv, D, dt, dev)[:, Hkv:]
    s["scale"] = D ** -0.5
    s["o"] = torch.zeros((N, Hq, D), dtype=dt, device=dev)
    s["lse"] = torch.zeros((N, Hq), device=dev)
    if case["op"] == "bwd":
        out = _fwd(s)
        s["o"], s["lse"] = out["o"], out["lse"]
        s["do"] = torch.randn((N, Hq, D), generator=g, device=dev).to(dt)
        s["dq"], s["dk"], s["dv"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"]), torch.zeros_like(s["k"])
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------------ one pass, in plain torch
def _turn(x, s, back):
    """Rows [N, H, D] in 32 bits, turned (or turned back) by their positions."""
    rot = s["rot"]
    a = s["pos"].double()[:, None] * s["freq"]  # far positions: 64 bits
    cos, sin = (torch.cos(a) * s["factor"]).float()[:, None], (torch.sin(a) * s["factor"]).float()[:, None]
    if back:
        sin = -sin
    y = x.clone()
    if s["il"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h] = a * cos - b * sin
        y[..., h:rot] = b * cos + a * sin
    return y


def _rope(x, w, s):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w
    return _turn(y, s, False).to(x.dtype)


def _rope_bwd(dy, x, w, s):
    """Gradients of the rows and of the weights."""
    g = _turn(dy.float(), s, True)
    if w is None:
        return g.to(dy.dtype), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    n = x * r
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx.to(dy.dtype), (g * n).double().sum((0, 1)).float()


def _masked(a, n, m, window):
    """Scores [h, G, n, m] with -inf where the mask leaves nothing."""
    t = torch.arange(n, device=a.device)[:, None] + (m - n)
    j = torch.arange(m, device=a.device)
    hide = j > t
    if window:
        hide = hide | (j <= t - window)
    return a.masked_fill_(hide, -math.inf)


def _blocks(s):
    """(query rows, key rows, first key head, last key head) of what is worked on at once."""
    G = s["Hq"] // s["Hkv"]
    for r in range(s["R"]):
        a, b, c, d = s["qs"][r], s["qs"][r + 1], s["ks"][r], s["ks"][r + 1]
        step = max(1, (1 << 28) // max(1, G * (b - a) * (d - c)))
        for h in range(0, s["Hkv"], step):
            yield slice(a, b), slice(c, d), h, min(s["Hkv"], h + step)


def _fwd(s):
    o, lse = torch.zeros_like(s["q"]), torch.zeros((s["N"], s["Hq"]), device=s["q"].device)
    G, D = s["Hq"] // s["Hkv"], s["D"]
    for qr, kr, h, e in _blocks(s):
        n, m = qr.stop - qr.start, kr.stop - kr.start
        if n == 0:
            continue
        if m == 0:
            lse[qr, h * G:e * G] = -math.inf
            continue
        q = s["q"][qr, h * G:e * G].float().view(n, e - h, G, D).permute(1, 2, 0, 3)  # [h, G, n, D]
        k, v = (s[x][kr, h:e].float().transpose(0, 1)[:, None] for x in "kv")  # [h, 1, m, D]
        a = _masked(torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]), n, m, s["window"])
        top = a.amax(-1, keepdim=True)
        p = a.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        z = p.sum(-1, keepdim=True)
        y = torch.matmul(p, v)
        y = torch.where(z > 0, y / z, 0.0)
        o[qr, h * G:e * G] = y.permute(2, 0, 1, 3).flatten(1, 2).to(o.dtype)
        lse[qr, h * G:e * G] = (top + torch.log(z))[..., 0].permute(2, 0, 1).flatten(1, 2)
    return dict(o=o, lse=lse)


def _bwd(s):
    dq, dk, dv = torch.zeros_like(s["q"]), torch.zeros_like(s["k"]), torch.zeros_like(s["k"])
    G, D, scale = s["Hq"] // s["Hkv"], s["D"], s["scale"]
    for qr, kr, h, e in _blocks(s):
        n, m = qr.stop - qr.start, kr.stop - kr.start
        if n == 0 or m == 0:
            continue
        q, o, do = (s[x][qr, h * G:e * G].float().view(n, e - h, G, D).permute(1, 2, 0, 3) for x in ("q", "o", "do"))
        k, v = (s[x][kr, h:e].float().transpose(0, 1)[:, None] for x in "kv")
        lse = s["lse"][qr, h * G:e * G].view(n, e - h, G).permute(1, 2, 0)[..., None]
        a = _masked(torch.matmul(q, k.transpose(-1, -2)).mul_(scale), n, m, s["window"])
        p = a.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
        dv[kr, h:e] = torch.matmul(p.flatten(1, 2).transpose(-1, -2), do.flatten(1, 2)).transpose(0, 1).to(dv.dtype)
        dp = torch.matmul(do, v.transpose(-1, -2)).sub_((o * do).sum(-1, keepdim=True))
        ds = dp.mul_(p).mul_(scale)
        dq[qr, h * G:e * G] = torch.matmul(ds, k).permute(2, 0, 1, 3).flatten(1, 2).to(dq.dtype)
        dk[kr, h:e] = torch.matmul(ds.flatten(1, 2).transpose(-1, -2), q.flatten(1, 2)).transpose(0, 1).to(dk.dtype)
    return dict(dq=dq, dk=dk, dv=dv)


# ------------------------------------------------------------------ one pass, as a user of the framework makes it
def _handles(s):
    """What a program keeps from call to call: the table of frequencies, or the plan of the batch and a workspace."""
    import sparse_causal_flash_gb300 as scfa

    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    if s["op"].startswith("rope"):
        s["table"] = scfa.rope_table(s["freq"])
        if s["op"] == "rope_bwd":
            s["ws"] = scfa.workspace(scfa.rope_workspace_size(s["N"], Hq, Hkv, D))
        return
    s["plan"] = scfa.workspace(scfa.packed_plan_size(s["N"], s["M"], s["R"], Hq, Hkv))
    s["ws"] = scfa.workspace(scfa.packed_workspace_size(s["op"] == "bwd", s["N"], s["M"], s["R"], Hq, Hkv, D))
    scfa.scfa_packed_plan(s["q_start"], s["k_start"], s["N"], s["M"], Hq, Hkv, s["window"], s["plan"])


def _call(s):
    import sparse_causal_flash_gb300 as scfa

    op = s["op"]
    if op == "rope":
        scfa.scfa_rope_fwd(s["q"], s["k"], s["pos"], s["table"], s["q_out"], s["k_out"], interleaved=s["il"],
                           factor=s["factor"], wq=s["wq"], wk=s["wk"], eps=s["eps"])
        return dict(q=s["q_out"], k=s["k_out"]) if s["Hkv"] else dict(q=s["q_out"])
    if op == "rope_bwd":
        kw = dict(q=s["q"], k=s["k"], wq=s["wq"], wk=s["wk"], dwq=s["dwq"], dwk=s["dwk"], ws=s["ws"]) if s["norm"] else {}
        scfa.scfa_rope_bwd(s["dq"], s["dk"], s["pos"], s["table"], s["dq_out"], s["dk_out"], interleaved=s["il"],
                           factor=s["factor"], eps=s["eps"], **kw)
        out = dict(dq=s["dq_out"], dk=s["dk_out"], dwq=s["dwq"], dwk=s["dwk"])
        return {n: t for n, t in out.items() if t is not None}
    if op == "fwd":
        scfa.scfa_packed_fwd(s["q"], s["k"], s["v"], s["plan"], s["scale"], s["o"], s["lse"], s["ws"])
        return dict(o=s["o"], lse=s["lse"])
    scfa.scfa_packed_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["plan"], s["scale"], s["dq"], s["dk"], s["dv"],
                         s["ws"])
    return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])


def run(s):
    if own:
        return _call(s)
    op = s["op"]
    if op == "rope":
        out = dict(q=_rope(s["q"], s["wq"], s))
        if s["Hkv"]:
            out["k"] = _rope(s["k"], s["wk"], s)
        return out
    if op == "rope_bwd":
        out = {}
        out["dq"], dwq = _rope_bwd(s["dq"], s["q"], s["wq"], s)
        dwk = None
        if s["Hkv"]:
            out["dk"], dwk = _rope_bwd(s["dk"], s["k"], s["wk"], s)
        if dwq is not None:
            out["dwq"] = dwq
        if dwk is not None:
            out["dwk"] = dwk
        return out
    return _fwd(s) if op == "fwd" else _bwd(s)


def work(case):
    c = case
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"].startswith("rope"):
        row = 2 * c["N"] * (Hq + Hkv) * D
        n = 3 if c["op"] == "rope_bwd" and c["norm"] else 2
        return dict(bytes=n * row + 4 * c["N"] + 4 * c["rot"], flops=c["N"] * (Hq + Hkv) * (3 * c["rot"] + 4 * D * c["norm"]))
    lens = _lengths(c)
    n, m = sum(x for x, _ in lens), sum(y for _, y in lens)
    seen = sum(_seen(x, y, c["window"]) for x, y in lens)
    if c["op"] == "fwd":  # q in, o out, k and v in
        return dict(bytes=n * Hq * (4 * D + 4) + 4 * m * Hkv * D, flops=4 * D * Hq * seen)
    # q, o, do in, dq out; k, v in, dk, dv out
    return dict(bytes=n * Hq * (8 * D + 4) + 8 * m * Hkv * D, flops=10 * D * Hq * seen)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rope(x, w, s):
    """float64 rows [N, H, D]: each pair is a complex number that is multiplied by factor e^(i p f)."""
    N, H, D = x.shape
    if w is not None:
        x = x / torch.sqrt(torch.einsum("nhd,nhd->nh", x, x)[..., None] / D + s["eps"]) * w
    c = torch.arange(s["rot"] // 2, device=x.device)
    even, odd = (2 * c, 2 * c + 1) if s["il"] else (c, c + s["rot"] // 2)
    z = torch.complex(x[:, :, even], x[:, :, odd])
    z = z * torch.polar(torch.full((N, 1, c.numel()), float(s["factor"]), dtype=torch.float64, device=x.device),
                        torch.outer(s["pos"].double(), s["freq"])[:, None])
    place = torch.cat((even, odd, torch.arange(s["rot"], D, device=x.device)))
    return torch.cat((z.real, z.imag, x[:, :, s["rot"]:]), -1)[:, :, torch.argsort(place)]


def _exact_head(q, k, v, n, m, window):
    """float64 o [n, D] and lse [n] of one query head (q already scaled)."""
    x = q @ k.T
    last = torch.arange(n, device=q.device) + m - n  # the last key that each query sees
    back = last[:, None] - torch.arange(m, device=q.device)  # how far a key lies behind it
    ok = (back >= 0) & (back < (window or m + n + 1))
    some = ok.any(1)
    x = torch.where(ok, x, -math.inf)
    z = torch.logsumexp(torch.where(some[:, None], x, 0.0), 1)
    return torch.exp(x - z[:, None]) @ v, torch.where(some, z, -math.inf)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op.startswith("rope"):
        out = {}
        for x in ("q", "k") if case["Hkv"] else ("q",):
            w = None if s["w" + x] is None else s["w" + x].double()
            rows = s[x].double()
            if op == "rope":
                out[x] = _exact_rope(rows, w, s)
                continue
            with torch.enable_grad():
                rows.requires_grad_(True)
                if w is not None:
                    w.requires_grad_(True)
                y = _exact_rope(rows, w, s)
                grads = torch.autograd.grad(y, [rows] + ([w] if w is not None else []), s["d" + x].double())
            out["d" + x] = grads[0]
            if w is not None:
                out["dw" + x] = grads[1]
        return {n: out[n] for n in ("q", "k", "dq", "dk", "dwq", "dwk") if n in out}
    G, D, dev = s["Hq"] // s["Hkv"], s["D"], s["q"].device
    new = dict(dtype=torch.float64, device=dev)
    o, lse = torch.zeros((s["N"], s["Hq"], D), **new), torch.zeros((s["N"], s["Hq"]), **new)
    dq, dk, dv = torch.zeros((s["N"], s["Hq"], D), **new), torch.zeros((s["M"], s["Hkv"], D), **new), \
        torch.zeros((s["M"], s["Hkv"], D), **new)
    for r in range(s["R"]):
        a, b, c, d = s["qs"][r], s["qs"][r + 1], s["ks"][r], s["ks"][r + 1]
        if a == b:
            continue
        if c == d:
            lse[a:b] = -math.inf
            continue
        for h in range(s["Hq"]):
            q, k, v = s["q"][a:b, h].double(), s["k"][c:d, h // G].double(), s["v"][c:d, h // G].double()
            if op == "fwd":
                o[a:b, h], lse[a:b, h] = _exact_head(q / math.sqrt(D), k, v, b - a, d - c, s["window"])
                continue
            with torch.enable_grad():
                for t in (q, k, v):
                    t.requires_grad_(True)
                y, _ = _exact_head(q / math.sqrt(D), k, v, b - a, d - c, s["window"])
                gq, gk, gv = torch.autograd.grad(y, (q, k, v), s["do"][a:b, h].double())
            dq[a:b, h] = gq
            dk[c:d, h // G] += gk
            dv[c:d, h // G] += gv
    return {"o": o, "lse": lse} if op == "fwd" else {"dq": dq, "dk": dk, "dv": dv}
