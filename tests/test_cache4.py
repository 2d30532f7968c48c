"""The paged 4-bit cache without a GPU: its oracle against hand-worked values and
invariants, and the refusals of the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache4 as oc


@pytest.fixture(scope="module")
def scfa():
    from sparse_causal_flash_gb300 import build
    build.build()
    import sparse_causal_flash_gb300 as s
    return s


@pytest.mark.parametrize("a,byte,value", [
    (7.0, 15 * 8, 1.0), (0.0, 0, 2.0 ** -15), (7 * 2.0 ** -15, 0, 2.0 ** -15), (14.0, 16 * 8, 2.0),
    (7 * 1.0625, 15 * 8, 1.0),  # a tie between 1 and 1.125 goes to the even one
    (7 * 1.1875, 15 * 8 + 2, 1.25),  # a tie between 1.125 and 1.25
    (7 * 1.97, 16 * 8, 2.0), (64512.0, 28 * 8 + 1, 9216.0), (1e30, 28 * 8 + 1, 9216.0), (np.inf, 28 * 8 + 1, 9216.0)])
def test_scale_byte(a, byte, value):
    assert oc.scale_byte(a) == byte
    assert oc.scale_value(byte) == value


def test_quantise_hand_case():
    x = np.zeros(32)
    x[:6] = [7.0, -3.5, 0.5, 1.5, -0.5, np.nan]
    c, b = oc.quantise(x)
    assert b.tolist() == [15 * 8]
    assert c[:6].tolist() == [7, -4, 0, 2, 0, 0]  # ties to even
    x[6] = -np.inf
    c, b = oc.quantise(x)
    assert oc.values(x)[6] == -64512.0 and c[0] == 0


def test_values_are_exact_in_both_types_and_near():
    g = np.random.default_rng(1)
    x = g.standard_normal((400, 64)) * np.exp(3 * g.standard_normal((400, 1)))
    v = oc.values(x)
    for dt in (torch.bfloat16, torch.float16):
        assert np.array_equal(torch.tensor(v).to(dt).double().numpy(), v)
    c, b = oc.quantise(x)
    s = np.repeat(oc.scale_value(b), 32, -1)
    assert np.all(np.abs(x - v) <= s / 2 * (1 + 1e-12))  # no code saturates below the largest scale
    assert np.array_equal(oc.values(v), v) or np.all(np.abs(oc.values(v) - v) <= s / 2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page_size", [16, 64])
def test_addresses_fill_a_page_once(D, page_size):
    seen, scales = set(), set()
    for slot in range(2 * page_size, 3 * page_size):
        for ch in range(D):
            for is_v in (False, True):
                at, high, sc = oc.addresses(slot, 1, ch, 3, D, page_size, is_v)
                assert (at, high) not in seen
                seen.add((at, high))
                scales.add(sc)
    page = page_size * (D + D // 16)
    both = {a for a, _ in seen} | scales
    assert both == set(range((2 * 3 + 1) * page, (2 * 3 + 2) * page))
    assert len(scales) == page_size * D // 16 and not scales & {a for a, _ in seen}


def test_plan_hand_case():
    table = np.full((2, 3), -1)
    table[0, 0] = 4
    keep = np.array([1, 0, 1, 1, 1], np.uint8)
    out = oc.plan([15, 0], [3, 1], keep, [7, 2, 5], 3, table, 5, 16, 8)
    assert out["slot"].tolist() == [4 * 16 + 15, -1, 5 * 16, 2 * 16, -1]
    assert out["vis"].tolist() == [16, 16, 17, 1, 0]
    assert out["n_free"] == 1 and out["len"].tolist() == [17, 1] and out["q_start"].tolist() == [0, 3, 4]
    assert out["table"].tolist() == [[4, 5, -1], [2, -1, -1]]
    assert oc.plan([15, 0], [3, 1], keep, [7], 1, table, 5, 16, 8) == "no pages"
    assert oc.plan([48, 0], [1, 0], None, [7], 1, table, 5, 16, 8) == "invalid"
    assert oc.plan([0, 0], [3, 3], None, [7], 1, table, 5, 16, 8) == "invalid"


def test_attention_of_the_oracle_is_softmax():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal(64), g.standard_normal((9, 64)), g.standard_normal((9, 64))
    o, lse = oc.attention(q, k, v, 0.125)
    p = torch.softmax(torch.tensor(k @ q * 0.125), 0).numpy()
    assert np.allclose(o, p @ v) and np.isclose(lse, torch.logsumexp(torch.tensor(k @ q * 0.125), 0).item())
    o, lse = oc.attention(q, k[:0], v[:0], 0.125)
    assert not o.any() and lse == -np.inf


FAKE = ctypes.c_void_p(4096)


def plan_args(**kw):
    a = dict(len=FAKE, new=FAKE, keep=None, free=FAKE, n_free=FAKE, table=FAKE, N=8, R=4, mp=4, ps=64, pages=9,
             out=FAKE, fout=FAKE, qs=FAKE, slot=FAKE, vis=FAKE, ws=FAKE, nb=1 << 20, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(len=None), 1), (dict(table=None), 1), (dict(ws=None), 1), (dict(N=0), 1), (dict(R=-1), 1), (dict(mp=0), 1),
    (dict(pages=0), 1), (dict(ps=48), 2), (dict(ps=512), 2), (dict(pages=1 << 26), 2), (dict(mp=1 << 26), 2),
    (dict(ws=ctypes.c_void_p(4097)), 3), (dict(nb=100), 3)])
def test_plan_refusals(scfa, kw, code):
    assert scfa._lib.scfa_cache4_plan(*plan_args(**kw)) == code


def rows_args(read, **kw):
    a = dict(k=FAKE, kt=512, kh=64, v=FAKE, vt=512, vh=64, slot=FAKE, N=8, H=8, D=64, dt=0, cache=FAKE, ps=64, pages=9)
    a.update(kw)
    if not read:
        return list(a.values()) + [None]
    return [a[x] for x in ("cache", "ps", "pages", "slot", "N", "H", "D", "dt", "k", "kt", "kh", "v", "vt", "vh")] + [None]


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(slot=None), 1), (dict(cache=None), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(D=96), 2),
    (dict(D=32), 2), (dict(dt=2), 2), (dict(dt=-1), 2), (dict(ps=24), 2), (dict(pages=0), 1), (dict(pages=1 << 25), 2),
    (dict(kt=513), 1), (dict(vh=4), 1), (dict(v=ctypes.c_void_p(4104)), 1), (dict(cache=ctypes.c_void_p(4104)), 1)])
def test_append_and_read_refusals(scfa, read, kw, code):
    fn = scfa._lib.scfa_cache4_read if read else scfa._lib.scfa_cache4_append
    assert fn(*rows_args(read, **kw)) == code


def attn_args(**kw):
    a = dict(q=FAKE, qt=512, qh=64, cache=FAKE, ps=64, pages=9, table=FAKE, mp=4, qs=FAKE, vis=FAKE, N=8, R=4, Hq=8,
             Hkv=4, D=64, scale=0.125, dt=0, o=FAKE, ot=512, oh=64, lse=FAKE, ws=FAKE, nb=1 << 30, flags=0, st=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(vis=None), 1), (dict(lse=None), 1), (dict(ws=None), 1), (dict(N=0), 1), (dict(R=0), 1),
    (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(Hq=2), 1), (dict(D=80), 2), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1), (dict(dt=3), 2), (dict(ps=8), 2),
    (dict(mp=0), 1), (dict(pages=0), 1), (dict(mp=1 << 26), 2), (dict(qt=12), 1), (dict(oh=68), 1), (dict(o=ctypes.c_void_p(4098)), 1),
    (dict(ws=ctypes.c_void_p(4100)), 3), (dict(nb=128), 3)])
def test_attn_refusals(scfa, kw, code):
    assert scfa._lib.scfa_cache4_attn(*attn_args(**kw)) == code


def test_sizes(scfa):
    assert scfa.cache4_page_bytes(64, 128) == 64 * 136 and scfa.cache4_page_bytes(16, 64) == 1088
    assert scfa.cache4_page_bytes(48, 64) == 0 and scfa.cache4_page_bytes(64, 96) == 0
    assert scfa.cache4_plan_workspace_size(0, 1) == 0 < scfa.cache4_plan_workspace_size(1, 1)
    assert scfa.cache4_attn_workspace_size(4, 1, 8, 3, 64) == 0 < scfa.cache4_attn_workspace_size(4, 1, 9, 3, 64)


def test_binding_refuses_tensors_it_cannot_take(scfa):
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    slot = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((3, 2, 64 * 68), dtype=torch.uint8)
    with pytest.raises(ValueError):  # not on a GPU
        scfa.scfa_cache4_append(k, k, slot, cache, 64)
    with pytest.raises(ValueError):
        scfa.scfa_cache4_read(cache, 64, slot, k, k)
    with pytest.raises(ValueError):
        scfa.scfa_cache4_attn(k, cache, 64, slot.view(2, 2), slot[:3], slot, 0.125, k, torch.zeros(4, 2), cache.view(-1))
    with pytest.raises(ValueError):
        scfa.scfa_cache4_plan(slot, slot, None, slot, slot[:1], slot.view(4, 1), 64, 4, slot, slot[:1], slot, slot, slot,
                              cache.view(-1))
    from sparse_causal_flash_gb300.cache import KVCache4
    for kw in (dict(D=96), dict(page_size=48), dict(dtype=torch.float32), dict(Hq=5), dict(Hq=0), dict(R=0), dict(n_pages=0),
               dict(max_len=0), dict(max_tokens=0)):
        with pytest.raises(ValueError):
            KVCache4(**{**dict(R=2, n_pages=4, Hq=4, Hkv=2, D=64, max_len=64, max_tokens=2, device="cpu"), **kw})


@pytest.mark.parametrize("scale", [2.36e38, 3e38])
def test_a_scale_past_fp32_in_log2_units_is_refused(scfa, scale):
    assert scfa._lib.scfa_cache4_attn(*attn_args(scale=scale)) == 1
    from sparse_causal_flash_gb300.cache import KVCache4
    c = KVCache4(R=2, n_pages=4, Hq=4, Hkv=2, D=64, max_len=64, max_tokens=2, device="cpu")
    q, kv = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scale"):
        c.step(q, kv, kv, torch.ones(2, dtype=torch.int32), scale)


def test_the_largest_scale_of_a_step_is_one_that_attn_takes():
    from sparse_causal_flash_gb300.cache import _SCALES
    log2e = 1.4426950408889634
    most, above = np.float32(_SCALES[1]), np.nextafter(np.float32(_SCALES[1]), np.float32(np.inf))
    assert float(most) == _SCALES[1] and np.isfinite(np.float32(float(most) * log2e))
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(float(above) * log2e))


def test_status_words_of_a_new_cache_are_zero(scfa, monkeypatch):
    """Whatever the memory held before."""
    from sparse_causal_flash_gb300 import cache
    monkeypatch.setattr(cache, "workspace", lambda n, dev: torch.full((max(n, 256),), 7, dtype=torch.uint8, device=dev))
    c = cache.KVCache4(R=2, n_pages=4, Hq=4, Hkv=2, D=64, max_len=64, max_tokens=2, device="cpu")
    for ws in (c.ws_plan, c.ws_attn):
        assert int(ws[:4].view(torch.int32)[0]) == 0


class OnGpu:
    """What the binding asks of a tensor, for one said to lie on a GPU."""

    def __init__(self, *shape, dtype=torch.int32, dev=0, strides=None):
        t = torch.empty(1, dtype=dtype).expand(shape)
        self.shape, self.dtype, self.dev, self.strides = t.shape, dtype, dev, strides
        self.device = torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def get_device(self):
        return self.dev

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides or torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return self.strides is None or self.strides == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("ws,fine", [
    (dict(), True), (dict(dev=-1), False), (dict(dev=1), False), (dict(dtype=torch.int32), False), (dict(strides=(2,)), False)])
def test_binding_refuses_workspaces_it_cannot_take(scfa, monkeypatch, ws, fine):
    """The kernels write the workspace: one in host memory, on another device or of other strides would be a wild address."""
    calls = []
    monkeypatch.setattr(scfa, "_launch", lambda fn, *a: calls.append(fn))
    ws, u8, bf = OnGpu(1 << 20, **{"dtype": torch.uint8, **ws}), torch.uint8, torch.bfloat16
    v = {n: OnGpu(n) for n in (1, 4, 5, 9)}
    plan = lambda: scfa.scfa_cache4_plan(v[4], v[4], None, v[9], v[1], OnGpu(4, 3), 64, 9, v[4], v[1], v[5], v[4], v[4], ws)
    rows = OnGpu(4, 2, 64, dtype=bf)
    attn = lambda: scfa.scfa_cache4_attn(rows, OnGpu(9, 2, 64 * 68, dtype=u8), 64, OnGpu(4, 3), v[5], v[4], 0.125, rows,
                                         OnGpu(4, 2, dtype=torch.float32), ws)
    for call in (plan, attn):
        if fine:
            call()
        else:
            with pytest.raises(ValueError, match="ws"):
                call()
    assert len(calls) == (2 if fine else 0)


@pytest.mark.parametrize("ps,mp", [(16, 2 ** 27 - 1), (16, 2 ** 27 - 15), (64, 2 ** 25 - 1), (128, 2 ** 24 - 1)])
def test_a_block_table_of_positions_past_ints_is_refused(scfa, ps, mp):
    """Behind 2^31 - 256 the end of a unit of 128 tokens is no 32-bit int."""
    assert 2 ** 31 - 256 < ps * mp < 2 ** 31
    assert scfa._lib.scfa_cache4_plan(*plan_args(ps=ps, mp=mp)) == 2
    assert scfa._lib.scfa_cache4_attn(*attn_args(ps=ps, mp=mp)) == 2


@pytest.mark.parametrize("kw", [dict(kt=0), dict(vt=0), dict(kh=0), dict(vh=32), dict(kt=64), dict(kt=-56), dict(vt=256, vh=256)])
def test_rows_to_write_that_share_elements_are_refused(scfa, kw):
    """An expanded output would hold whichever row came last."""
    assert scfa._lib.scfa_cache4_read(*rows_args(True, **kw)) == 1
    if "kt" in kw or "kh" in kw:
        o = {{"kt": "ot", "kh": "oh"}[x]: v for x, v in kw.items()}
        assert scfa._lib.scfa_cache4_attn(*attn_args(**o)) == 1


def test_strides_of_a_single_row_are_not_looked_at(scfa):
    """No launch: the call is refused for its dtype behind, or its workspace before, the strides."""
    assert scfa._lib.scfa_cache4_attn(*attn_args(N=1, ot=0, nb=128)) == 3
    assert scfa._lib.scfa_cache4_attn(*attn_args(Hq=1, Hkv=1, oh=0, nb=128)) == 3
