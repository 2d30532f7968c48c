"""Rotary positions without a GPU: the oracle against hand-worked values, autograd and differences; the table of
frequencies; the refusals of the C ABI and of the binding."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import rope as orope


@pytest.fixture(scope="module")
def scfa():
    from sparse_causal_flash_gb300 import build
    build.build()
    import sparse_causal_flash_gb300 as s
    return s


# ---------------------------------------------------------------- the oracle
@pytest.mark.parametrize("interleaved,at", [(False, (0, 2)), (True, (0, 1))])
def test_quarter_turn_by_hand(interleaved, at):
    x = np.zeros((1, 1, 6))
    x[0, 0, list(at)] = 3.0, 4.0
    x[0, 0, 5] = 7.0  # behind the turned channels
    y = orope.turn(x, [1], [math.pi / 2, 0.0], interleaved, factor=2.0)
    want = np.zeros(6)
    want[list(at)] = -8.0, 6.0
    want[5] = 7.0
    assert np.allclose(y[0, 0], want, atol=1e-15)


def test_scores_depend_on_the_distance_only():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    a = (orope.turn(q, [17], f) * orope.turn(k, [5], f)).sum()
    b = (orope.turn(q, [1012], f) * orope.turn(k, [1000], f)).sum()
    assert abs(a - b) < 1e-10


@pytest.mark.parametrize("with_norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradients(with_norm, interleaved):
    g = np.random.default_rng(1)
    x, dy, w = g.standard_normal((3, 2, 16)), g.standard_normal((3, 2, 16)), 1 + 0.3 * g.standard_normal(16)
    f, pos = g.random(5), np.array([0, 7, -3])
    kw = dict(interleaved=interleaved, factor=1.3)
    if with_norm:
        kw.update(w=w, eps=1e-3)
    dx, dw = orope.backward(dy, pos, f, x=x, **kw)

    def loss(x, w):
        return (orope.forward(x, pos, f, **{**kw, **({"w": w} if with_norm else {})}) * dy).sum()

    h = 1e-6
    for _ in range(12):
        u = g.standard_normal(x.shape)
        assert abs((loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-6
    if with_norm:
        u = g.standard_normal(16)
        assert abs((loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h) - (dw * u).sum()) < 1e-6


# ---------------------------------------------------------------- frequencies
def test_table_is_exact(scfa):
    f = np.concatenate([10000.0 ** (-np.arange(64) / 64), [math.pi, -math.pi, 3 * math.pi, 0.0, -1e-9, 100.0]])
    table = scfa.rope_table(f, "cpu")
    for x, t in zip(f.tolist(), table.tolist()):
        turns = Fraction(x / (2 * math.pi))  # rounded to float64, then exact
        d = (Fraction(t % 2 ** 64, 2 ** 64) - turns) % 1
        # the table has 2^-64 turns; x / (2 pi) minus its whole turns is exact
        assert min(d, 1 - d) <= Fraction(1, 2 ** 64)


@pytest.mark.parametrize("scaling", ["", "linear", "base", "parts"])
def test_frequencies(scfa, scaling):
    from sparse_causal_flash_gb300.rope import rope_frequencies
    rot, s, trained = 64, 8.0, 4096
    plain, _ = rope_frequencies(rot)
    f, factor = rope_frequencies(rot, scaling=scaling, stretch=s, trained=trained)
    assert np.allclose(plain.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    ratio = (f / plain).numpy()
    if scaling == "":
        assert np.array_equal(ratio, np.ones(32)) and factor == 1.0
    elif scaling == "linear":
        assert np.allclose(ratio, 1 / s) and factor == 1.0
    elif scaling == "base":
        assert abs(ratio[0] - 1) < 1e-12 and abs(ratio[-1] - 1 / s) < 1e-12 and np.all(np.diff(ratio) < 0)
    else:
        turns = trained * plain.numpy() / (2 * math.pi)
        assert np.allclose(ratio[turns >= 32], 1) and np.allclose(ratio[turns <= 1], 1 / s)
        assert abs(factor - (0.1 * math.log(s) + 1)) < 1e-15 and np.all(np.diff(ratio) <= 1e-15)
    for bad in (dict(rot=63), dict(rot=64, scaling="other"), dict(rot=64, scaling="parts"), dict(rot=64, stretch=0.5)):
        with pytest.raises(ValueError):
            rope_frequencies(**bad)


# ---------------------------------------------------------------- refusals
FAKE = ctypes.c_void_p(4096)


def fwd_args(**kw):
    a = dict(q=FAKE, qt=512, qh=64, k=FAKE, kt=512, kh=64, pos=FAKE, count=None, table=FAKE, N=8, Hq=4, Hkv=2, D=64, rot=64,
             il=0, factor=1.0, wq=None, wk=None, eps=1e-6, dt=0, qo=FAKE, qot=256, qoh=64, ko=FAKE, kot=128, koh=64, st=None)
    a.update(kw)
    return list(a.values())


def bwd_args(**kw):
    a = dict(dq=FAKE, dqt=512, dqh=64, dk=FAKE, dkt=512, dkh=64, q=FAKE, qt=512, qh=64, k=FAKE, kt=512, kh=64, pos=FAKE,
             count=None, table=FAKE, N=8, Hq=4, Hkv=2, D=64, rot=64, il=0, factor=1.0, wq=FAKE, wk=FAKE, eps=1e-6, dt=0,
             qo=FAKE, qot=256, qoh=64, ko=FAKE, kot=128, koh=64, dwq=FAKE, dwk=FAKE, ws=FAKE, nb=1 << 24, st=None)
    a.update(kw)
    return list(a.values())


BOTH = [(dict(pos=None), 1), (dict(N=-1), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1), (dict(rot=63), 1), (dict(rot=66), 1),
        (dict(rot=-2), 1), (dict(table=None), 1), (dict(il=2), 1), (dict(factor=float("inf")), 1),
        (dict(factor=float("nan")), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(D=96), 2), (dict(dt=7), 2),
        (dict(N=1 << 29), 2), (dict(qo=None), 1), (dict(qo=ctypes.c_void_p(4100)), 1), (dict(ko=None), 1),
        (dict(qot=12), 1), (dict(qoh=32), 1), (dict(kot=64, koh=64), 1)]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qt=513), 1), (dict(kh=4), 1), (dict(wk=FAKE), 1), (dict(wq=FAKE), 1),
    (dict(q=ctypes.c_void_p(4098)), 1)])
def test_fwd_refusals(scfa, kw, code):
    assert scfa._lib.scfa_rope_fwd(*fwd_args(**kw)) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(dq=None), 1), (dict(dk=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(wk=None), 1), (dict(dwq=None), 1),
    (dict(dwk=None), 1), (dict(wq=None), 1), (dict(wq=None, wk=None), 1), (dict(ws=None), 3), (dict(nb=100), 3),
    (dict(ws=ctypes.c_void_p(4097)), 3), (dict(qt=4), 1)])
def test_bwd_refusals(scfa, kw, code):
    assert scfa._lib.scfa_rope_bwd(*bwd_args(**kw)) == code


@pytest.mark.parametrize("kw", [dict(table=ctypes.c_void_p(4104)), dict(wq=ctypes.c_void_p(4100), wk=FAKE),
                                dict(wq=FAKE, wk=ctypes.c_void_p(4108))])
def test_tables_and_weights_start_on_16_bytes(scfa, kw):
    assert scfa._lib.scfa_rope_fwd(*fwd_args(**kw)) == 1
    assert scfa._lib.scfa_rope_bwd(*bwd_args(**kw)) == 1


def test_no_tokens_is_no_error(scfa):
    assert scfa._lib.scfa_rope_fwd(*fwd_args(N=0, q=None, k=None, qo=None, ko=None)) == 0
    assert scfa._lib.scfa_rope_bwd(*bwd_args(N=0, dq=None, dk=None, qo=None, ko=None, wq=None, wk=None, dwq=None, dwk=None,
                                             ws=None, nb=0)) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(scfa):
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table = scfa.rope_table([1.0, 0.5], "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        scfa.scfa_rope_fwd(x, None, torch.zeros(2, dtype=torch.int32), table, x, None)
    with pytest.raises(ValueError):
        scfa.rope_table([float("nan")], "cpu")
    with pytest.raises(ValueError):
        scfa.rope_table([[1.0]], "cpu")


def test_frequencies_of_ones_own_make_pairs(scfa):
    """Channels that turn are twice the frequencies: an odd number of channels is refused, also with frequencies given."""
    from sparse_causal_flash_gb300.rope import Rope
    r = Rope(4, inv_freq=[1.0, 0.5], factor=1.5, device="cpu")
    assert (r.rot, r.factor, r.table.numel()) == (4, 1.5, 2)
    for rot, f in ((5, [1.0, 0.5]), (1, []), (-1, [1.0]), (4, [1.0]), (4, [1.0, 0.5, 0.2])):
        with pytest.raises(ValueError):
            Rope(rot, inv_freq=f, device="cpu")
