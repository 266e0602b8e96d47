"""Rotary positions in every form, without a GPU: refusals by the C ABI and the binding, the scaled
frequencies against their definitions, and pins of the oracle's turn."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_attn_fwd_08_gb300 as A
import oracle

BAD = ctypes.c_void_p(0x100000)  # never dereferenced: every case fails validation first
FAR = ctypes.c_void_p(0x900000)
ODD = ctypes.c_void_p(0x100001)
FREQS = (ctypes.c_double * 128)(*[0.5] * 128)


def call(**kw):
    a = dict(dt=2, x=BAD, xs=512, y=FAR, ys=512, positions=None, pos=0, period=8, rows=16, H=4, hd=128, rd=64, rs=0, inter=0,
             freqs=FREQS, amplitude=1.0, backward=0, stream=None)
    a.update(kw)
    return A.lib().attn_rope_ex(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=3), A.ERR_INVALID_ARG), (dict(dt=-1), A.ERR_INVALID_ARG),
    (dict(rows=-1), A.ERR_INVALID_ARG), (dict(H=0), A.ERR_INVALID_ARG), (dict(H=65536), A.ERR_INVALID_ARG),
    (dict(hd=0), A.ERR_INVALID_ARG), (dict(rd=0), A.ERR_INVALID_ARG), (dict(rd=63), A.ERR_INVALID_ARG),
    (dict(rd=130), A.ERR_INVALID_ARG), (dict(rs=-2), A.ERR_INVALID_ARG), (dict(rs=66), A.ERR_INVALID_ARG),
    (dict(rs=2 ** 31 - 1), A.ERR_INVALID_ARG),
    (dict(inter=2), A.ERR_INVALID_ARG), (dict(backward=-1), A.ERR_INVALID_ARG),
    (dict(amplitude=float("nan")), A.ERR_INVALID_ARG), (dict(amplitude=float("inf")), A.ERR_INVALID_ARG),
    (dict(freqs=None), A.ERR_INVALID_ARG), (dict(freqs=(ctypes.c_double * 32)(*[2.0 ** 33] * 32)), A.ERR_INVALID_ARG),
    (dict(freqs=(ctypes.c_double * 32)(*[float("nan")] * 32)), A.ERR_INVALID_ARG),
    (dict(hd=1026, xs=8192, ys=8192), A.ERR_UNSUPPORTED), (dict(hd=512, rd=258, xs=2048, ys=2048), A.ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 1), A.ERR_UNSUPPORTED),
    (dict(pos=-1), A.ERR_INVALID_ARG), (dict(period=0), A.ERR_INVALID_ARG), (dict(pos=2 ** 31 - 8, period=9), A.ERR_INVALID_ARG),
    (dict(xs=511), A.ERR_INVALID_ARG), (dict(ys=500), A.ERR_INVALID_ARG), (dict(xs=2 ** 60), A.ERR_INVALID_ARG),
    (dict(x=None), A.ERR_INVALID_ARG), (dict(y=None), A.ERR_INVALID_ARG), (dict(x=ODD), A.ERR_INVALID_ARG),
    (dict(y=ODD), A.ERR_INVALID_ARG), (dict(positions=ODD), A.ERR_INVALID_ARG),
    (dict(y=BAD, xs=512, ys=1024), A.ERR_INVALID_ARG),                      # in place with another stride
    (dict(y=ctypes.c_void_p(0x100010)), A.ERR_INVALID_ARG),                 # rows that overlap
    (dict(y=ctypes.c_void_p(0x100000 + 2 * 256), xs=1024, ys=1024), A.ERR_INVALID_ARG),
    (dict(x=ctypes.c_void_p(0x100000 + 2 * 256), y=BAD, xs=768, ys=768), A.ERR_INVALID_ARG),
    (dict(rows=0, x=None, y=None), A.OK),
])
def test_rules(kw, expect):
    assert call(**kw) == expect


# ------------------------------------------------------------------ the binding
def test_binding_refuses():
    f = A.attn_rope_freqs(64)
    x = torch.zeros(6, 4 * 128, dtype=torch.bfloat16)
    for bad in (dict(H=3), dict(layout="neighbours"), dict(rotary_start=65), dict(rotary_start=-1),
                dict(positions=torch.zeros(6, dtype=torch.int64)), dict(positions=torch.zeros(5, dtype=torch.int32)),
                dict(positions=torch.zeros(12, dtype=torch.int32)[::2]), dict(out=torch.zeros(6, 512)),
                dict(out=torch.zeros(5, 512, dtype=torch.bfloat16)), dict()):  # (the last: host tensors)
        with pytest.raises(ValueError):
            A.attn_rope_ex(x, f, **dict(dict(H=4), **bad))
    with pytest.raises(ValueError):
        A.attn_rope_ex(x[0], f, H=4)
    with pytest.raises(ValueError):  # overlapping rows
        A.attn_rope_ex(torch.zeros(2000, dtype=torch.bfloat16).as_strided((6, 512), (256, 1)), f, H=4)
    with pytest.raises(ValueError):  # batches that are not evenly spaced
        A.attn_rope_ex(torch.zeros(2, 9, 512, dtype=torch.bfloat16)[:, :6], f, H=4)
    with pytest.raises(TypeError):
        A.attn_rope_ex(x.long(), f, H=4)


@pytest.mark.parametrize("H", [0, -4])
def test_binding_refuses_no_heads(H):
    with pytest.raises(ValueError, match="H = "):
        A.attn_rope_ex(torch.zeros(6, 512, dtype=torch.bfloat16), A.attn_rope_freqs(64), H=H)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(theta=0.0), dict(theta=float("inf")), dict(factor=2.0),
    dict(scaling="wide", factor=2.0), dict(scaling="linear", factor=0.0), dict(scaling="base", rotary_dim=2, factor=2.0),
    dict(scaling="ramp", factor=2.0), dict(scaling="bands", factor=2.0, original_length=0),
    dict(scaling="bands", factor=2.0, original_length=100, slow=4.0), dict(scaling="ramp", factor=2.0, original_length=100, theta=0.5),
    dict(scaling="linear", factor=2.0, amplitude=float("nan"))])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        A.attn_rope_freqs(**dict(dict(rotary_dim=64), **kw))


@pytest.mark.parametrize("kw", [
    dict(scaling="ramp", original_length=float("inf")), dict(scaling="ramp", original_length=100, fast=float("inf")),
    dict(scaling="base", rotary_dim=4, factor=1e300), dict(scaling="base", rotary_dim=4, factor=1e-300)])
def test_frequencies_refuse_what_is_not_finite(kw):
    with pytest.raises(ValueError, match="finite|no double"):
        A.attn_rope_freqs(**dict(dict(rotary_dim=64, factor=2.0), **kw))


def test_raw_frequencies():
    f = A.RopeFreqs([1.0, -0.25], 2.0)
    assert f.rotary_dim == 4 and f.inv_freq == (1.0, -0.25) and f.amplitude == 2.0
    for bad in ([], [0.0] * 129, [float("nan")], [2.0 ** 33]):
        with pytest.raises(ValueError):
            A.RopeFreqs(bad)


def near(a, b):
    return np.abs(np.array(a) - np.array(b)).max() <= 1e-14 * np.abs(b).max()


def test_frequencies_plain_linear_base():
    i = np.arange(32)
    f = 10000.0 ** (-i / 32)
    assert near(A.attn_rope_freqs(64).inv_freq, f)
    assert near(A.attn_rope_freqs(64, scaling="linear", factor=4).inv_freq, f / 4)
    g = A.attn_rope_freqs(64, scaling="base", factor=4.0).inv_freq
    assert g[0] == 1.0 and abs(g[-1] / f[-1] * 4 - 1) < 1e-13  # the first pair stays, the last is divided by the factor


def test_frequencies_ramp():
    d, theta, L, s = 128, 10000.0, 4096, 8.0
    f = theta ** (-2.0 * np.arange(d // 2) / d)
    r = A.attn_rope_freqs(d, theta, scaling="ramp", factor=s, original_length=L)
    turns = L * f / (2 * math.pi)
    ratio = np.array(r.inv_freq) / f
    # pairs beyond the two borders, but for the one at which each is rounded outwards
    assert np.allclose(ratio[:np.flatnonzero(turns > 32).max()], 1, rtol=1e-14)
    assert np.allclose(ratio[np.flatnonzero(turns < 1).min() + 1:], 1 / s, rtol=1e-14)
    mid = ratio[(ratio < 1) & (ratio > 1.0001 / s)]
    assert len(mid) > 5 and np.allclose(np.diff(mid), np.diff(mid)[0], rtol=1e-9)  # a straight ramp
    assert abs(r.amplitude - (0.1 * math.log(8) + 1)) < 1e-15
    assert A.attn_rope_freqs(d, scaling="ramp", factor=s, original_length=L, amplitude=1.0).amplitude == 1.0


@pytest.mark.parametrize("L,slow,fast", [(4, 1.0, 32.0), (6.28, 1.0, 32.0), (100, 32.0, 64.0), (2, 0.1, 0.2), (10, 1.0, 32.0)])
def test_frequencies_ramp_where_pairs_turn_slowly(L, slow, fast):
    """Pairs that make at most `slow` turns are scaled whole, also where no pair makes more."""
    f = 10000.0 ** (-np.arange(32) / 32)
    got = np.array(A.attn_rope_freqs(64, scaling="ramp", factor=8.0, original_length=L, slow=slow, fast=fast).inv_freq)
    turns = L * f / (2 * math.pi)
    behind = np.flatnonzero(turns <= slow)
    behind = behind if turns[0] <= slow else behind[1:]  # (the border is rounded outwards to a whole pair)
    assert len(behind) and near(got[behind], f[behind] / 8)


def test_frequencies_ramp_where_all_turn_fast():
    f = 10000.0 ** (-np.arange(32) / 32)
    assert near(A.attn_rope_freqs(64, scaling="ramp", factor=8.0, original_length=10 ** 12).inv_freq, f)


def test_frequencies_bands():
    d, theta, L, s = 128, 500000.0, 8192, 8.0
    f = theta ** (-2.0 * np.arange(d // 2) / d)
    r = A.attn_rope_freqs(d, theta, scaling="bands", factor=s, original_length=L)
    turns = L * f / (2 * math.pi)
    got = np.array(r.inv_freq)
    assert near(got[turns >= 4], f[turns >= 4]) and near(got[turns <= 1], f[turns <= 1] / s) and r.amplitude == 1.0
    m = (turns > 1) & (turns < 4)
    w = (turns[m] - 1) / 3
    assert m.sum() > 2 and near(got[m], (1 - w) * f[m] / s + w * f[m])


# ------------------------------------------------------------------ the oracle
def test_oracle_half_layout_is_the_rotate_half_turn():
    x = np.random.default_rng(1).standard_normal((7, 3 * 16))
    f = 10000.0 ** (-2.0 * np.arange(8) / 16)
    got = oracle.turn_part(x, range(5, 12), H=3, inv_freq=f)
    assert np.abs(got - oracle.rope(x[None], head_dim=16, pos=5)[0]).max() < 1e-13


def test_oracle_layouts_parts_and_transpose():
    rng = np.random.default_rng(2)
    x, f = rng.standard_normal((5, 2 * 12)), [0.3, 0.02, -1.7]
    pos = [0, 1, -4, 100, 7]
    h = oracle.turn_part(x, pos, H=2, inv_freq=f, start=4, amplitude=1.5)
    # the interleaved turn is the half turn of the elements in another order
    order = np.arange(12)
    order[4:10] = [4, 7, 5, 8, 6, 9]
    y = x.reshape(5, 2, 12)[:, :, order].reshape(5, 24)
    g = oracle.turn_part(y, pos, H=2, inv_freq=f, start=4, amplitude=1.5, interleaved=True)
    assert np.abs(g.reshape(5, 2, 12) - h.reshape(5, 2, 12)[:, :, order]).max() < 1e-14
    assert (h.reshape(5, 2, 12)[:, :, [0, 1, 2, 3, 10, 11]] == x.reshape(5, 2, 12)[:, :, [0, 1, 2, 3, 10, 11]]).all()
    # one pair, written out
    a, b, t = x[2, 4], x[2, 7], -4 * 0.3
    assert abs(h[2, 4] - 1.5 * (a * math.cos(t) - b * math.sin(t))) < 1e-14
    assert abs(h[2, 7] - 1.5 * (b * math.cos(t) + a * math.sin(t))) < 1e-14
    # <R x, y> = <x, R^T y>, by row
    w = rng.standard_normal(x.shape)
    back = oracle.turn_part(w, pos, H=2, inv_freq=f, start=4, amplitude=1.5, backward=True)
    assert np.abs((h * w).sum(1) - (x * back).sum(1)).max() < 1e-12


def test_oracle_angle_at_far_positions():
    """theta = pi / 8192 in doubles: its turns at position 2^30 are known from the double's own value."""
    f = 2.0 ** -20 + 2.0 ** -50
    got = oracle.turn_part(np.array([[1.0, 0.0]]), [2 ** 30], H=1, inv_freq=[f])
    t = 1024.0 + 2.0 ** -20  # exact
    assert abs(got[0, 0] - math.cos(t)) < 1e-12 and abs(got[0, 1] - math.sin(t)) < 1e-12
