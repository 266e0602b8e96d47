"""Rotary positions in every form on the GPU against the fp64 oracle: layouts, parts of heads, types, odd sizes
and alignments, positions of every kind, the gradient, in place and into strided rows.

Tolerance.  A turned element is A (a c - b s), formed in fp32 from c and s that are off by at most e of
the pair's length r = |A| sqrt(a^2 + b^2) (e = 2^-20 for 16-bit elements, 2^-22 for fp32), with three roundings
of at most 2^-24 r each (the product with A, the product, the sum: 2^-22 r in all), then rounded once:
u |y| + (e + 2^-22) r, u half a step of the type (bf16 2^-8, fp16 2^-11, fp32 2^-24), at least half its
smallest step.  Elements beside the part are the input's bits.
"""
import numpy as np
import pytest
import torch

import oracle
import attention_attn_fwd_08_gb300 as A

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def rows_of(n, width, dt, seed, stride=None, off=0):
    """Rows on the GPU, `stride` apart, the first `off` elements into their buffer."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, width), generator=g).to(T[dt])
    if stride is None and not off:
        return x.to(DEV)
    stride = stride or width
    buf = torch.full((n * stride + off + 64,), 7.0, dtype=T[dt], device=DEV)
    v = buf.as_strided((n, width), (stride, 1), off)
    v.copy_(x)
    return v


def check(dt, x0, y, pos, H, freqs, start, layout, backward):
    kw = dict(H=H, inv_freq=freqs.inv_freq, start=start, interleaved=layout == "interleaved", amplitude=freqs.amplitude,
              backward=backward)
    x, got = f64(x0), f64(y)
    ref = oracle.turn_part(x, pos, **kw)
    n, hd, d = x.shape[0], x.shape[1] // H, freqs.rotary_dim
    part = lambda a: a.reshape(n, H, hd)[:, :, start:start + d]
    p = part(x)
    r = np.hypot(p[..., 0::2], p[..., 1::2]).repeat(2, axis=2) if layout == "interleaved" else \
        np.tile(np.hypot(p[..., :d // 2], p[..., d // 2:]), 2)
    e = 2.0 ** -22 if dt == "f32" else 2.0 ** -20
    tol = U[dt] * np.abs(part(ref)) + (e + 2.0 ** -22) * abs(freqs.amplitude) * r + TINY[dt]
    off = np.abs(part(got) - part(ref))
    assert (off <= tol).all(), "off by %.3g where %.3g is allowed" % (off.max(), tol.flat[off.argmax()])
    for a, b in ((0, start), (start + d, hd)):
        assert (got.reshape(n, H, hd)[:, :, a:b] == x.reshape(n, H, hd)[:, :, a:b]).all()


def run(dt, n, H, hd, freqs, layout, start=0, backward=False, seed=1, xs=None, off=0, positions=None, inplace=False):
    x = rows_of(n, H * hd, dt, seed, xs, off)
    x0 = x.clone()
    pos = np.arange(n) if positions is None else np.asarray(positions)
    pd = None if positions is None else torch.tensor(pos, dtype=torch.int32, device=DEV)
    y = A.attn_rope_ex(x, freqs, H=H, positions=pd, layout=layout, rotary_start=start, backward=backward, out=x if inplace else None)
    torch.cuda.synchronize()
    assert inplace == (y.data_ptr() == x.data_ptr())
    check(dt, x0, y, pos, H, freqs, start, layout, backward)
    if not inplace:
        assert (x == x0).all()
    return x0, y


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,part,start", [(128, 128, 0), (64, 32, 0), (64, 32, 32), (80, 20, 0), (96, 24, 8), (256, 256, 0),
                                           (10, 6, 3), (2, 2, 0), (192, 64, 128), (1024, 256, 512), (72, 18, 1)])
def test_layouts_types_and_parts(dt, layout, hd, part, start):
    for backward in (False, True):
        run(dt, 19, 5, hd, A.attn_rope_freqs(part), layout, start, backward, seed=hd + part)


@pytest.mark.parametrize("n,H", [(1, 1), (1, 65), (3, 40), (700, 3), (5003, 2), (2, 700), (1, 4097)])
@pytest.mark.parametrize("layout,dt", [("half", "bf16"), ("interleaved", "f32"), ("half", "f16")])
def test_sizes(n, H, layout, dt):
    run(dt, n, H, 32, A.attn_rope_freqs(32 if layout == "half" else 16), layout, seed=n + H)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt,xs,off", [("bf16", 8 * 64 + 8, 0), ("bf16", 8 * 64 + 4, 0), ("bf16", 8 * 64 + 1, 0), ("bf16", None, 4),
                                       ("f16", None, 1), ("f32", 8 * 64 + 2, 2), ("f32", 8 * 64 + 1, 0), ("bf16", 8 * 64 + 2, 2)])
@pytest.mark.parametrize("inplace", [False, True])
def test_strides_and_alignments(layout, dt, xs, off, inplace):
    run(dt, 33, 8, 64, A.attn_rope_freqs(48), layout, 8, xs=xs, off=off, inplace=inplace)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_positions_of_every_kind(dt):
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 1000000, 1000000, 30000, -77777, 65535, 5]
    f = A.attn_rope_freqs(64, 500000.0, scaling="ramp", factor=16.0, original_length=8192)
    run(dt, len(pos), 3, 64, f, "half", positions=pos)
    # frequencies of every size and sign, and none
    f = A.RopeFreqs([2.0 ** 32, -2.0 ** 31 - 0.3, 7.1, 1.0, 0.1, 1e-9, 0.0, -1e-300], -0.75)
    run(dt, len(pos), 3, 20, f, "interleaved", positions=pos, start=2)


@pytest.mark.parametrize("backward", [False, True])
def test_far_rows_keep_their_angle(backward):
    run("f32", 64, 1, 128, A.attn_rope_freqs(128, scaling="base", factor=32.0), "half", positions=list(range(2 ** 30, 2 ** 30 + 64)),
        backward=backward)


def test_batches_without_positions():
    f = A.attn_rope_freqs(64)
    x = rows_of(3 * 50, 4 * 64, "bf16", 5).view(3, 50, 256)
    y = A.attn_rope_ex(x, f, H=4, pos=1000)
    check("bf16", x.view(150, 256), y.view(150, 256), np.tile(1000 + np.arange(50), 3), 4, f, 0, "half", False)
    p = torch.arange(150, dtype=torch.int32, device=DEV).view(3, 50)
    y = A.attn_rope_ex(x, f, H=4, positions=p)
    check("bf16", x.view(150, 256), y.view(150, 256), np.arange(150), 4, f, 0, "half", False)
    assert A.attn_rope_ex(x[:, :0], f, H=4).shape == (3, 0, 256)
    assert A.attn_rope_ex(x[:0], f, H=4).shape == (0, 50, 256)
    # a batch of one row each, and one batch
    for v in (x[:, 7:8], x[1:2], x[1:2, 7:8]):
        y = A.attn_rope_ex(v, f, H=4, pos=9)
        n = v.numel() // 256
        check("bf16", v.reshape(n, 256), y.view(n, 256), 9 + np.arange(n) % v.shape[1], 4, f, 0, "half", False)


def test_columns_of_a_fused_projection():
    """Query and key heads in place inside [q | k | v] rows, and out of them into other columns; what lies beside stays."""
    f = A.attn_rope_freqs(64, scaling="linear", factor=2.0)
    qkv = rows_of(37, 8 * 64, "bf16", 6)
    q0 = qkv.clone()
    A.attn_rope_ex(qkv[:, :6 * 64], f, H=6, out=qkv[:, :6 * 64])
    check("bf16", q0[:, :384], qkv[:, :384], np.arange(37), 6, f, 0, "half", False)
    assert (qkv[:, 384:] == q0[:, 384:]).all()
    # columns 0-2 into columns 4-6 of the same rows
    w = q0.clone()
    A.attn_rope_ex(w[:, :192], f, H=3, out=w[:, 256:448])
    check("bf16", q0[:, :192], w[:, 256:448], np.arange(37), 3, f, 0, "half", False)
    assert (w[:, :256] == q0[:, :256]).all() and (w[:, 448:] == q0[:, 448:]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """The directional derivative of <w, rope(x)> along e, by differences of the kernel's own outputs (a linear
    map: exact up to its rounding), is <backward(w), e>."""
    f = A.attn_rope_freqs(32, scaling="ramp", factor=8.0, original_length=1024)
    x, w, e = (rows_of(40, 2 * 48, "f32", s) for s in (11, 12, 13))
    kw = dict(H=2, layout=layout, rotary_start=16, pos=3000)
    d = (A.attn_rope_ex(x + e, f, **kw).double() - A.attn_rope_ex(x - e, f, **kw).double()) / 2
    left = (w.double() * d).sum()
    right = (A.attn_rope_ex(w, f, backward=True, **kw).double() * e.double()).sum()
    # each output off by at most 2^-21 of its pair's length (about 2), over 40 * 96 products
    assert abs(left - right) <= 2.0 ** -21 * 4 * (w.abs().double().sum() + e.abs().double().sum())


def test_values_that_are_not_finite_stay_in_their_pair():
    x = rows_of(4, 64, "bf16", 9)
    x[1, 3], x[2, 40] = float("nan"), float("inf")
    y = A.attn_rope_ex(x, A.attn_rope_freqs(64), H=1, pos=3)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 3] = want[1, 35] = want[2, 40] = want[2, 8] = True
    assert (bad == want).all()


def test_streams_capture_and_other_rows():
    f = A.attn_rope_freqs(128)
    x = rows_of(64, 40 * 128, "bf16", 21)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    ref = A.attn_rope_ex(x, f, H=40, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = A.attn_rope_ex(x, f, H=40, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attn_rope_ex(x, f, H=40, positions=pos, out=out)
    pos += 100  # read at replay
    g.replay()
    torch.cuda.synchronize()
    check("bf16", x, out, 100 + np.arange(64), 40, f, 0, "half", False)


def test_rows_past_four_gigabytes():
    """Offsets beyond 32 bits: the last rows of a buffer of more than 2^32 bytes."""
    f, n, w = A.attn_rope_freqs(128), 1100000, 16 * 128
    x = torch.empty((n, w), dtype=torch.bfloat16, device=DEV)
    tail = rows_of(5, w, "bf16", 31)
    x[:2], x[-5:] = tail[:2], tail
    y = A.attn_rope_ex(x, f, H=16)
    torch.cuda.synchronize()
    check("bf16", tail, y[-5:], np.arange(n - 5, n), 16, f, 0, "half", False)
    check("bf16", tail[:2], y[:2], np.arange(2), 16, f, 0, "half", False)
