"""Attention of prompt chunks over a paged cache, without a GPU: refusals by the C ABI before any launch
and by the binding before any pointer reaches the library, the workspace's size, and pins of the
oracle."""
import ctypes

import numpy as np
import pytest
import torch

import attention_attn_fwd_08_gb300 as A
import oracle

BAD = ctypes.c_void_p(0x1000)  # never dereferenced: every case fails validation first
ODD = ctypes.c_void_p(0x1002)
HALF = ctypes.c_void_p(0x1008)


def prefill(**kw):
    a = dict(dt=2, cache=3, q=BAD, qs=1024, kc=BAD, vc=BAD, ksc=BAD, vsc=BAD, o=BAD, lse=None, ws=BAD, wsb=1 << 40, cu=BAD,
             lengths=BAD, table=BAD, batch=2, total=8, num_pages=10, page=16, max_pages=4, H=8, Hkv=4, hd=128, scale=0.1,
             causal=1, window=0, softcap=0.0, stream=None)
    a.update(kw)
    return A.lib().attn_paged_prefill(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dt=7), A.ERR_INVALID_ARG), (dict(dt=3), A.ERR_INVALID_ARG), (dict(cache=5), A.ERR_INVALID_ARG),
    (dict(cache=-1), A.ERR_INVALID_ARG), (dict(dt=0), A.ERR_UNSUPPORTED), (dict(cache=0), A.ERR_UNSUPPORTED),
    (dict(cache=1), A.ERR_INVALID_ARG),                     # a 16-bit cache of the other type
    (dict(num_pages=-1), A.ERR_INVALID_ARG), (dict(max_pages=-1), A.ERR_INVALID_ARG),
    (dict(page=8), A.ERR_UNSUPPORTED), (dict(page=48), A.ERR_UNSUPPORTED), (dict(page=512), A.ERR_UNSUPPORTED),
    (dict(page=0), A.ERR_UNSUPPORTED), (dict(hd=96), A.ERR_UNSUPPORTED), (dict(hd=32), A.ERR_UNSUPPORTED),
    (dict(num_pages=1 << 26), A.ERR_UNSUPPORTED),           # more than 2^31 rows of one head
    (dict(max_pages=1 << 27), A.ERR_UNSUPPORTED),
    (dict(kc=None), A.ERR_INVALID_ARG), (dict(vc=ODD), A.ERR_INVALID_ARG), (dict(vc=HALF), A.ERR_INVALID_ARG),
    (dict(ksc=None), A.ERR_INVALID_ARG), (dict(vsc=ODD), A.ERR_INVALID_ARG),
    (dict(table=None), A.ERR_INVALID_ARG), (dict(table=ODD), A.ERR_INVALID_ARG),
    (dict(batch=-1), A.ERR_INVALID_ARG), (dict(batch=65536), A.ERR_INVALID_ARG), (dict(total=-1), A.ERR_INVALID_ARG),
    (dict(H=6), A.ERR_INVALID_ARG), (dict(Hkv=0), A.ERR_INVALID_ARG), (dict(H=0), A.ERR_INVALID_ARG),
    (dict(H=516, qs=516 * 128), A.ERR_UNSUPPORTED),         # a group of 129 heads
    (dict(total=2 ** 31 - 8), A.ERR_UNSUPPORTED),
    (dict(q=None), A.ERR_INVALID_ARG), (dict(q=HALF), A.ERR_INVALID_ARG), (dict(qs=1016), A.ERR_INVALID_ARG),
    (dict(qs=1028), A.ERR_INVALID_ARG), (dict(qs=(1 << 38) + 8), A.ERR_INVALID_ARG),
    (dict(o=None), A.ERR_INVALID_ARG), (dict(o=HALF), A.ERR_INVALID_ARG), (dict(lse=ODD), A.ERR_INVALID_ARG),
    (dict(cu=None), A.ERR_INVALID_ARG), (dict(cu=ODD), A.ERR_INVALID_ARG),
    (dict(lengths=None), A.ERR_INVALID_ARG), (dict(lengths=ODD), A.ERR_INVALID_ARG),
    (dict(scale=0.0), A.ERR_INVALID_ARG), (dict(scale=float("nan")), A.ERR_INVALID_ARG),
    (dict(softcap=-1.0), A.ERR_INVALID_ARG), (dict(window=-1), A.ERR_INVALID_ARG), (dict(causal=2), A.ERR_INVALID_ARG),
    (dict(ws=None), A.ERR_INVALID_ARG), (dict(ws=HALF), A.ERR_INVALID_ARG), (dict(wsb=8), A.ERR_INVALID_ARG),
    (dict(batch=0, table=None), A.OK), (dict(total=0, q=None, o=None, ws=None), A.OK),
])
def test_rules(kw, expect):
    assert prefill(**kw) == expect


def test_workspace_size():
    f = A.attn_paged_prefill_workspace_size
    for bad in ((0, 1, 8, 4, 64), (-1, 1, 8, 4, 64), (1, 0, 8, 4, 64), (1, 65536, 8, 4, 64), (1, 1, 8, 3, 64), (1, 1, 8, 4, 96),
                (1, 1, 516, 4, 64), (1, 1, 8, 0, 64), (2 ** 31 - 8, 1, 8, 8, 64)):
        assert f(*bad) == 0
    for total in (1, 300, 65536, 2 ** 31 - 600):
        for B in (1, 5, 65535):
            for G in (1, 7, 128):
                for hd in (64, 128, 256):
                    n = f(total, B, G * 3, 3, hd)
                    assert n > 0 and n % 4 == 0
                    # one byte less is refused, of the size that is asked for
                    kw = dict(total=total, batch=B, H=G * 3, Hkv=3, hd=hd, qs=G * 3 * hd, num_pages=1, max_pages=1)
                    assert prefill(wsb=n - 1, **kw) == A.ERR_INVALID_ARG


def test_workspace_size_has_room_for_any_beginning():
    """The layout begins on a multiple of 256 inside a workspace that begins on any multiple of 16: 240 bytes at most lie
    before it.  What it holds: the plan's lists, and 304 slots of partial rows, (m, l) and fp32 O each."""
    up = lambda n: -(-n // 256) * 256
    for total in (1, 29, 4096, 70001):
        for B in (1, 37, 1500):
            for G in (1, 3, 4, 128):
                for hd in (64, 128, 256):
                    rows = 128 if hd == 256 else 256
                    n = total // (rows // 128 * (128 // G)) + B  # items
                    lists = 256 + up(152 * 16) + up((B + 1) * 4) + up(n * 32) + up((n + 1) * 8)
                    assert A.attn_paged_prefill_workspace_size(total, B, G, 1, hd) >= 240 + lists + 304 * rows * (8 + 4 * hd)


# ------------------------------------------------------------------ the binding
B, Hkv, H, hd, page, P, most = 3, 2, 4, 64, 16, 9, 4


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def cache(dtype=torch.bfloat16):
    c = dict(k_cache=torch.zeros((P, Hkv, page, hd), dtype=dtype), v_cache=torch.zeros((P, Hkv, page, hd), dtype=dtype),
             page_table=i32(B, most))
    if dtype.itemsize == 1:
        c.update(k_scale=torch.ones(P, Hkv), v_scale=torch.ones(P, Hkv))
    return c


def call(c, **kw):
    a = dict(q=bf(5, H * hd), lengths=i32(B), cu_new=i32(B + 1), H=H, Hkv=Hkv)
    a.update(c)
    a.update(kw)
    return A.attn_paged_prefill(**a)


def test_binding_refuses_wrong_caches():
    c = cache()
    for change, kw, what in (({}, {}, "CUDA tensors"), (dict(k_cache=c["k_cache"][0]), {}, "k_cache"), ({}, dict(Hkv=4), "k_cache"),
                             (dict(v_cache=c["v_cache"][:5]), {}, "v_cache"), (dict(v_cache=c["v_cache"].half()), {}, "v_cache"),
                             (dict(page_table=c["page_table"].long()), {}, "page_table"),
                             (dict(page_table=i32(most, B).t()), {}, "contiguous")):
        with pytest.raises(ValueError, match=what):
            call(dict(c, **change), **kw)
    with pytest.raises(TypeError, match="cache dtype"):
        call(dict(c, k_cache=c["k_cache"].float()))
    with pytest.raises(ValueError, match="rows' dtype"):
        call(cache(torch.float16))
    e = cache(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="k_scale"):
        call(dict(e, k_scale=None))
    with pytest.raises(ValueError, match="v_scale"):
        call(dict(e, v_scale=torch.ones(P, 1)))
    with pytest.raises(TypeError, match="rows of a paged cache"):
        call(e, q=torch.zeros(5, H * hd))


@pytest.mark.parametrize("kw,what", [
    (dict(q=bf(5, H * hd + 8)), "q must"), (dict(q=bf(5, 2, H * hd)), "q must"), (dict(q=bf(H * hd, 5).t()), "q must"),
    (dict(q=bf(1, H * hd).expand(5, -1)), "q must"),
    (dict(lengths=i32(B + 1)), "lengths"), (dict(lengths=i32(B).long()), "lengths"), (dict(cu_new=i32(B)), "cu_new"),
    (dict(cu_new=i32(2 * B + 2)[::2]), "cu_new"),
    (dict(o=bf(4, H * hd)), "o must"), (dict(o=bf(5, H * hd).half()), "o must"), (dict(o=bf(5, 2 * H * hd)[:, :H * hd]), "contiguous"),
    (dict(lse=torch.zeros(5, H)), "lse"), (dict(lse=torch.zeros(H, 5, dtype=torch.float64)), "lse"),
    (dict(workspace=torch.zeros(100, dtype=torch.uint8)[::2]), "workspace"),
])
def test_binding_refuses_wrong_tensors(monkeypatch, kw, what):
    # (the cache check that asks for CUDA tensors comes first: the rest is checked with that one rule answered)
    monkeypatch.setattr(A, "_pools", lambda k, v, ks, vs, t, n, dt: (2, 2, P, page, hd, B, most))
    with pytest.raises(ValueError, match=what):
        call(cache(), **kw)


# ------------------------------------------------------------------ the oracle
def tokens_of(g, lengths, width):
    return [(g.standard_normal((n, width)), g.standard_normal((n, width))) for n in lengths]


@pytest.mark.parametrize("kw", [dict(), dict(window=4, softcap=2.0), dict(causal=False, window=3), dict(causal=False)])
def test_oracle_is_the_dense_one_on_each_sequence(kw):
    g = np.random.default_rng(3)
    Hq, Hk, d = 4, 2, 8
    lengths, new = [10, 3, 0, 6, 7], [4, 3, 0, 1, 0]
    tokens = tokens_of(g, lengths, Hk * d)
    cu = np.concatenate([[1], 1 + np.cumsum(new)])  # (row 0 is in no sequence, nor is the last)
    q = g.standard_normal((cu[-1] + 1, Hq * d))
    o, lse = oracle.paged_prefill(q, tokens, lengths, cu, H=Hq, Hkv=Hk, scale=0.3, **kw)
    assert np.isnan(o[[0, -1]]).all() and np.isnan(lse[:, [0, -1]]).all() and np.isfinite(o[1:-1]).all()
    for b in (0, 1, 3):
        r = slice(cu[b], cu[b + 1])
        ro, rl = oracle.fwd(q[None, r], tokens[b][0][None], tokens[b][1][None], H=Hq, Hkv=Hk, scale=0.3,
                            q_offset=lengths[b] - new[b], **dict(dict(causal=True), **kw))
        np.testing.assert_allclose(o[r], ro[0], atol=1e-13)
        np.testing.assert_allclose(lse[:, r], rl[0], atol=1e-13)


def test_oracle_is_the_decode_where_each_sequence_has_as_many_rows():
    g = np.random.default_rng(4)
    Hq, Hk, d, n = 6, 2, 8, 3
    lengths = [9, 2, 0]  # (rows at positions -1, 0, 1 of the second, none visible to any of the third)
    tokens = tokens_of(g, lengths, Hk * d)
    tokens[0][0][4] = np.nan  # a token in a page that does not exist
    q = g.standard_normal((3, n, Hq * d))
    for kw in (dict(), dict(window=3, softcap=1.5), dict(causal=False, window=2), dict(absolute=True)):
        o, lse = oracle.paged_prefill(q.reshape(9, -1), tokens, lengths, [0, 3, 6, 9], H=Hq, Hkv=Hk, scale=0.4, **kw)
        ro, rl = oracle.paged_decode(q, tokens, lengths, H=Hq, Hkv=Hk, scale=0.4, **kw)
        np.testing.assert_allclose(o.reshape(3, n, -1), ro, atol=1e-13)
        np.testing.assert_allclose(lse.reshape(Hq, 3, n).transpose(1, 0, 2), rl, atol=1e-13)
    assert np.isneginf(lse[:, 6:]).all() and (o[6:] == 0).all()
