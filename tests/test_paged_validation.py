"""Refusals of the paged-cache calls, by the C ABI before any launch and by the binding
before any pointer reaches the library.  Runs without a GPU."""
import ctypes

import pytest
import torch

import attention_attn_fwd_08_gb300 as A

BAD = ctypes.c_void_p(0x1000)  # never dereferenced: every case fails validation first
ODD = ctypes.c_void_p(0x1002)


def append(**kw):
    a = dict(dt=2, cache=3, k=BAD, ks=512, v=BAD, vs=512, q=None, qs=0, q_out=None, kc=BAD, vc=BAD, ksc=BAD, vsc=BAD, cu=BAD,
             lengths=BAD, table=BAD, batch=2, total=8, num_pages=10, page=16, max_pages=4, H=8, Hkv=4, hd=128, theta=1e4,
             stream=None)
    a.update(kw)
    return A.lib().attn_paged_append(*a.values())


def decode(**kw):
    a = dict(dt=2, cache=3, q=BAD, kc=BAD, vc=BAD, ksc=BAD, vsc=BAD, o=BAD, lse=None, ws=BAD, wsb=1 << 30, lengths=BAD, table=BAD,
             B=2, Lq=1, num_pages=10, page=16, max_pages=4, H=8, Hkv=4, hd=128, scale=0.1, causal=1, window=0, softcap=0.0,
             stream=None)
    a.update(kw)
    return A.lib().attn_paged_decode(*a.values())


def gather(**kw):
    a = dict(dt=2, cache=3, kc=BAD, vc=BAD, ksc=BAD, vsc=BAD, ko=BAD, vo=BAD, cu=BAD, table=BAD, batch=2, total=8, num_pages=10,
             page=16, max_pages=4, Hkv=4, hd=128, stream=None)
    a.update(kw)
    return A.lib().attn_paged_gather(*a.values())


SHARED = [
    (dict(dt=7), A.ERR_INVALID_ARG), (dict(dt=3), A.ERR_INVALID_ARG), (dict(cache=5), A.ERR_INVALID_ARG),
    (dict(cache=-1), A.ERR_INVALID_ARG),
    (dict(dt=0), A.ERR_UNSUPPORTED), (dict(cache=0), A.ERR_UNSUPPORTED),
    (dict(cache=1), A.ERR_INVALID_ARG),                     # a 16-bit cache of the other type
    (dict(num_pages=-1), A.ERR_INVALID_ARG), (dict(max_pages=-1), A.ERR_INVALID_ARG),
    (dict(page=8), A.ERR_UNSUPPORTED), (dict(page=48), A.ERR_UNSUPPORTED), (dict(page=512), A.ERR_UNSUPPORTED),
    (dict(page=0), A.ERR_UNSUPPORTED),
    (dict(hd=96), A.ERR_UNSUPPORTED), (dict(hd=32), A.ERR_UNSUPPORTED),
    (dict(num_pages=1 << 26), A.ERR_UNSUPPORTED),           # more than 2^31 rows of one head
    (dict(max_pages=1 << 27), A.ERR_UNSUPPORTED),
    (dict(kc=None), A.ERR_INVALID_ARG), (dict(vc=ODD), A.ERR_INVALID_ARG),
    (dict(ksc=None), A.ERR_INVALID_ARG), (dict(vsc=ODD), A.ERR_INVALID_ARG),
    (dict(table=None), A.ERR_INVALID_ARG), (dict(table=ODD), A.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("call", [append, decode, gather])
@pytest.mark.parametrize("kw,expect", SHARED)
def test_shared_rules(call, kw, expect):
    assert call(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(batch=-1), A.ERR_INVALID_ARG), (dict(batch=65536), A.ERR_INVALID_ARG), (dict(total=-1), A.ERR_INVALID_ARG),
    (dict(H=6), A.ERR_INVALID_ARG), (dict(Hkv=0), A.ERR_INVALID_ARG),
    (dict(ks=504), A.ERR_INVALID_ARG), (dict(vs=516), A.ERR_INVALID_ARG), (dict(k=None), A.ERR_INVALID_ARG),
    (dict(v=ctypes.c_void_p(0x1008)), A.ERR_INVALID_ARG),
    (dict(q=BAD, qs=1024), A.ERR_INVALID_ARG),              # no q_out
    (dict(q_out=BAD), A.ERR_INVALID_ARG),                   # no q
    (dict(q=BAD, qs=1016, q_out=ctypes.c_void_p(0x2000)), A.ERR_INVALID_ARG),
    (dict(q=BAD, qs=2048, q_out=BAD), A.ERR_INVALID_ARG),   # in place, but strided
    (dict(cu=None), A.ERR_INVALID_ARG), (dict(cu=ODD), A.ERR_INVALID_ARG), (dict(lengths=ODD), A.ERR_INVALID_ARG),
    (dict(theta=-1.0), A.ERR_INVALID_ARG), (dict(theta=float("nan")), A.ERR_INVALID_ARG),
    (dict(theta=float("inf")), A.ERR_INVALID_ARG),
    (dict(batch=0, table=None, kc=None), A.OK), (dict(total=0), A.OK),
])
def test_append_rules(kw, expect):
    assert append(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), A.ERR_INVALID_ARG), (dict(Lq=-1), A.ERR_INVALID_ARG), (dict(H=6), A.ERR_INVALID_ARG),
    (dict(Lq=17), A.ERR_UNSUPPORTED), (dict(H=64, Hkv=4, Lq=5), A.ERR_UNSUPPORTED),
    (dict(scale=0.0), A.ERR_INVALID_ARG), (dict(softcap=-1.0), A.ERR_INVALID_ARG), (dict(window=-1), A.ERR_INVALID_ARG),
    (dict(causal=2), A.ERR_INVALID_ARG), (dict(q=None), A.ERR_INVALID_ARG), (dict(o=ODD), A.ERR_INVALID_ARG),
    (dict(lse=ODD), A.ERR_INVALID_ARG), (dict(lengths=None), A.ERR_INVALID_ARG), (dict(ws=None), A.ERR_INVALID_ARG),
    (dict(ws=ctypes.c_void_p(0x1008)), A.ERR_INVALID_ARG), (dict(wsb=8), A.ERR_INVALID_ARG),
    (dict(B=0, table=None), A.OK), (dict(Lq=0), A.OK),
])
def test_decode_rules(kw, expect):
    assert decode(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(batch=-1), A.ERR_INVALID_ARG), (dict(total=-1), A.ERR_INVALID_ARG), (dict(ko=None), A.ERR_INVALID_ARG),
    (dict(vo=ODD), A.ERR_INVALID_ARG), (dict(cu=None), A.ERR_INVALID_ARG), (dict(Hkv=0), A.ERR_INVALID_ARG),
    (dict(batch=0, table=None), A.OK), (dict(total=0), A.OK),
])
def test_gather_rules(kw, expect):
    assert gather(**kw) == expect


def test_workspace_size():
    f = A.attn_paged_decode_workspace_size
    assert f(4, 2, 32, 8, 128) > 0
    for bad in ((0, 1, 8, 4, 64), (1, 0, 8, 4, 64), (1, 17, 8, 8, 64), (1, 1, 8, 3, 64), (1, 1, 8, 4, 96), (1, 9, 64, 8, 64),
                (1, 1, 1 << 30, 1, 64)):
        assert f(*bad) == 0


# ------------------------------------------------------------------ the binding
B, Hkv, H, hd, page, P, most = 3, 2, 4, 64, 16, 9, 4


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache(dtype=torch.bfloat16):
    c = dict(k_cache=torch.zeros((P, Hkv, page, hd), dtype=dtype), v_cache=torch.zeros((P, Hkv, page, hd), dtype=dtype),
             page_table=i32(B, most))
    if dtype.itemsize == 1:
        c.update(k_scale=torch.ones(P, Hkv), v_scale=torch.ones(P, Hkv))
    return c


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def call_append(c, **kw):
    a = dict(k=bf(5, Hkv * hd), v=bf(5, Hkv * hd), lengths=i32(B), cu_new=i32(B + 1), H=H, Hkv=Hkv)
    a.update(c)
    a.update(kw)
    return A.attn_paged_append(**a)


def call_decode(c, **kw):
    a = dict(q=bf(B, 2, H * hd), lengths=i32(B), H=H, Hkv=Hkv)
    a.update(c)
    a.update(kw)
    return A.attn_paged_decode(**a)


def call_gather(c, **kw):
    a = dict(cu_seqlens=i32(B + 1), total=5, Hkv=Hkv, dtype=torch.bfloat16)
    a.update(c)
    a.update(kw)
    return A.attn_paged_gather(**a)


@pytest.mark.parametrize("call", [call_append, call_decode, call_gather])
def test_binding_refuses_wrong_caches(call):
    c = cache()
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(c)
    with pytest.raises(ValueError, match="k_cache"):
        call(dict(c, k_cache=c["k_cache"][0]))
    with pytest.raises(ValueError, match="k_cache"):
        call(c, Hkv=4)
    with pytest.raises(ValueError, match="v_cache"):
        call(dict(c, v_cache=c["v_cache"][:5]))
    with pytest.raises(ValueError, match="v_cache"):
        call(dict(c, v_cache=c["v_cache"].half()))
    with pytest.raises(TypeError, match="cache dtype"):
        call(dict(c, k_cache=c["k_cache"].float()))
    with pytest.raises(ValueError, match="rows' dtype"):
        call(cache(torch.float16))
    with pytest.raises(ValueError, match="page_table"):
        call(dict(c, page_table=c["page_table"].long()))
    with pytest.raises(ValueError, match="page_table"):
        call(dict(c, page_table=c["page_table"][0]))
    with pytest.raises(ValueError, match="contiguous"):
        call(dict(c, page_table=i32(most, B).t()))
    e = cache(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(e)
    with pytest.raises(ValueError, match="k_scale"):
        call(dict(e, k_scale=None))
    with pytest.raises(ValueError, match="v_scale"):
        call(dict(e, v_scale=torch.ones(P, 1)))
    with pytest.raises(ValueError, match="v_scale"):
        call(dict(e, v_scale=torch.ones(P, Hkv, dtype=torch.float64)))


def test_binding_refuses_wrong_append_rows():
    c = cache()
    wide = bf(5, 4 * Hkv * hd)
    with pytest.raises(ValueError, match="CUDA tensors"):
        call_append(c, k=wide[:, :Hkv * hd], v=wide[:, -Hkv * hd:])  # strided rows are fine
    for kw, what in ((dict(v=bf(4, Hkv * hd)), "v must"), (dict(v=bf(5, Hkv * hd).half()), "v must"),
                     (dict(k=bf(Hkv * hd, 5).t()), "k must"), (dict(k=bf(1, Hkv * hd).expand(5, -1)), "k must"),
                     (dict(cu_new=i32(B)), "cu_new"), (dict(lengths=i32(B).long()), "lengths"), (dict(q=bf(5, Hkv * hd)), "q must"),
                     (dict(q_out=bf(5, H * hd)), "q_out"), (dict(q=bf(5, H * hd), q_out=bf(4, H * hd)), "q_out"),
                     (dict(rope_theta=0.0), "rope_theta"), (dict(rope_theta=float("nan")), "rope_theta")):
        with pytest.raises(ValueError, match=what):
            _on_gpu_shapes(call_append, cache(), **kw)
    with pytest.raises(TypeError, match="rows of a paged cache"):
        call_append(cache(torch.float8_e5m2), k=torch.zeros(5, Hkv * hd), v=torch.zeros(5, Hkv * hd))


def _on_gpu_shapes(call, c, **kw):
    """The call as the binding would check it on a GPU: the cache check that asks for CUDA
    tensors comes first, so the rest is checked with that one rule answered."""
    real = A._pools

    def pools(k_cache, v_cache, k_scale, v_scale, page_table, n, dtype):
        num, _, size, d = k_cache.shape
        return 2, 2, num, size, d, page_table.shape[0], page_table.shape[1]

    A._pools = pools
    try:
        return call(c, **kw)
    finally:
        A._pools = real


@pytest.mark.parametrize("kw,what", [
    (dict(q=bf(B, 2, H * hd + 4)), "q must"), (dict(q=bf(B + 1, 2, H * hd)), "q must"), (dict(q=bf(B, H * hd)), "q must"),
    (dict(lengths=i32(B + 1)), "lengths"), (dict(o=bf(B, 1, H * hd)), "o must"), (dict(lse=torch.zeros(B, H, 3)), "lse"),
    (dict(q=bf(2, B, H * hd).transpose(0, 1)), "contiguous"),
])
def test_binding_refuses_wrong_decode_tensors(kw, what):
    with pytest.raises(ValueError, match=what):
        _on_gpu_shapes(call_decode, cache(), **kw)


@pytest.mark.parametrize("kw,what", [
    (dict(cu_seqlens=i32(B)), "cu_seqlens"), (dict(k_out=bf(4, Hkv * hd)), "k_out"),
    (dict(v_out=bf(5, Hkv * hd).half()), "v_out"),
])
def test_binding_refuses_wrong_gather_tensors(kw, what):
    with pytest.raises(ValueError, match=what):
        _on_gpu_shapes(call_gather, cache(), **kw)


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        cuda_stream, device = 17, torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        A._on(torch.device("cuda", 0), Stream())


@pytest.mark.parametrize("theta", [2.0 ** -33, 1e-12, 1e-38, 1e-45])
def test_bases_below_the_least_are_refused(theta):
    assert append(theta=theta) == A.ERR_INVALID_ARG
    assert append(theta=2.0 ** -32, total=0) == A.OK
    assert append(theta=0.0, total=0) == A.OK


@pytest.mark.parametrize("theta", [1e-12, 1e-46, 5e-324, -0.0])
def test_binding_refuses_bases_that_fp32_would_lose(theta):
    """One below fp32's smallest would reach the library as 0, which means no turn."""
    with pytest.raises(ValueError, match="rope_theta"):
        _on_gpu_shapes(call_append, cache(), rope_theta=theta)
