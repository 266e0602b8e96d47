"""Edges of the paged cache on the GPU: block scales, far positions, rotation bases, arrays out of
range, against the fp64 oracle.  Tolerances as in test_paged_gpu.py."""
import decimal
import math

import numpy as np
import pytest
import torch

import oracle
import attention_attn_fwd_08_gb300 as A
from test_paged_gpu import DEV, Cache, check_decode, close, expect_flag, f64, i32, is8, near_steps, run_step, status_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,hd,page", [("e4m3", 64, 16), ("e5m2", 128, 64), ("e4m3", 256, 32), ("e5m2", 256, 16), ("e4m3", 128, 256)])
def test_single_tokens_grow_blocks_of_many_heads(kind, hd, page):
    """A token to each sequence, a warp to each block: it reads the scale that it then replaces."""
    c = Cache("bf16", kind, [9 + b % 5 for b in range(24)], 5, hd, page, seed=51)
    at = [b % 5 for b in range(24)]
    c.fill(at, 51)
    for step, spread in enumerate((1e-3, 300.0, 1e-2, 3e4, 1.0)):
        run_step(c, at, [1] * 24, spread, seed=60 + step, theta=None)
        at = [a + 1 for a in at]


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [9, 30, 17, 40]])
def test_append_to_blocks_of_negative_scale(kind, new):
    """A block that another program began may have a scale of either sign: one that is large enough
    stays, with the codes of the rows that are there, and one that is not grows by its magnitude."""
    before = [5, 20, 7, 3]
    c = Cache("bf16", kind, [b + n for b, n in zip(before, new)], 2, 64, 16, seed=52)
    c.fill(before, 52)
    factor = [-64.0, -1024.0, -2.0 ** -8, 1.0]
    pages = [int(c.table[b, before[b] // 16]) for b in range(4)]
    for pg, m in zip(pages, factor):
        c.ks[pg] *= m
        c.vs[pg] *= m
    old = c.host()
    run_step(c, before, new, 1.0, seed=53, theta=None)
    got = c.host()
    for b in (0, 1):  # kept: the scale, and every code under it
        n = before[b] % 16
        for w in (0, 1):
            np.testing.assert_array_equal(got[2 + w][pages[b]], old[2 + w][pages[b]])
            np.testing.assert_array_equal(got[w][pages[b], :, :n], old[w][pages[b], :, :n])
    for w in (0, 1):  # grown: a power of two, the rows' values as they were
        new_scale = got[2 + w][pages[2]]
        assert (new_scale > np.abs(old[2 + w][pages[2]])).all() and (np.log2(new_scale) % 1 == 0).all()
        v = oracle.f8_values(kind)
        before_v = v[old[w][pages[2], :, :7]] * old[2 + w][pages[2]][:, None, None]
        after_v = v[got[w][pages[2], :, :7]] * new_scale[:, None, None]
        u, tiny = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[kind]
        assert (np.abs(after_v - before_v) <= np.maximum(u * np.abs(before_v), tiny * new_scale[:, None, None])).all()


def turned(x, pos, hd, theta):
    """A row's head vectors turned at one position, the angles from 120 digits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 120
        pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
        base = decimal.Decimal(float(np.float32(theta)))
        turns = [pos * base ** (decimal.Decimal(-2 * i) / hd) / (2 * pi) for i in range(hd // 2)]
        ang = 2 * math.pi * np.array([float(t - t.to_integral_value(decimal.ROUND_FLOOR)) for t in turns])
    y = x.reshape(-1, 2, hd // 2)
    c, s = np.cos(ang), np.sin(ang)
    return np.stack([y[:, 0] * c - y[:, 1] * s, y[:, 1] * c + y[:, 0] * s], 1).reshape(x.shape)


@pytest.mark.parametrize("theta", [2.0 ** -32, 1e-8, 1e-4, 0.3, 1.0, 10000.0, 5e6, 1e30])
@pytest.mark.parametrize("far", [3, 1000003])
@pytest.mark.parametrize("hd", [64, 256])
def test_append_angles_of_every_base(theta, far, hd):
    """Bases from 2^-32 on, those below 1 that turn many times a position among them."""
    page = 256
    c = Cache("f16", "f16", [3], 2, hd, page, seed=1, most=far // page + 2)
    c.table[0, far // page] = 0
    c.table_d = i32(c.table)
    k = torch.randn((1, 2 * hd), generator=torch.Generator().manual_seed(8)).half().to(DEV)
    q_out = A.attn_paged_append(k, k, c.k, c.v, c.table_d, i32([far + 1]), i32([0, 1]), H=2, q=k, rope_theta=theta, **c.kw())
    status_ok()
    x = turned(f64(k)[0], far, hd, theta).reshape(2, hd)
    close(f64(q_out).reshape(2, hd), x, "f16")
    close(f64(c.k[0, :, far % page]), x, "f16")


@pytest.mark.parametrize("causal", [False, True])
def test_decode_windows_past_32_bits(causal):
    """A window that no 32-bit integer holds leaves out nothing; a negative one is refused."""
    lengths = [200, 31]
    c = Cache("f16", "f16", lengths, 2, 64, 16, seed=54)
    c.fill(lengths, 54)
    q = torch.randn((2, 3, 4 * 64), generator=torch.Generator().manual_seed(3)).half().to(DEV)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40 + 7):
        o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=4, window=window, causal=causal, **c.kw())
        status_ok()
        check_decode(c, q, lengths, o, lse, causal=causal)
    for window in (-1, -2 ** 32 + 5, -2 ** 32):
        with pytest.raises(A.AttnError):
            A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=4, window=window, causal=causal, **c.kw())


@pytest.mark.parametrize("hd,G,Lq", [(128, 4, 1), (64, 2, 3), (256, 2, 2), (128, 4, 16)])
@pytest.mark.parametrize("climb", [False, True])
def test_decode_values_near_the_end_of_bf16(hd, G, Lq, climb):
    """Values whose weighted mean a bf16 holds easily, and whose sums leave fp32 once they are weighted by more than 1."""
    lengths = [300, 3000]
    c = Cache("bf16", "bf16", lengths, 2, hd, 16, seed=55)
    c.fill(lengths, 55, unequal=False)
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            pg = int(c.table[b, j])
            m = min(16, n - 16 * j)
            c.v[pg, :, :m] = (c.v[pg, :, :m].float().abs().clamp(max=4) * 2.0 ** (117 if b == 0 else 113)).to(torch.bfloat16)
            if climb:
                c.k[pg, :, :m] *= 1.0 + j / 8
    q = torch.randn((2, Lq, 2 * G * hd), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=2 * G, **c.kw())
    status_ok()
    check_decode(c, q, lengths, o, lse)


BAD_ARRAYS = [
    ([(0, 0, -1), (1, 0, 99), (2, 1, 2 ** 31 - 1), (3, 0, -2 ** 31)], [40, 20, 17, 16]),
    ([(0, 1, 10 ** 9)], [40, 20, 17, 16]),
    ([], [80, 20, 17, 16]),                       # the first sequence's last rows lie past its table
    ([], [40, 2 ** 31 - 1, 17, -2 ** 31]),
    ([(2, 0, -5)], [40, 60, 9, 16]),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("bad,lengths", BAD_ARRAYS)
@pytest.mark.parametrize("slots", [0, 60])
def test_append_stores_what_lies_in_range_and_nothing_else(kind, bad, lengths, slots):
    """Pages and positions out of range among good ones: pools, scales and turned queries to the last
    byte, with few rows to a sequence (60 empty slots behind) and with many."""
    c = Cache("bf16", kind, [40, 20, 17, 16] + [0] * slots, 2, 64, 16, seed=11)
    for b, j, pg in bad:
        c.table[b, j] = pg
    c.table_d = i32(c.table)
    lengths = lengths + [0] * slots
    cu = [0, 40, 60, 77, 93] + [93] * slots
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((97, 128), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn((97, 256), generator=g).to(torch.bfloat16).to(DEV)
    q_out = torch.full((97, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    host = c.host()
    A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, q=q, q_out=q_out, **c.kw())
    expect_flag()
    want = oracle.paged_append(f64(k), f64(v), *host, c.table, lengths, cu, Hkv=2, kind=kind if is8(kind) else None)
    for got, ref in zip(c.host(), want):
        if ref is not None:
            np.testing.assert_array_equal(got, ref)
    ref = np.full((97, 256), 9.0)
    stored = 0
    for b in range(4):
        for r in range(cu[b], cu[b + 1]):
            pos = lengths[b] - (cu[b + 1] - r)
            if pos >= 0 and pos // 16 < c.most and 0 <= c.table[b, pos // 16] < c.k.shape[0]:
                ref[r] = f64(q[r])
                stored += 1
    assert 0 < stored < 93
    np.testing.assert_array_equal(f64(q_out), ref)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("hd,page,Hkv,new", [
    (128, 64, 2, [1] * 40),                                    # a warp to each block
    (64, 32, 2, [70, 33, 64]),                                 # 128 threads, whole pages and their ends
    (64, 64, 3, [64, 129]),                                    # 256
    (128, 64, 2, [200, 64]),                                   # 512
    (128, 64, 2, [1] * 60 + [100] + [1] * 30 + [41]),          # long blocks found by a row
    (256, 64, 4, [40 + b for b in range(50)]),                 # 1024
    (128, 128, 1, [300]),                                      # 1024 pieces by 512 threads, twice
    (256, 128, 2, [131, 128]),                                 # 2048 pieces
    (128, 256, 1, [256, 5])])
def test_append_far_positions_into_8_bit_pages(kind, hd, page, Hkv, new):
    """Keys turned at positions of hundreds of thousands, by every team that stores blocks."""
    theta, B = 10000.0, len(new)
    first = [500001 + 977 * b for b in range(B)]
    first[0] = 700000 // page * page  # (one at a page's beginning)
    lengths = [a + n for a, n in zip(first, new)]
    used = [range(a // page, (n - 1) // page + 1) for a, n in zip(first, lengths)]
    P = sum(len(u) for u in used) + 1
    c = Cache("bf16", kind, [1] * B, Hkv, hd, page, seed=56, spare=P - B, most=max(lengths) // page + 1)
    perm = np.random.default_rng(57).permutation(P)
    c.table[:] = -1
    at = 0
    g = torch.Generator().manual_seed(58)
    for b, u in enumerate(used):
        c.table[b, u.start:u.stop] = perm[at:at + len(u)]
        pg, m = int(perm[at]), first[b] % page
        at += len(u)
        if m:  # rows of the block that an earlier call stored
            for pool, sc in ((c.k, c.ks), (c.v, c.vs)):
                sc[pg] = 2.0 ** -9
                pool.view(torch.uint8)[pg, :, :m] = torch.randint(0, 0x70, (Hkv, m, hd), generator=g, dtype=torch.uint8).to(DEV)
    c.table_d = i32(c.table)
    cu = np.cumsum([0] + list(new))
    k, v = (torch.randn((int(cu[-1]), Hkv * hd), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    host = c.host()
    A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=Hkv, rope_theta=theta, **c.kw())
    status_ok()
    rk, rv, rks, rvs, exact = oracle.paged_append(f64(k), f64(v), *host, c.table, lengths, cu, Hkv=Hkv, kind=kind, theta=theta)
    gk, gv, gks, gvs = c.host()
    for got, ref in ((gv, rv), (gks, rks), (gvs, rvs)):
        np.testing.assert_array_equal(got, ref)
    fresh = np.zeros(rk.shape, bool)
    values, top = oracle.f8_values(kind), oracle.F8_TOP[kind]
    for w, pg, row, x in exact:
        if w == 0:
            fresh[pg, :, row] = True
            pair = np.hypot(x[:, :hd // 2], x[:, hd // 2:])
            slack = 2.0 ** -20 * np.concatenate([pair, pair], 1)
            off = np.abs(values[gk[pg, :, row]] - np.clip(x, -top, top))
            assert (off <= near_steps(np.abs(x) + slack, kind) + slack).all()
    np.testing.assert_array_equal(gk[~fresh], rk[~fresh])
