"""Attention of chunks of new tokens over paged caches on the GPU against the fp64 oracle, and runs of it
with the rotation and the writer as a serving program makes them.  Every call goes through the C ABI.

Tolerances as for decode (test_paged_gpu.py): u(t) half a step of type t relative to the value; P is rounded to
16 bits before P V (the rows' type over 16-bit pages, fp16 over 8-bit ones): u(P) sum p|v| / l; fp16 p below 2^-14 by
2^-25 a key, where the largest p of a row is 2^-2 at least: 2^-23 a key relative to l; a score error ds changes
every p by a factor of at most 1 + 2 ds; O is rounded once.  ds: fp32 sums of hd products and the hardware
exponential, at most 2^-18 of the largest |scale q.k| sum of magnitudes, and 2^-19 of the softcap.  A value of an
8-bit page enters as an fp16 number whose scale (relative to a power of two) and product are rounded, 2 u(fp16),
where the scale is no power of two; below 2^-14 by 2^-25 of that power, at most 2^8 times a scale.
"""
import itertools
import math

import numpy as np
import pytest
import torch

import oracle
import attention_attn_fwd_08_gb300 as A
from test_paged_gpu import DEV, NAN, T, TINY, U, Cache, bits, expect_flag, f64, i32, is8, status_ok

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2"), ("f16", "e5m2")]


def check(c, q, lengths, cu, o, lse, tokens=None, rows=None, **flags):
    H, hd = q.shape[1] // c.hd, c.hd
    kw = dict(H=H, Hkv=c.Hkv, scale=1.0 / math.sqrt(hd))
    kw.update(flags)
    tok = c.tokens(lengths) if tokens is None else tokens
    ro, rl = oracle.paged_prefill(f64(q), tok, lengths, cu, **kw)
    ra, _ = oracle.paged_prefill(f64(q), tok, lengths, cu, absolute=True, **kw)
    og, lg = f64(o), f64(lse)
    for b, n in enumerate(lengths):
        r = np.arange(cu[b], cu[b + 1])
        r = r if rows is None else np.intersect1d(r, rows)
        if len(r) == 0:
            continue
        k, v = (np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in tok[b])
        qa = np.abs(f64(q)[r]).reshape(len(r), H, hd)
        smax = kw["scale"] * qa.max() * np.abs(k).reshape(n, c.Hkv, hd).sum(2).max(initial=0.0)
        ds = 2.0 ** -18 * smax + 2.0 ** -19 * kw.get("softcap", 0.0)
        up = 3 * U["f16"] if is8(c.kind) else U[c.dt]
        flush = n * 2.0 ** -23 * np.abs(v).max(initial=0.0) if is8(c.kind) or c.dt == "f16" else 0.0
        if is8(c.kind):
            vs = f64(c.vs)
            flush += 2.0 ** -25 * 2.0 ** 8 * np.abs(vs[np.isfinite(vs)]).max(initial=0.0)
        tol = U[c.dt] * np.abs(ro[r]) + (up + 2 * ds + 2.0 ** -16) * 1.02 * ra[r] + flush + TINY[c.dt]
        assert np.isfinite(og[r]).all(), "sequence %d: not finite" % b
        bad = np.abs(og[r] - ro[r]) > tol
        assert not bad.any(), "sequence %d, %d rows of %d tokens: O off by %.3g where %.3g is allowed, first at row %d" % (
            b, len(r), n, np.abs(og[r] - ro[r])[bad].max(), tol[bad].min(), np.argwhere(bad)[0][0])
        inf = np.isneginf(rl[:, r])
        assert (np.isneginf(lg[:, r]) == inf).all()
        assert (np.abs(lg[:, r][~inf] - rl[:, r][~inf]) <= ds + 2.0 ** -17 + 2.0 ** -20 * np.abs(rl[:, r][~inf])).all()


def queries(rows, width, dt, seed, stride=None):
    x = torch.randn((rows, width), generator=torch.Generator().manual_seed(seed)).to(T[dt]).to(DEV)
    if stride is None:
        return x
    buf = torch.full((rows, stride), float("nan"), dtype=T[dt], device=DEV)
    buf[:, :width] = x
    return buf[:, :width]


def run(dt, kind, lengths, new, H, Hkv, hd, page, seed, pad=3, stride=None, **flags):
    """One call, checked in full; rows behind the last sequence keep what they held."""
    c = Cache(dt, kind, lengths, Hkv, hd, page, seed)
    c.fill(lengths, seed)
    cu = np.cumsum([0] + list(new))
    n = int(cu[-1])
    q = queries(n + pad, H * hd, dt, seed + 1, stride)
    o = torch.full((n + pad, H * hd), 7.0, dtype=T[dt], device=DEV)
    lse = torch.full((H, n + pad), 7.0, device=DEV)
    A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, o=o, lse=lse, **c.kw(), **flags)
    status_ok()
    check(c, q, lengths, cu, o, lse, **flags)
    assert (o[n:] == 7).all() and (lse[:, n:] == 7).all()
    return c, q, cu, o, lse


@pytest.mark.parametrize("dt,kind", TYPES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_types_and_heads(dt, kind, hd, page):
    run(dt, kind, [1, 5, 40, 200, 130, 7, 333, 0, 129], [1, 5, 33, 64, 130, 0, 90, 0, 129], 8, 2, hd, page, seed=hd + page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 1), (7, 1), (6, 2), (3, 3), (64, 1), (128, 1), (65, 1), (10, 2)])
def test_groups_and_pages(kind, page, H, Hkv):
    run("bf16", kind, [129, 300, 1, 17], [100, 20, 1, 17], H, Hkv, 64, page, seed=H * 31 + page)


@pytest.mark.parametrize("hd,H,Hkv", [(128, 5, 1), (256, 7, 1), (256, 2, 2), (128, 24, 3), (256, 128, 1)])
@pytest.mark.parametrize("dt,kind", [("f16", "f16"), ("f16", "e5m2"), ("bf16", "bf16")])
def test_wide_heads_and_groups(hd, H, Hkv, dt, kind):
    run(dt, kind, [131, 70, 400], [131, 3, 40], H, Hkv, hd, 32, seed=hd + H)


FLAGS = [dict(window=1), dict(window=17), dict(window=64), dict(window=100, softcap=5.0), dict(softcap=30.0), dict(causal=False),
         dict(causal=False, window=33), dict(scale=0.9), dict(causal=False, window=5, softcap=1.0), dict(window=129), dict(window=400)]


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 128), ("f16", "e5m2", 64), ("bf16", "e4m3", 256), ("f16", "f16", 256),
                                        ("bf16", "e4m3", 128)])
@pytest.mark.parametrize("flags", FLAGS)
def test_masks(dt, kind, hd, flags):
    run(dt, kind, [700, 5, 64, 266, 1, 300], [150, 5, 64, 60, 1, 300], 4, 2, hd, 16, seed=5, **flags)


@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 8, 640 + 60, 640 + 59, 639])
@pytest.mark.parametrize("causal", [False, True])
def test_widest_windows_and_rows_at_negative_positions(window, causal):
    """More rows than tokens: those at negative positions see nothing under the causal mask."""
    c, q, cu, o, lse = run("f16", "f16", [3, 7, 40, 640, 0], [8, 7, 25, 20, 3], 4, 2, 64, 16, seed=46, window=window, causal=causal)
    assert torch.isneginf(lse[:, 60:63]).all() and (o[60:63] == 0).all()
    if causal:
        assert (o[:5] == 0).all() and torch.isneginf(lse[:, :5]).all()


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 128), ("bf16", "e4m3", 128), ("f16", "e5m2", 256), ("f16", "f16", 64)])
def test_long_and_ragged(dt, kind, hd):
    run(dt, kind, [5000, 1, 0, 2047, 1500, 130], [300, 1, 0, 17, 700, 130], 8, 2, hd, 64, seed=8)


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 128), ("bf16", "e4m3", 128), ("f16", "e5m2", 256), ("f16", "f16", 256)])
@pytest.mark.parametrize("new", [1, 29, 130])
def test_few_rows_over_one_long_sequence(dt, kind, hd, new):
    """The keys split over many CTAs, and joined."""
    run(dt, kind, [12011], [new], 4, 1, hd, 16, seed=9 + new)


def test_wide_heads_bound_by_memory():
    """Many sequences of few rows at hd 256, whose tiles land late and out of their order, a few times over."""
    new = [37 - (23 * b) // 36 for b in range(37)]
    lengths = [1336 + (4907 * b) // 36 for b in range(37)]
    c, q, cu, o, lse = run("bf16", "bf16", lengths, new, 4, 2, 256, 16, seed=61)
    for _ in range(5):
        again, _ = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, **c.kw())
        status_ok()
        assert torch.equal(again[:int(cu[-1])], o[:int(cu[-1])])


def test_split_rows_that_see_nothing_in_some_parts():
    run("bf16", "bf16", [9000], [200], 2, 1, 128, 16, seed=19, window=2000)
    run("bf16", "e4m3", [9000], [400], 1, 1, 64, 16, seed=20, window=700)


@pytest.mark.parametrize("B", [300, 1500])
def test_many_short_sequences(B):
    new = [(b * 7) % 13 for b in range(B)]
    lengths = [m + (37 * b) % 61 if m else (b % 3) * 5 for b, m in enumerate(new)]
    run("bf16", "e4m3", lengths, new, 2, 1, 64, 16, seed=10)


def test_strided_queries_and_one_row():
    run("bf16", "bf16", [90, 260], [40, 33], 4, 2, 128, 16, seed=12, stride=4 * 128 + 2 * 2 * 128)
    run("bf16", "bf16", [90], [1], 4, 2, 128, 16, seed=13, pad=0)
    run("f16", "e4m3", [1], [1], 4, 2, 64, 16, seed=14, pad=0)


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 64), ("f16", "f16", 128), ("bf16", "e4m3", 128), ("bf16", "e5m2", 256),
                                        ("f16", "f16", 256), ("f16", "e5m2", 64)])
def test_what_a_row_does_not_see_has_no_effect(dt, kind, hd):
    """Keys and values that are not finite reach the rows that see them alone."""
    lengths, new = [330, 70, 500], [80, 70, 3]
    c = Cache(dt, kind, lengths, 2, hd, 16, seed=21)
    c.fill(lengths, 21)
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 4 * hd, dt, 4)
    kw = dict(H=4, window=50, **c.kw())
    tokens = c.tokens(lengths)
    bad = [NAN[kind], 0x7f] if is8(kind) else [float("nan"), float("inf")]
    wild = {0: [290, 329, 260], 1: [33, 69], 2: [497, 448]}
    for w, pool in enumerate((c.k, c.v)):
        raw = pool.view(torch.uint8) if is8(kind) else pool
        for b, ts in wild.items():
            for t in ts:
                raw[int(c.table[b, t // 16]), :, t % 16] = bad[w]
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), **kw)
    status_ok()
    clean = []
    for b in range(3):
        for i in range(new[b]):
            p = lengths[b] - new[b] + i
            hit = [t for t in wild[b] if p - 50 < t <= p]
            if hit:
                assert torch.isnan(o[cu[b] + i]).all(), (b, i)
            else:
                clean.append(cu[b] + i)
    assert len(clean) > 20
    check(c, q, lengths, cu, o, lse, tokens=tokens, rows=clean, window=50)


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 128), ("f16", "f16", 64), ("f16", "f16", 256), ("bf16", "e4m3", 128)])
def test_values_alone_that_are_not_finite(dt, kind, hd):
    """An infinite value: its column of the rows that see it is infinite, and nothing else."""
    lengths, new = [300], [200]
    c = Cache(dt, kind, lengths, 1, hd, 16, seed=22)
    c.fill(lengths, 22)
    if is8(kind):
        c.v.view(torch.uint8)[int(c.table[0, 250 // 16]), 0, 250 % 16, 5] = NAN[kind]
    else:
        c.v[int(c.table[0, 250 // 16]), 0, 250 % 16, 5] = float("inf")
    q = queries(200, 2 * hd, dt, 5)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32([0, 200]), H=2, **c.kw())
    status_ok()
    got = ~torch.isfinite(o.view(200, 2, hd))
    want = torch.zeros_like(got)
    want[150:, :, 5] = True
    assert (got == want).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "e4m3", 256), ("f16", "e5m2", 128)])
@pytest.mark.parametrize("softcap", [0.0, 60.0])
def test_scores_that_climb(dt, kind, hd, softcap):
    """Keys that grow along the sequence: the rows' references move again and again; and some that fall back."""
    lengths, new = [1900, 633], [300, 500]
    c = Cache(dt, kind, lengths, 2, hd, 16, seed=41)
    c.fill(lengths, 41, unequal=False)
    grow = [1.0, 1.0, 4.0, 4.0, 12.0, 30.0, 1.0, 50.0]
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            m = grow[j % len(grow)] if b else 1.0 + j / 3
            pg = int(c.table[b, j])
            if is8(kind):
                c.ks[pg] *= m
            else:
                c.k[pg] *= m
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 4 * hd, dt, 7)
    kw = dict(scale=0.5 / math.sqrt(hd), softcap=softcap)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, **c.kw(), **kw)
    status_ok()
    check(c, q, lengths, cu, o, lse, **kw)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 77])
def test_scores_that_climb_inside_a_tile(kind, hd, window):
    """Pages whose scales rise and fall, and change sign, from one to the next: references move in the middle of a tile, whose
    earlier weights are then scaled too (a power of two; weights below 2^-14 are rounded by 2^-25 twice, where l is 2^-1
    at least: 2^-23 a key relative to l as before)."""
    lengths, new = [700, 333, 90], [200, 333, 5]
    c = Cache("bf16", kind, lengths, 2, hd, 16, seed=47)
    c.fill(lengths, 47, unequal=False)
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            c.ks[int(c.table[b, j])] *= (0.25, 1.0, -3.0, 12.0, 0.0, 40.0, -2.0, 60.0, 5.0)[j % 9]
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 8 * hd, "bf16", 17)
    kw = dict(scale=0.5 / math.sqrt(hd), window=window)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=8, **c.kw(), **kw)
    status_ok()
    check(c, q, lengths, cu, o, lse, **kw)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("climb", [False, True])
def test_values_near_the_end_of_bf16(hd, climb):
    """Values whose weighted mean a bf16 holds easily, and whose sums leave fp32 once they are weighted by more than 1."""
    lengths, new = [300, 3000], [40, 70]
    c = Cache("bf16", "bf16", lengths, 2, hd, 16, seed=55)
    c.fill(lengths, 55, unequal=False)
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            pg, m = int(c.table[b, j]), min(16, n - 16 * j)
            c.v[pg, :, :m] = (c.v[pg, :, :m].float().abs().clamp(max=4) * 2.0 ** (117 if b == 0 else 113)).to(torch.bfloat16)
            if climb:
                c.k[pg, :, :m] *= 1.0 + j / 8
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 4 * hd, "bf16", 3)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, **c.kw())
    status_ok()
    check(c, q, lengths, cu, o, lse)


@pytest.mark.parametrize("dt,kind", [("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_scales_unlike_each_other(dt, kind, page):
    """Scales of zero, of either sign, and far apart."""
    lengths, new = [700, 260, 300], [100, 33, 300]
    c = Cache(dt, kind, lengths, 2, 128, page, seed=43)
    c.fill(lengths, 43)
    for b in range(3):
        for j in range((lengths[b] + page - 1) // page):
            pg = int(c.table[b, j])
            if b == 0 and j % 3 == 1:
                c.vs[pg] = 0.0
            if b == 0 and j % 3 == 2:
                c.ks[pg, 0], c.ks[pg, 1] = 0.0, -c.ks[pg, 1]
            if b == 1:
                c.vs[pg] *= 2.0 ** ((20 if dt == "bf16" else 6) - 12 * (j % 6))
            if b == 2:
                c.vs[pg, 0] *= -1.0
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 8 * 128, dt, 8)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=8, **c.kw())
    status_ok()
    check(c, q, lengths, cu, o, lse)


def test_sequences_that_share_pages():
    c = Cache("bf16", "e4m3", [200, 200, 200], 2, 64, 16, seed=44)
    c.fill([200, 200, 200], 44)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :5] = c.table[0, :5]
    c.table_d = i32(c.table)
    cu = [0, 30, 71, 74]
    q = queries(74, 4 * 64, "bf16", 9)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32([130, 200, 77]), i32(cu), H=4, **c.kw())
    status_ok()
    check(c, q, [130, 200, 77], cu, o, lse)


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 64), ("f16", "e4m3", 128), ("bf16", "e5m2", 256)])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_bad_pages_are_not_seen(dt, kind, hd, page):
    lengths, new = [900, 200, 90], [300, 20, 90]
    c = Cache(dt, kind, lengths, 2, hd, page, seed=6)
    c.fill(lengths, 6)
    for (b, j), bad in zip(((0, 1), (0, 3), (1, 0), (2, 0)), (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31)):
        if j * page < lengths[b]:
            c.table[b, j] = bad
    c.table_d = i32(c.table)
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 4 * hd, dt, 5)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, **c.kw())
    expect_flag()
    check(c, q, lengths, cu, o, lse)


def test_pages_before_every_window_are_not_read():
    lengths, new = [900, 400], [33, 20]
    c = Cache("bf16", "e4m3", lengths, 2, 64, 16, seed=16)
    c.fill(lengths, 16)
    tokens = c.tokens(lengths)
    c.table[0, :(900 - 33 - 99) // 16] = -1
    c.table[1, :(400 - 20 - 99) // 16] = 10 ** 9
    c.table_d = i32(c.table)
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), 4 * 64, "bf16", 5)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, window=100, **c.kw())
    status_ok()
    check(c, q, lengths, cu, o, lse, tokens=tokens, window=100)


def test_lengths_out_of_range():
    c = Cache("bf16", "bf16", [64, 64, 20], 2, 64, 16, seed=7)
    c.fill([64, 64, 20], 7)
    cu = [0, 20, 50, 57]
    q = queries(57, 4 * 64, "bf16", 6)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32([2 ** 31 - 1, 64, -2 ** 31]), i32(cu), H=4, **c.kw())
    expect_flag()  # past the table: read as the capacity
    check(c, q, [64, 64, 0], cu, o, lse)


@pytest.mark.parametrize("cu,whole", [([0, 40, 30, 60], [0, 2]), ([0, 20, 61, 60], [0]), ([-5, 20, 40, 60], [1, 2]),
                                      ([0, 20, 40, 2 ** 31 - 1], [0, 1]), ([10, 20, 40, 50], [0, 1, 2]),
                                      ([0, 60, 0, 60], [])])
def test_prefix_sums_out_of_range(cu, whole):
    """Sequences whose rows lie in the tensor are attended as ever; nothing outside it is touched."""
    lengths = [70, 64, 80]
    c = Cache("bf16", "bf16", lengths, 2, 64, 16, seed=17)
    c.fill(lengths, 17)
    q = queries(60, 4 * 64, "bf16", 6)
    o = torch.full((60, 4 * 64), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, o=o, **c.kw())
    if whole == [0, 1, 2]:
        status_ok()
        assert (o[:10] == 7).all() and (o[50:] == 7).all()
    else:
        expect_flag()
    tok = c.tokens(lengths)
    for b in whole:
        if cu == [0, 40, 30, 60] and b == 0:
            continue  # (its last rows are the third sequence's too)
        r = [cu[b], cu[b + 1]]
        check(c, q, [lengths[b]], r, o, lse, tokens=[tok[b]], rows=np.arange(40, 60) if cu == [0, 40, 30, 60] else None)


def test_without_a_cache():
    q = torch.ones((5, 4 * 64), dtype=torch.bfloat16, device=DEV)
    for P, most in ((0, 3), (3, 0)):
        pool = torch.zeros((P, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
        o = torch.full_like(q, 7.0)
        o, lse = A.attn_paged_prefill(q, pool, pool, torch.zeros((2, most), dtype=torch.int32, device=DEV), i32([5, 5]), i32([0, 1, 4]),
                                      H=4, Hkv=2, o=o)
        status_ok()
        assert (o[:4] == 0).all() and torch.isneginf(lse[:, :4]).all() and (o[4] == 7).all()


def test_nothing_to_do():
    c = Cache("bf16", "bf16", [20], 2, 64, 16, seed=1)
    o, lse = A.attn_paged_prefill(queries(0, 256, "bf16", 1), c.k, c.v, c.table_d, i32([20]), i32([0, 0]), H=4, **c.kw())
    assert o.shape == (0, 256) and lse.shape == (4, 0)
    o, lse = A.attn_paged_prefill(queries(4, 256, "bf16", 1), c.k, c.v, c.table_d[:0], i32([]), i32([0]), H=4, **c.kw())
    out = torch.full_like(o, 7.0)
    A.attn_paged_prefill(queries(4, 256, "bf16", 1), c.k, c.v, c.table_d, i32([20]), i32([0, 0]), H=4, o=out, **c.kw())
    status_ok()
    assert (out == 7).all()


def test_twice_is_the_same_bits_and_leaves_its_inputs():
    lengths, new = [2700, 31, 640], [70, 31, 500]
    c, q, cu, o, lse = run("bf16", "e4m3", lengths, new, 8, 2, 128, 32, seed=12, pad=0)
    before = bits(c.k).copy(), bits(c.v).copy()
    ws = torch.full((A.attn_paged_prefill_workspace_size(len(q), 3, 8, 2, 128),), 0xff, dtype=torch.uint8, device=DEV)
    out = torch.full_like(o, 7.0)
    got, none = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=8, o=out, want_lse=False, workspace=ws, **c.kw())
    status_ok()
    assert got is out and none is None
    np.testing.assert_array_equal(bits(o), bits(out))
    np.testing.assert_array_equal(before[0], bits(c.k))
    np.testing.assert_array_equal(before[1], bits(c.v))


@pytest.mark.parametrize("dt,kind,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 128), ("f16", "f16", 256), ("bf16", "e4m3", 128)])
def test_workspaces_and_outputs_that_begin_anywhere(dt, kind, hd):
    """A workspace 16 bytes and more into a larger tensor, and an O at 16 modulo 32: the same bits, for a sequence whose items are cut
    and one whose item is not, and nothing outside is touched."""
    lengths, new, H = [5003, 40], [29, 40], 8
    c = Cache(dt, kind, lengths, 2, hd, 16, seed=52)
    c.fill(lengths, 52)
    cu, n = np.cumsum([0] + new), sum(new)
    q = queries(n, H * hd, dt, 53)
    args = (q, c.k, c.v, c.table_d, i32(lengths), i32(cu))
    size = A.attn_paged_prefill_workspace_size(n, 2, H, 2, hd)
    buf = torch.empty(size + 1024, dtype=torch.uint8, device=DEV)
    rows = torch.empty(n * H * hd + 64, dtype=T[dt], device=DEV)
    assert buf.data_ptr() % 256 == 0 and rows.data_ptr() % 256 == 0
    ref, lse = A.attn_paged_prefill(*args, H=H, workspace=buf[:size], **c.kw())
    status_ok()
    check(c, q, lengths, cu, ref, lse)
    for at, o_at in ((16, 0), (48, 8), (240, 8), (256, 24), (336, 0)):
        buf.fill_(0x5a)
        rows.fill_(7.0)
        o = rows[o_at:o_at + n * H * hd].view(n, H * hd)
        got, l2 = A.attn_paged_prefill(*args, H=H, workspace=buf[at:at + size], o=o, **c.kw())
        status_ok()
        assert torch.equal(got, ref) and torch.equal(l2, lse)
        assert (buf[:at] == 0x5a).all() and (buf[at + size:] == 0x5a).all()
        assert (rows[:o_at] == 7).all() and (rows[o_at + n * H * hd:] == 7).all()


def test_two_calls_at_once():
    calls = []
    for i, (lengths, new) in enumerate((([3000, 17, 900], [200, 17, 1]), ([64, 2100, 5], [64, 300, 2]))):
        c = Cache("bf16", "e4m3", lengths, 4, 128, 16, seed=46 + i)
        c.fill(lengths, 46 + i)
        cu = np.cumsum([0] + new)
        calls.append((c, queries(int(cu[-1]), 16 * 128, "bf16", i), lengths, cu, i32(lengths), i32(cu), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (c, q, lengths, cu, ld, cd, stream) in enumerate(calls):
            got[k].append(A.attn_paged_prefill(q, c.k, c.v, c.table_d, ld, cd, H=16, stream=stream, **c.kw()))
    status_ok()
    for k, (c, q, lengths, cu, ld, cd, stream) in enumerate(calls):
        check(c, q, lengths, cu, *got[k][0])
        for o, lse in got[k][1:]:
            np.testing.assert_array_equal(bits(o), bits(got[k][0][0]))


def test_calls_on_another_stream_and_by_handle():
    lengths, cu = [300, 77], [0, 100, 120]
    c = Cache("bf16", "e4m3", lengths, 2, 128, 32, seed=19)
    c.fill(lengths, 19)
    q, ld, cd = queries(120, 8 * 128, "bf16", 1), i32(lengths), i32(cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda._sleep(20000000)  # the current stream is busy; nothing waits for it
        o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, ld, cd, H=8, stream=handle, **c.kw())
        side.synchronize()
        check(c, q, lengths, cu, o, lse)
    torch.cuda.synchronize()
    status_ok()


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("dt,kind,layout,part", [("bf16", "bf16", "interleaved", 128), ("f16", "e4m3", "half", 64),
                                                 ("bf16", "e5m2", "interleaved", 32)])
def test_a_prompt_served_in_chunks(dt, kind, layout, part):
    """Each chunk's queries and keys turned in place in the projection's rows (any rotary form), stored, and attended
    over the pages; against attention on what went in, the cache's own rounding between, and against the pages."""
    H, Hkv, hd, page = 8, 2, 128, 16
    f = A.attn_rope_freqs(part, scaling="ramp", factor=4.0, original_length=64)
    upto = [[37, 64, 200], [38, 190, 200], [238, 191, 333], [239, 192, 334]]
    c = Cache(dt, kind, upto[-1], Hkv, hd, page, seed=30)
    g = torch.Generator().manual_seed(31)
    at, hist = [0, 0, 0], [([], []), ([], []), ([], [])]
    for lengths in upto:
        new = [u - a for u, a in zip(lengths, at)]
        cu = np.cumsum([0] + new)
        qkv = torch.randn((int(cu[-1]), (H + 2 * Hkv) * hd), generator=g).to(T[dt]).to(DEV)
        raw = f64(qkv)
        pos = np.concatenate([np.arange(a, u) for a, u in zip(at, lengths)])
        qk, q, k, v = qkv[:, :-Hkv * hd], qkv[:, :H * hd], qkv[:, H * hd:-Hkv * hd], qkv[:, -Hkv * hd:]
        A.attn_rope_ex(qk, f, H=H + Hkv, positions=i32(pos), layout=layout, rotary_start=hd - part, out=qk)
        A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, **c.kw())
        o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, **c.kw())
        status_ok()
        check(c, q, lengths, cu, o, lse)
        turned = oracle.turn_part(raw[:, :-Hkv * hd], pos, H=H + Hkv, inv_freq=f.inv_freq, start=hd - part,
                                  interleaved=layout == "interleaved", amplitude=f.amplitude)
        for b in range(3):
            hist[b][0].append(turned[cu[b]:cu[b + 1], H * hd:])
            hist[b][1].append(raw[cu[b]:cu[b + 1], -Hkv * hd:])
        tok = [tuple(np.concatenate(x) for x in h) for h in hist]
        ro, _ = oracle.paged_prefill(turned[:, :H * hd], tok, lengths, cu, H=H, Hkv=Hkv, scale=1 / math.sqrt(hd))
        assert np.linalg.norm(f64(o) - ro) <= 3 * U[kind] * np.linalg.norm(ro)
        at = lengths


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_row_each_is_the_decode(kind):
    lengths = [300, 1, 77, 4000]
    c, q, cu, o, lse = run("bf16", kind, lengths, [1] * 4, 8, 2, 128, 16, seed=50, pad=0)
    od, ld = A.attn_paged_decode(q.view(4, 1, -1), c.k, c.v, c.table_d, i32(lengths), H=8, **c.kw())
    status_ok()
    # (over 8-bit pages with other scales than powers of two the two read an element differently: half a step)
    assert (o.float() - od[:, 0].float()).abs().max() <= (2.0 ** -6 if kind == "bf16" else 2.0 ** -5) * od.float().abs().max()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_captured_chunk_is_replayed_as_the_cache_grows(kind):
    """One graph of rotation, append and attention; lengths, prefix sums, table, rows and pages change between replays."""
    B, H, Hkv, hd, page, rows = 3, 4, 2, 64, 16, 90
    full = [400, 133, 120]
    f = A.attn_rope_freqs(hd)
    c = Cache("bf16", kind, full, Hkv, hd, page, seed=17)
    c.fill([14, 31, 2], 17)
    qkv = torch.zeros((rows, (H + 2 * Hkv) * hd), dtype=torch.bfloat16, device=DEV)
    pos, lengths, cu, table = i32([0] * rows), i32([0] * B), i32([0] * (B + 1)), torch.full_like(c.table_d, -1)
    ws = torch.empty(A.attn_paged_prefill_workspace_size(rows, B, H, Hkv, hd), dtype=torch.uint8, device=DEV)
    o, lse = torch.full((rows, H * hd), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((H, rows), 7.0, device=DEV)
    turned = torch.empty((rows, (H + Hkv) * hd), dtype=torch.bfloat16, device=DEV)

    def step():
        A.attn_rope_ex(qkv[:, :-Hkv * hd], f, H=H + Hkv, positions=pos, out=turned)
        A.attn_paged_append(turned[:, H * hd:], qkv[:, -Hkv * hd:], c.k, c.v, table, lengths, cu, H=H, **c.kw())
        A.attn_paged_prefill(turned[:, :H * hd], c.k, c.v, table, lengths, cu, H=H, o=o, lse=lse, workspace=ws, **c.kw())

    step()  # an empty batch
    status_ok()
    assert (o == 7).all() and (lse == 7).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    table.copy_(c.table_d)
    at = [14, 31, 2]
    for i, new in enumerate(([1, 30, 3], [80, 1, 0], [0, 0, 90], [90, 0, 0], [7, 8, 9])):
        at = [a + n for a, n in zip(at, new)]
        s = np.cumsum([0] + new)
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(i)).to(qkv.dtype))
        p = np.concatenate([np.arange(a - n, a) for a, n in zip(at, new)] + [np.zeros(rows - s[-1], int)])
        lengths.copy_(i32(at)), cu.copy_(i32(s)), pos.copy_(i32(p)), o.fill_(7.0)
        graph.replay()
        status_ok()
        check(c, turned[:, :H * hd], at, s, o, lse)
        assert (o[s[-1]:] == 7).all()


def test_pages_past_four_gigabytes():
    """Offsets that pass 32 bits, in the pool of each type."""
    for dt, kind, hd in (("bf16", "e4m3", 128), ("f16", "f16", 64)):
        Hkv, page = 8, 64
        P = (2 ** 32 + 2 ** 26) // (Hkv * page * hd)
        es = 1 if is8(kind) else 2
        free, _ = torch.cuda.mem_get_info()
        if free < 2 * es * P * Hkv * page * hd + 2 ** 31:
            pytest.skip("not enough free memory")
        c = Cache(dt, kind, [100], Hkv, hd, page, seed=23, spare=0)
        c.k, c.v = (torch.zeros((P, Hkv, page, hd), dtype=torch.uint8 if is8(kind) else T[kind], device=DEV).view(T[kind])
                    for _ in range(2))
        if is8(kind):
            c.ks, c.vs = torch.ones((P, Hkv), device=DEV), torch.ones((P, Hkv), device=DEV)
        c.table[0] = [P - 1, P - 2]
        c.table_d = i32(c.table)
        x, y = queries(100, Hkv * hd, dt, 2), queries(100, Hkv * hd, dt, 3)
        A.attn_paged_append(x, y, c.k, c.v, c.table_d, i32([100]), i32([0, 100]), H=Hkv, **c.kw())
        ko, vo = A.attn_paged_gather(c.k, c.v, c.table_d, i32([0, 100]), 100, dtype=T[dt], **c.kw())
        q = queries(40, Hkv * hd, dt, 4)
        o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32([100]), i32([0, 40]), H=Hkv, **c.kw())
        status_ok()
        check(c, q, [100], [0, 40], o, lse, tokens=[(f64(ko), f64(vo))])
        del c
        torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_many_short_parts_behind_values_that_are_looked_over(kind, hd):
    """Chunks whose every tile is cut by the causal mask or has values that are not finite, so that looking V
    over lags behind the tiles that come after it: each call ends, and two give the same bits."""
    H, Hkv, page = 8, 2, 16
    dt = torch.bfloat16
    cd = torch.float8_e4m3fn if kind == "e4m3" else dt
    g = torch.Generator(device="cuda").manual_seed(hd)
    new = [1 + (37 * i) % 190 for i in range(40)]
    lengths = [n + (53 * i) % 300 for i, n in enumerate(new)]
    per = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(per), generator=torch.Generator().manual_seed(1)).int()
    table = torch.full((len(new), max(per)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    k = torch.randn((sum(per), Hkv, page, hd), device="cuda", generator=g).to(dt)
    v = torch.randn((sum(per), Hkv, page, hd), device="cuda", generator=g).to(dt)
    kw = dict(H=H, Hkv=Hkv, causal=True)
    if kind == "e4m3":
        kw.update(k_scale=torch.ones(sum(per), Hkv, device="cuda"), v_scale=torch.ones(sum(per), Hkv, device="cuda"))
    k, v = k.to(cd), v.to(cd)
    last = [int(table[b, n - 1]) for b, n in enumerate(per)]
    v8 = v.view(torch.uint8) if kind == "e4m3" else v
    for b, n in enumerate(lengths):  # the last key is seen by the last row alone
        v8[last[b], :, (n - 1) % page] = 0x7f if kind == "e4m3" else float("nan")
    q = torch.randn((sum(new), H * hd), device="cuda", generator=g).to(dt)
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device="cuda")
    args = (q, k, v, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), cu)
    first = A.attn_paged_prefill(*args, **kw)
    for _ in range(20):
        again = A.attn_paged_prefill(*args, **kw)
    assert A.attn_get_device_status()[0] == A.OK
    rows = torch.ones(sum(new), dtype=torch.bool)
    rows[(cu[1:] - 1).cpu().long()] = False
    assert torch.isfinite(first[0][rows.cuda()].float()).all() and torch.isnan(first[0][~rows.cuda()].float()).all()
    assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])


SOFT = [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "bf16", 256), ("bf16", "e4m3", 128), ("f16", "e5m2", 256)]


def same_rows(got, ref, rows):
    return torch.equal(got[0][rows], ref[0][rows]) and torch.equal(got[1][:, rows], ref[1][:, rows])


@pytest.mark.parametrize("dt,kind,hd", SOFT)
@pytest.mark.parametrize("window", [0, 90])
def test_softcapped_rows_take_nothing_from_what_they_do_not_see(dt, kind, hd, window):
    """The same bits whatever finite keys and values lie behind the sequences, whatever keys lie ahead of a row or before
    its window, and whatever the query rows beside it hold; and rows of scores unlike each other side by side."""
    lengths, new, H = [330, 70, 500], [80, 70, 33], 7
    c = Cache(dt, kind, lengths, 1, hd, 16, seed=71)
    c.fill(lengths, 71)
    # every byte 0x7b: 6.1e4, 1.3e36, 352 or 5.7e4
    unused = torch.ones(c.k.shape[0], 16, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            unused[int(c.table[b, j]), :min(16, n - 16 * j)] = False

    def put(pool, where, byte):
        raw = pool.view(torch.uint8) if is8(kind) else pool.view(torch.int16)
        raw.masked_fill_(where[:, None, :, None], byte if is8(kind) else byte * 257)

    put(c.k, unused, 0), put(c.v, unused, 0)
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]) + 9, H * hd, dt, 72)
    flags = dict(softcap=50.0, window=window)

    def call(q=q, k=c.k, v=c.v):
        out = A.attn_paged_prefill(q, k, v, c.table_d, i32(lengths), i32(cu), H=H, **c.kw(), **flags)
        status_ok()
        return out

    ref, every = call(), np.arange(cu[-1])
    check(c, q, lengths, cu, *ref, **flags)
    k, v = c.k.clone(), c.v.clone()
    put(k, unused, 0x7b), put(v, unused, 0x7b)
    assert same_rows(call(k=k, v=v), ref, every)
    # rows behind the sequences, a whole sequence's, and a few amid one's
    loud = q.clone()
    other = np.concatenate([np.arange(cu[1], cu[2]), [5, 17, 18, 40, 64], np.arange(cu[3], len(q))])
    loud[other] *= 64
    got = call(q=loud)
    assert same_rows(got, ref, np.setdiff1d(every, other))
    check(c, loud, lengths, cu, *got, **flags)
    # keys that the rows behind the first 33 alone see, or (in a window) those before them alone
    for b in (0, 2):
        at = lengths[b] - new[b] + 33 - (2 if b else 0)
        for before in (False, True):
            if before and not window:
                continue
            t = np.arange(0, at - window + 1) if before else np.arange(at, lengths[b])
            where = torch.zeros_like(unused)
            where[c.table[b, t // 16], t % 16] = True
            k = c.k.clone()
            put(k, where, 0x57)  # 117, 2.4e14, 120 or 120
            i = at - (lengths[b] - new[b])
            rows = np.arange(cu[b] + i, cu[b + 1]) if before else np.arange(cu[b], cu[b] + i)
            assert len(rows) and same_rows(call(k=k), ref, rows)


def test_softcapped_calls_repeat_their_bits_after_others():
    """Groups of 7 heads leave rows of the tensor cores' tile unused: what other calls left in their place changes nothing."""
    lengths, new = [700, 129], [150, 129]
    cu = np.cumsum([0] + new)
    calls = []
    for dt, kind, hd in SOFT:
        c = Cache(dt, kind, lengths, 1, hd, 16, seed=73)
        c.fill(lengths, 73)
        for H, factor in ((7, 1.0), (8, 100.0)):
            calls.append((c, queries(int(cu[-1]), H * hd, dt, 74) * factor, H))

    def call(c, q, H):
        out = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, softcap=50.0, **c.kw())
        status_ok()
        return out

    quiet, loud = calls[0::2], calls[1::2]
    ref = [call(*x) for x in quiet]
    for x in loud:
        call(*x)
        for y, r in zip(quiet, ref):
            assert same_rows(call(*y), r, np.arange(cu[-1]))
            call(*x)


@pytest.mark.parametrize("dt,kind,hd", SOFT)
@pytest.mark.parametrize("softcap", [1e-7, 1e-3])
def test_scores_of_zero_under_a_small_softcap(dt, kind, hd, softcap):
    """Keys of zeros, some and a sequence's all, and a query row of zeros, under a softcap so small that the scores' ratio to it has
    an eighth power which fp32 does not hold."""
    lengths, new, H = [330, 70], [80, 70], 4
    c = Cache(dt, kind, lengths, 2, hd, 16, seed=75)
    c.fill(lengths, 75)
    raw = c.k.view(torch.uint8) if is8(kind) else c.k
    for b, ts in ((0, range(20, 290, 3)), (1, range(70))):
        for t in ts:
            raw[int(c.table[b, t // 16]), :, t % 16] = 0
    cu = np.cumsum([0] + new)
    q = queries(int(cu[-1]), H * hd, dt, 76)
    q[11] = 0
    o, lse = A.attn_paged_prefill(q, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, softcap=softcap, **c.kw())
    status_ok()
    check(c, q, lengths, cu, o, lse, softcap=softcap)


@pytest.mark.parametrize("dt,kind,hd", SOFT)
@pytest.mark.parametrize("scale,softcap", [(1e-6, 0.1), (1e-4, 30.0), (1e-9, 1e-3)])
def test_small_scales_under_a_softcap(dt, kind, hd, scale, softcap):
    """The fit's highest coefficient is near or below fp32's smallest number: keys that are not seen stay unseen."""
    lengths, new = [330, 70], [80, 70]
    run(dt, kind, lengths, new, 4, 2, hd, 16, seed=78, scale=scale, softcap=softcap)
    run(dt, kind, lengths, new, 4, 2, hd, 16, seed=79, scale=scale, softcap=softcap, window=40)
