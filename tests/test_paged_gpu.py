"""The paged key/value cache on the GPU against the fp64 oracle: appending with the
rotation, decode over 16- and 8-bit pages, reading pages back, and runs of the three as a
serving program makes them.  Every call goes through the C ABI.

Tolerances.  u(t) is half a step of type t relative to the value (bf16 2^-8, fp16 2^-11,
e4m3 2^-4, e5m2 2^-3).
  stored rows without a turn: the oracle's codes exactly (one rounding of an exact quotient).
  turned rows: one rounding, u * |x| (at least half the type's smallest step), of a value
    whose sine and cosine are off by at most 2^-20 of the pair's length.
  decode: P is rounded to 16 bits before P V (fp16 over 8-bit pages, the rows' type over
    16-bit pages), so O is off by at most u(P) sum p|v| / l, and fp16 P below 2^-14 by 2^-25
    a key; a score error of ds changes every p by a factor of at most 1 + 2 ds; O is rounded
    once, u(O) |O|.  ds: fp32 sums of hd products and the hardware exponential, at most
    2^-18 of the largest |scale q.k| sum of magnitudes here, and 2^-19 of the softcap.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import attention_attn_fwd_08_gb300 as A

pytestmark = pytest.mark.gpu

T = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
NAN = {"e4m3": 0x7f, "e5m2": 0x7e}
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def is8(kind):
    return kind in NAN


def bits(t):
    return t.detach().cpu().view(torch.uint8 if t.element_size() == 1 else torch.int16).numpy()


def status_ok():
    torch.cuda.synchronize()
    st, word = A.attn_get_device_status()
    assert st == A.OK, "device status word %#x" % word


def expect_flag():
    torch.cuda.synchronize()
    st, word = A.attn_get_device_status()
    assert st == A.ERR_INVALID_ARG and word == 1 << 10, (st, hex(word))


class Cache:
    """A pool whose pages are dealt out in a shuffled order; everything that no token fills is NaN."""

    def __init__(self, dt, kind, capacity, Hkv, hd, page, seed, spare=2, most=None):
        self.dt, self.kind, self.Hkv, self.hd, self.page = dt, kind, Hkv, hd, page
        rng = np.random.default_rng(seed)
        used = [(n + page - 1) // page for n in capacity]
        self.most = most or max(used + [1])
        P = sum(used) + spare
        perm = rng.permutation(P)
        self.table = np.full((len(capacity), self.most), -1, np.int64)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = perm[at:at + n]
            at += n
        shape = (P, Hkv, page, hd)
        if is8(kind):
            self.k = torch.full(shape, NAN[kind], dtype=torch.uint8, device=DEV).view(T[kind])
            self.v = torch.full(shape, NAN[kind], dtype=torch.uint8, device=DEV).view(T[kind])
            self.ks = torch.full((P, Hkv), float("nan"), device=DEV)
            self.vs = torch.full((P, Hkv), float("nan"), device=DEV)
        else:
            self.k = torch.full(shape, float("nan"), dtype=T[kind], device=DEV)
            self.v = self.k.clone()
            self.ks = self.vs = None
        self.table_d = i32(self.table)

    def kw(self):
        return dict(Hkv=self.Hkv, k_scale=self.ks, v_scale=self.vs)

    def host(self):
        """(k, v, k_scale, v_scale) as the oracle takes them."""
        if is8(self.kind):
            return bits(self.k).copy(), bits(self.v).copy(), f64(self.ks), f64(self.vs)
        return f64(self.k), f64(self.v), None, None

    def fill(self, lengths, seed, unequal=True):
        """Random tokens, put in place by torch: every block of its own size, any scales."""
        g = torch.Generator().manual_seed(seed)
        for b, n in enumerate(lengths):
            for j in range((n + self.page - 1) // self.page):
                pg, m = int(self.table[b, j]), min(self.page, n - j * self.page)
                for pool, sc in ((self.k, self.ks), (self.v, self.vs)):
                    x = torch.randn((self.Hkv, m, self.hd), generator=g)
                    if unequal:
                        x *= 2.0 ** torch.randint(-2, 2, (self.Hkv, 1, 1), generator=g)
                    x = x.to(DEV)
                    if sc is not None:
                        s = x.abs().amax(dim=(1, 2)) / oracle.F8_TOP[self.kind]
                        sc[pg] = s
                        x = x / s[:, None, None]
                        # (8-bit types have no indexed assignment everywhere: write the bytes)
                        pool.view(torch.uint8)[pg, :, :m] = x.to(pool.dtype).view(torch.uint8)
                    else:
                        pool[pg, :, :m] = x.to(pool.dtype)

    def tokens(self, lengths):
        k, v, ks, vs = self.host()
        kind = self.kind if is8(self.kind) else None
        return [(oracle.paged_tokens(k, ks, self.table[b], n, kind), oracle.paged_tokens(v, vs, self.table[b], n, kind))
                for b, n in enumerate(lengths)]


def check_decode(c, q, lengths, o, lse, tokens=None, **flags):
    H, hd = q.shape[2] // c.hd, c.hd
    kw = dict(H=H, Hkv=c.Hkv, scale=1.0 / math.sqrt(hd))
    kw.update(flags)
    tok = c.tokens(lengths) if tokens is None else tokens
    ro, rl = oracle.paged_decode(f64(q), tok, lengths, **kw)
    ra, _ = oracle.paged_decode(f64(q), tok, lengths, absolute=True, **kw)
    qa = np.abs(f64(q)).reshape(q.shape[0], q.shape[1], H, hd)
    og, lg = f64(o), f64(lse)
    assert np.isfinite(og).all()
    for b, n in enumerate(lengths):
        k = tok[b][0][~np.isnan(tok[b][0][:, 0])] if n else tok[b][0]
        v = tok[b][1][~np.isnan(tok[b][1][:, 0])] if n else tok[b][1]
        smax = kw["scale"] * (qa[b].max(axis=(0, 1)).max() * np.abs(k).reshape(len(k), c.Hkv, hd).sum(2).max(initial=0.0))
        ds = 2.0 ** -18 * smax + 2.0 ** -19 * kw.get("softcap", 0.0)
        up = U["f16"] if is8(c.kind) else U[c.dt]
        flush = len(k) * 2.0 ** -25 * np.abs(v).max(initial=0.0) if (is8(c.kind) or c.dt == "f16") and n else 0.0
        tol = U[c.dt] * np.abs(ro[b]) + (up + 2 * ds + 2.0 ** -16) * 1.02 * ra[b] + flush + TINY[c.dt]
        bad = np.abs(og[b] - ro[b]) > tol
        assert not bad.any(), "sequence %d of %d tokens: O off by %.3g where %.3g is allowed" % (
            b, n, np.abs(og[b] - ro[b])[bad].max(), tol[bad].min())
        inf = np.isneginf(rl[b])
        assert (np.isneginf(lg[b]) == inf).all()
        assert (np.abs(lg[b][~inf] - rl[b][~inf]) <= ds + 2.0 ** -17 + 2.0 ** -20 * np.abs(rl[b][~inf])).all()


def run_decode(dt, kind, lengths, H, Hkv, hd, page, Lq, seed, **flags):
    c = Cache(dt, kind, lengths, Hkv, hd, page, seed)
    c.fill(lengths, seed)
    q = torch.randn((len(lengths), Lq, H * hd), generator=torch.Generator().manual_seed(seed + 1)).to(T[dt]).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=H, **c.kw(), **flags)
    status_ok()
    check_decode(c, q, lengths, o, lse, **flags)
    return c, q, o, lse


# -------------------------------------------------------------------- decode
@pytest.mark.parametrize("dt,kind", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2"),
                                     ("f16", "e5m2")])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_types_and_heads(dt, kind, hd, page):
    run_decode(dt, kind, [1, 0, 15, 16, 17, 63, 64, 65, 200], 8, 2, hd, page, 1, seed=hd + page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv,Lq", [(4, 4, 1), (8, 1, 2), (6, 2, 5), (7, 1, 9), (4, 1, 16), (2, 2, 16), (3, 3, 11)])
def test_decode_groups_and_draft_rows(kind, page, H, Hkv, Lq):
    run_decode("bf16", kind, [3, 129, 300, 1, 16], H, Hkv, 64, page, Lq, seed=H * 31 + Lq + page)


@pytest.mark.parametrize("hd,G,Lq", [(128, 8, 8), (256, 4, 16), (128, 1, 1), (256, 2, 9), (128, 5, 7), (64, 8, 3), (128, 8, 4),
                                     (128, 3, 6), (64, 2, 16), (64, 4, 13), (256, 8, 3)])
@pytest.mark.parametrize("kind", ["f16", "e4m3", "e5m2"])
def test_decode_many_rows_wide_heads(hd, G, Lq, kind):
    run_decode("f16", kind, [131, 2, 777], 2 * G, 2, hd, 32, Lq, seed=hd + G)


@pytest.mark.parametrize("kind", ["bf16", "e5m2", "e4m3"])
@pytest.mark.parametrize("flags", [dict(window=1), dict(window=17), dict(window=64), dict(window=100, softcap=5.0),
                                   dict(softcap=30.0), dict(causal=False), dict(causal=False, window=33),
                                   dict(scale=0.9), dict(causal=False, window=5, softcap=1.0)])
def test_decode_masks(kind, flags):
    run_decode("bf16", kind, [300, 5, 64, 66, 1], 4, 2, 128, 16, 4, seed=5, **flags)


@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 8, 640 + 9, 640 + 8, 639])
@pytest.mark.parametrize("causal", [False, True])
def test_decode_widest_windows(window, causal):
    """Rows at negative positions, under windows wider than the cache and just not."""
    run_decode("f16", "f16", [3, 7, 40, 640], 4, 2, 64, 16, 8, seed=46, window=window, causal=causal)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_decode_long_and_ragged(kind):
    run_decode("bf16", kind, [5000, 1, 0, 2047, 130], 8, 2, 128, 64, 2, seed=8)


@pytest.mark.parametrize("kind", ["f16", "e5m2"])
def test_decode_one_long_sequence(kind):
    run_decode("f16", kind, [20011], 4, 1, 64, 16, 1, seed=9)


def test_decode_many_short_sequences():
    run_decode("bf16", "e4m3", [(37 * b) % 91 for b in range(300)], 2, 1, 64, 16, 1, seed=10)


@pytest.mark.parametrize("dt,kind", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("bf16", "e5m2")])
def test_decode_what_a_row_does_not_see_has_no_effect(dt, kind):
    """Keys and values of the last draft token that are not finite reach the last row alone;
    those before a window reach no row that does not see them."""
    lengths, Lq = [130, 70], 3
    c = Cache(dt, kind, lengths, 2, 64, 16, seed=21)
    c.fill(lengths, 21)
    q = torch.randn((2, Lq, 4 * 64), generator=torch.Generator().manual_seed(4)).to(T[dt]).to(DEV)
    kw = dict(H=4, window=50, **c.kw())
    o0, l0 = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), **kw)
    check_decode(c, q, lengths, o0, l0, window=50)
    tokens = c.tokens(lengths)
    bad = [NAN[kind], 0x7f] if is8(kind) else [float("nan"), float("inf")]
    for w, pool in enumerate((c.k, c.v)):
        raw = pool.view(torch.uint8) if is8(kind) else pool
        for b, n in enumerate(lengths):
            # seen by the last row alone: the last token; by the first row alone: its window's first
            for t in (n - 1, n - Lq + 1 - 50):
                raw[int(c.table[b, t // 16]), :, t % 16] = bad[w]
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), **kw)
    status_ok()
    assert torch.isnan(o[:, 0]).all() and torch.isnan(o[:, 2]).all()
    # The middle row sees neither: it is held to the finite tokens' result, with a result's own
    # tolerance (its P may be rounded relative to another maximum than before, so that it
    # need not be the same bits).
    o[:, [0, 2]], lse[:, :, [0, 2]] = o0[:, [0, 2]], l0[:, :, [0, 2]]
    check_decode(c, q, lengths, o, lse, tokens=tokens, window=50)


@pytest.mark.parametrize("kind,Lq", [("bf16", 1), ("f16", 4), ("e4m3", 1), ("e5m2", 4), ("e4m3", 9)])
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("softcap", [0.0, 60.0])
def test_decode_scores_that_climb(kind, Lq, hd, softcap):
    """Keys that grow along the sequence: the rows' references have to move again and again, by more
    than 16 bits of p hold; and some that fall back, whose p are far below the reference's."""
    lengths = [900, 333]
    dt = "f16" if kind == "f16" else "bf16"
    c = Cache(dt, kind, lengths, 2, hd, 16, seed=41)
    c.fill(lengths, 41, unequal=False)
    q = torch.randn((2, Lq, 4 * hd), generator=torch.Generator().manual_seed(7)).to(T[dt]).to(DEV)
    grow = [1.0, 1.0, 4.0, 4.0, 12.0, 30.0, 1.0, 50.0]
    for b, n in enumerate(lengths):
        for j in range((n + 15) // 16):
            m = grow[j % len(grow)] if b else 1.0 + j
            pg = int(c.table[b, j])
            if is8(kind):
                c.ks[pg] *= m
            else:
                c.k[pg] *= m
    kw = dict(scale=0.5 / math.sqrt(hd), softcap=softcap)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=4, **c.kw(), **kw)
    status_ok()
    check_decode(c, q, lengths, o, lse, **kw)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("page,Lq", [(16, 1), (16, 3), (64, 1), (128, 5)])
def test_decode_scales_unlike_each_other(kind, page, Lq):
    """Scales of zero (blocks of zeros), of the first block alone, of either sign, 2^-40 to 2^20 apart."""
    lengths = [700, 260, 700, 300]
    c = Cache("bf16", kind, lengths, 2, 128, page, seed=43)
    c.fill(lengths, 43)
    for b in range(4):
        for j in range((lengths[b] + page - 1) // page):
            pg = int(c.table[b, j])
            if b == 0 and j % 3 == 1:
                c.vs[pg] = 0.0
            if b == 0 and j % 3 == 2:
                c.ks[pg, 0], c.ks[pg, 1] = 0.0, -c.ks[pg, 1]
            if b == 1:
                c.vs[pg] *= 2.0 ** (20 - 12 * (j % 6))
            if b == 2 and j == 0:
                c.vs[pg] = 0.0
            if b == 3:
                c.vs[pg, 0] *= -1.0
    q = torch.randn((4, Lq, 8 * 128), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=8, **c.kw())
    status_ok()
    check_decode(c, q, lengths, o, lse)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("first", [2.0 ** -58, 2.0 ** -30, 1.0])
def test_decode_scales_at_the_ends_of_their_range(kind, first):
    """Small blocks before the largest ones, all codes the largest: no sum leaves fp32 on the way."""
    n = 4000
    c = Cache("bf16", kind, [n], 2, 64, 16, seed=47)
    c.fill([n], 47)
    c.v.view(torch.uint8).fill_({"e4m3": 0x7E, "e5m2": 0x7B}[kind])
    c.vs.fill_(2.0 ** 40)
    c.vs[int(c.table[0, 0])] = first
    q = torch.randn((1, 2, 4 * 64), generator=torch.Generator().manual_seed(10)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([n]), H=4, **c.kw())
    status_ok()
    check_decode(c, q, [n], o, lse)


def test_decode_sequences_that_share_pages():
    """A common prefix: several sequences' tables name the same pages."""
    c = Cache("bf16", "e4m3", [200, 200, 200], 2, 64, 16, seed=44)
    c.fill([200, 200, 200], 44)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :5] = c.table[0, :5]
    c.table_d = i32(c.table)
    q = torch.randn((3, 1, 4 * 64), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([130, 200, 77]), H=4, **c.kw())
    status_ok()
    check_decode(c, q, [130, 200, 77], o, lse)


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_decode_mostly_empty_slots(kind):
    """A large padded batch: long runs of slots without a token, a few sequences among them."""
    lengths = [0] * 1500
    for b, n in ((3, 70), (4, 1), (640, 500), (1111, 64), (1112, 130), (1499, 17)):
        lengths[b] = n
    c, q, o, lse = run_decode("f16", kind, lengths, 4, 2, 64, 16, 2, seed=45)
    assert (o[700:1111] == 0).all()


def test_decode_two_calls_at_once():
    """Two streams, each call with the workspace that the binding makes for it."""
    calls = []
    for i, lengths in enumerate(([3000, 17, 900], [64, 2100, 5])):
        c = Cache("bf16", "e4m3", lengths, 4, 128, 16, seed=46 + i)
        c.fill(lengths, 46 + i)
        q = torch.randn((3, 2, 16 * 128), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(DEV)
        calls.append((c, q, lengths, i32(lengths), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, (c, q, lengths, ld, stream) in enumerate(calls):
            got[k].append(A.attn_paged_decode(q, c.k, c.v, c.table_d, ld, H=16, stream=stream, **c.kw()))
    status_ok()
    for k, (c, q, lengths, ld, stream) in enumerate(calls):
        check_decode(c, q, lengths, *got[k][0])
        for o, lse in got[k][1:]:
            np.testing.assert_array_equal(bits(o), bits(got[k][0][0]))


def test_decode_rows_that_see_nothing():
    """A block longer than its sequence: the rows at negative positions see nothing."""
    c, q, o, lse = run_decode("bf16", "e4m3", [0, 2, 0], 4, 2, 64, 16, 5, seed=3)
    assert (o[0] == 0).all() and (o[1, :3] == 0).all() and torch.isneginf(lse[1, :, :3]).all()


def test_decode_without_a_cache():
    q = torch.ones((2, 1, 4 * 64), dtype=torch.bfloat16, device=DEV)
    for P, most in ((0, 3), (3, 0)):
        pool = torch.zeros((P, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
        o, lse = A.attn_paged_decode(q, pool, pool, torch.zeros((2, most), dtype=torch.int32, device=DEV), i32([5, 5]), H=4, Hkv=2)
        status_ok()
        assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode_bad_pages_are_not_seen(kind, page):
    lengths = [400, 200, 90]
    c = Cache("bf16", kind, lengths, 2, 64, page, seed=6)
    c.fill(lengths, 6)
    for (b, j), bad in zip(((0, 1), (0, 3), (1, 0), (2, 0)), (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31)):
        if j * page < lengths[b]:
            c.table[b, j] = bad
    c.table_d = i32(c.table)
    q = torch.randn((3, 2, 4 * 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32(lengths), H=4, **c.kw())
    expect_flag()
    check_decode(c, q, lengths, o, lse)


def test_decode_lengths_out_of_range():
    lengths = [64, 64, 20]
    c = Cache("bf16", "bf16", lengths, 2, 64, 16, seed=7)
    c.fill(lengths, 7)
    q = torch.randn((3, 1, 4 * 64), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([2 ** 31 - 1, 64, -2 ** 31]), H=4, **c.kw())
    expect_flag()  # past the table: read as the capacity
    check_decode(c, q, [64, 64, 0], o, lse)


def test_decode_twice_is_the_same_bits_and_leaves_its_inputs():
    c, q, o, lse = run_decode("bf16", "e4m3", [700, 31, 64], 8, 2, 128, 32, 3, seed=12)
    before = bits(c.k).copy(), bits(c.v).copy()
    ws = torch.full((A.attn_paged_decode_workspace_size(3, 3, 8, 2, 128),), 0xff, dtype=torch.uint8, device=DEV)
    o2, lse2 = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([700, 31, 64]), H=8, workspace=ws, **c.kw())
    np.testing.assert_array_equal(bits(o), bits(o2))
    np.testing.assert_array_equal(f64(lse), f64(lse2))
    np.testing.assert_array_equal(before[0], bits(c.k))
    np.testing.assert_array_equal(before[1], bits(c.v))


def test_decode_without_lse_and_into_given_outputs():
    c, q, o, _ = run_decode("f16", "f16", [90, 3], 4, 4, 64, 16, 2, seed=13)
    out = torch.full_like(o, 7.0)
    got, none = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([90, 3]), H=4, o=out, want_lse=False, **c.kw())
    assert got is out and none is None
    np.testing.assert_array_equal(bits(out), bits(o))


# -------------------------------------------------------------------- append
def near_steps(x, kind):
    return np.maximum(U[kind] * np.abs(x), TINY[kind])


def run_append(dt, kind, before, new, H, Hkv, hd, page, theta, seed, pad=3, turn_q=True, spread=1.0, c=None):
    """One append on a filled cache, checked in full: every byte of both pools and scales."""
    lengths = [a + n for a, n in zip(before, new)]
    c = c or Cache(dt, kind, lengths, Hkv, hd, page, seed)
    if any(before):
        c.fill(before, seed)
    cu = np.cumsum([0] + list(new))
    rows = int(cu[-1]) + pad
    qkv = torch.randn((rows, (H + 2 * Hkv) * hd), generator=torch.Generator().manual_seed(seed + 3)) * spread
    qkv = qkv.to(T[dt]).to(DEV)
    q, k, v = qkv[:, :H * hd], qkv[:, H * hd:(H + Hkv) * hd], qkv[:, (H + Hkv) * hd:]
    q_out = torch.full((rows, H * hd), 9.0, dtype=T[dt], device=DEV) if turn_q else None
    host = c.host()
    A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=H, q=q if turn_q else None, q_out=q_out,
                        rope_theta=theta, **c.kw())
    status_ok()
    n = int(cu[-1])
    k8 = kind if is8(kind) else None
    rk, rv, rks, rvs, exact = oracle.paged_append(f64(k), f64(v), *host, c.table, lengths, cu, Hkv=Hkv, kind=k8, theta=theta)
    gk, gv, gks, gvs = c.host()
    np.testing.assert_array_equal(gv, rv)  # nothing turned: the oracle's values, and nothing else touched
    if k8:
        np.testing.assert_array_equal(gks, rks)
        np.testing.assert_array_equal(gvs, rvs)
    if not theta:
        np.testing.assert_array_equal(gk, rk)
    else:
        fresh = np.zeros(rk.shape, bool)
        at = 0
        for b in range(len(lengths)):
            for t in range(max(lengths[b] - new[b], 0), lengths[b]):
                fresh[c.table[b, t // page], :, t % page] = True
        np.testing.assert_array_equal(gk[~fresh], rk[~fresh])
        if k8:
            for w, pg, row, x in exact:
                if w == 0:
                    got = oracle.f8_values(kind)[gk[pg, :, row]]
                    x = np.clip(x, -oracle.F8_TOP[kind], oracle.F8_TOP[kind])
                    pair = np.hypot(x[:, :hd // 2], x[:, hd // 2:])
                    slack = 2.0 ** -20 * np.concatenate([pair, pair], 1)
                    assert (np.abs(got - x) <= near_steps(np.abs(x) + slack, kind) + slack).all()
        else:
            for b in range(len(lengths)):
                for i in range(new[b]):
                    t = lengths[b] - new[b] + i
                    if t < 0:
                        continue
                    x = oracle.turn_rows(f64(k[cu[b] + i:cu[b] + i + 1]), [t], hd, theta).reshape(Hkv, hd)
                    close(gk[c.table[b, t // page], :, t % page], x, kind)
    if turn_q:
        got = f64(q_out)
        for b in range(len(lengths)):
            pos = np.arange(lengths[b] - new[b], lengths[b])
            x = f64(q[cu[b]:cu[b + 1]])
            x = oracle.turn_rows(x, pos, hd, theta) if theta else x
            live = pos >= 0
            close(got[cu[b]:cu[b + 1]][live].reshape(-1, H, hd), x[live].reshape(-1, H, hd), dt)
            assert (got[cu[b]:cu[b + 1]][~live] == 9.0).all()
        assert (got[n:] == 9.0).all()
    return c, lengths


def close(got, x, kind):
    half = x.shape[-1] // 2
    pair = np.hypot(x[..., :half], x[..., half:])
    slack = 2.0 ** -20 * np.concatenate([pair, pair], -1)
    assert (np.abs(got - x) <= near_steps(np.abs(x) + slack, kind) + slack).all()


@pytest.mark.parametrize("dt,kind", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2"),
                                     ("f16", "e5m2")])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("theta", [None, 10000.0])
def test_append_types_and_heads(dt, kind, hd, theta):
    run_append(dt, kind, [0, 5, 16, 31, 40], [1, 1, 1, 1, 1], 4, 2, hd, 16, theta, seed=hd)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_append_ragged_chunks(kind, page):
    run_append("bf16", kind, [0, 3, 16, 100, 63, 7], [70, 0, 300, 1, 65, 2], 6, 3, 64, page, 500.0, seed=page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_long_prompt(kind):
    run_append("bf16", kind, [0, 17], [900, 1300], 2, 1, 128, 64, 10000.0, seed=2)


def test_append_many_sequences():
    """More sequences than one round of the row search takes, some with nothing new."""
    new = [(b * 7) % 3 for b in range(1100)]
    run_append("bf16", "e4m3", [(b * 5) % 40 for b in range(1100)], new, 1, 1, 64, 16, 10000.0, seed=4, turn_q=False)


@pytest.mark.parametrize("kind,hd,page,Hkv,theta", [("e4m3", 256, 64, 2, 500.0), ("e5m2", 128, 128, 2, None),
                                                    ("e4m3", 64, 256, 3, 10000.0), ("e4m3", 64, 64, 12, 10000.0),
                                                    ("e5m2", 64, 32, 11, 10000.0), ("e4m3", 128, 256, 2, 10000.0)])
def test_append_blocks_of_every_size(kind, hd, page, Hkv, theta):
    """Blocks of 128 to 2048 pieces of 16 elements, enough of them for several heads to a team."""
    new = [(b * 37) % 71 for b in range(80)]
    run_append("bf16", kind, [(b * 23) % 50 for b in range(80)], new, Hkv, Hkv, hd, page, theta, seed=5 + page, turn_q=hd == 64)


@pytest.mark.parametrize("kind,hd,page", [("e4m3", 128, 64), ("e5m2", 128, 16), ("e4m3", 64, 16), ("e5m2", 64, 32), ("e4m3", 256, 16),
                                          ("e4m3", 256, 128), ("bf16", 128, 64)])
def test_append_chunks_among_single_tokens(kind, hd, page):
    """Running prompts' chunks beside many sequences with a token each: blocks of 1 row to whole pages."""
    new = [1] * 100
    for b, n in ((0, 17), (9, 0), (10, 66), (11, 3), (30, 5), (31, 8), (32, 9), (60, 100), (99, 73)):
        new[b] = n
    before = [(b * 31) % 90 for b in range(100)]
    before[10] = -7  # (rows before the sequence's beginning are not stored)
    run_append("bf16", kind, before, new, 4, 2, hd, page, 10000.0, seed=6 + page)


def test_append_far_positions_keep_their_angle():
    """Positions of hundreds of thousands: fp32 angles would be off by hundredths."""
    page, far = 256, 700001
    c = Cache("f16", "f16", [3], 1, 64, page, seed=1, most=far // page + 2)
    c.table[0, far // page] = 0
    c.table_d = i32(c.table)
    k = torch.randn((1, 64), generator=torch.Generator().manual_seed(8)).half().to(DEV)
    q_out = A.attn_paged_append(k, k, c.k, c.v, c.table_d, i32([far + 1]), i32([0, 1]), H=1, q=k, rope_theta=10000.0, **c.kw())
    status_ok()
    x = oracle.turn_rows(f64(k), [far], 64, 10000.0)
    close(f64(q_out), x, "f16")
    close(f64(c.k[0, 0, far % page])[None], x, "f16")


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_append_grows_a_block(kind):
    """Steps of ever larger tokens: each moves the block's earlier codes."""
    c = Cache("bf16", kind, [40, 20], 2, 64, 32, seed=5)
    at = [0, 0]
    for step, spread in enumerate((1e-3, 0.02, 1.0, 0.5, 300.0, 3e4, 1.0)):
        new = [5, 2]
        lengths = [a + n for a, n in zip(at, new)]
        run_step(c, at, new, spread, seed=40 + step, theta=None)
        at = lengths


def run_step(c, at, new, spread, seed, theta):
    lengths, cu = [a + n for a, n in zip(at, new)], np.cumsum([0] + new)
    g = torch.Generator().manual_seed(seed)
    k, v = ((torch.randn((int(cu[-1]), c.Hkv * c.hd), generator=g) * spread).to(T[c.dt]).to(DEV) for _ in range(2))
    host = c.host()
    A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=c.Hkv, rope_theta=theta, **c.kw())
    status_ok()
    want = oracle.paged_append(f64(k), f64(v), *host, c.table, lengths, cu, Hkv=c.Hkv, kind=c.kind if is8(c.kind) else None,
                               theta=theta)
    for got, ref in zip(c.host(), want):
        if ref is not None:
            np.testing.assert_array_equal(got, ref)
    return k, v


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e5m2"])
def test_append_values_that_are_not_finite_and_zeros(kind):
    c = Cache("bf16", kind, [32, 32], 2, 64, 16, seed=9)
    k = torch.randn((24, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    k[0, 5], k[3, 70], k[9, 1] = float("inf"), float("-inf"), float("nan")
    k[12:] = 0.0
    v = -k
    host = c.host()
    A.attn_paged_append(k.to(DEV), v.to(DEV), c.k, c.v, c.table_d, i32([12, 12]), i32([0, 12, 24]), H=2, **c.kw())
    status_ok()
    want = oracle.paged_append(f64(k), f64(v), *host, c.table, [12, 12], [0, 12, 24], Hkv=2, kind=kind if is8(kind) else None)
    values = oracle.f8_values(kind) if is8(kind) else None
    for got, ref in list(zip(c.host(), want))[:2]:
        if values is not None:  # a NaN has two codes
            got, ref = values[got], values[ref]
        np.testing.assert_array_equal(got, ref)
    for got, ref in list(zip(c.host(), want))[2:4]:
        if ref is not None:
            np.testing.assert_array_equal(got, ref)
    if is8(kind):
        assert (f64(c.ks)[c.table[1, 0]] == 2.0 ** -64).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_padding_slots_and_rows_are_left_alone(kind):
    """Slots of length 0 with a row each, a block longer than its sequence, rows behind cu[-1] and before cu[0]."""
    c = Cache(dt="bf16", kind=kind, capacity=[20, 0, 2, 0], Hkv=2, hd=64, page=16, seed=3)
    run_append("bf16", kind, [19, -1, -3, -2], [1, 1, 5, 2], 4, 2, 64, 16, 10000.0, seed=3, c=_filled(c, [19, 0, 0, 0]))
    k = torch.ones((8, 128), dtype=torch.bfloat16, device=DEV)
    host = c.host()
    A.attn_paged_append(k, k, c.k, c.v, c.table_d, i32([20, 0, 2, 0]), i32([8, 8, 8, 8, 8]), H=2, **c.kw())
    status_ok()
    for got, ref in zip(c.host(), host):
        if ref is not None:
            np.testing.assert_array_equal(got, ref)


def _filled(c, lengths):
    c.fill(lengths, 77)
    c.fill = lambda *a: None
    return c


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_bad_pages_lengths_and_prefix_sums(kind):
    """Nothing outside the pages that the arrays name in range is written, and the status says so."""
    for table_bad, lengths, cu in (
            ([-1, 99, 2 ** 31 - 1, -2 ** 31], [40, 20, 17, 16], [0, 40, 60, 77, 93]),
            (None, [80, 2 ** 31 - 1, 17, -2 ** 31], [0, 40, 60, 77, 93]),
            (None, [40, 20, 17, 16], [0, 50, 20, 77, 93]),
            (None, [40, 20, 17, 16], [-5, 40, 60, 2 ** 31 - 1, -2 ** 31])):
        c = Cache("bf16", kind, [40, 20, 17, 16], 2, 64, 16, seed=11)
        if table_bad:
            c.table[:, 0] = table_bad
        c.table_d = i32(c.table)
        g = torch.Generator().manual_seed(2)
        k, v = (torch.randn((93, 128), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        q_out = torch.zeros((93, 256), dtype=torch.bfloat16, device=DEV)
        q = torch.ones((93, 256), dtype=torch.bfloat16, device=DEV)
        host = c.host()
        A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32(cu), H=4, q=q, q_out=q_out, rope_theta=100.0, **c.kw())
        expect_flag()
        spare = np.setdiff1d(np.arange(c.k.shape[0]), c.table.ravel())
        for got, ref in zip(c.host()[:2], host[:2]):
            np.testing.assert_array_equal(got[spare], ref[spare])


def test_append_in_place_queries_and_strides():
    """q turned in place; k and v as columns of wider rows, a multiple of 8 apart."""
    g = torch.Generator().manual_seed(6)
    c = Cache("f16", "f16", [9, 30], 2, 64, 16, seed=2)
    wide = torch.randn((12, 512 + 8), generator=g).half().to(DEV)
    q = torch.randn((12, 256), generator=g).half().to(DEV)
    want = oracle.turn_rows(f64(q), list(range(4, 9)) + list(range(23, 30)), 64, 50.0)
    out = A.attn_paged_append(wide[:, 8:136], wide[:, 200:328], c.k, c.v, c.table_d, i32([9, 30]), i32([0, 5, 12]), H=4, q=q,
                              q_out=q, rope_theta=50.0, **c.kw())
    status_ok()
    assert out is q
    close(f64(q).reshape(-1, 4, 64), want.reshape(-1, 4, 64), "f16")
    np.testing.assert_array_equal(f64(c.v[int(c.table[0, 0]), :, 4:9]), f64(wide[:5, 200:328]).reshape(5, 2, 64).transpose(1, 0, 2))


# -------------------------------------------------------------------- gather
@pytest.mark.parametrize("dt,kind", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e5m2"),
                                     ("f16", "e5m2")])
@pytest.mark.parametrize("hd,page", [(64, 16), (128, 64), (256, 32), (128, 256)])
def test_gather(dt, kind, hd, page):
    lengths = [70, 0, 1, 257, 16]
    c = Cache(dt, kind, lengths, 3, hd, page, seed=hd + page)
    c.fill(lengths, 1)
    cu = np.cumsum([2] + lengths)  # two rows before the first sequence, three behind the last
    n = int(cu[-1]) + 3
    ko = torch.full((n, 3 * hd), 5.0, dtype=T[dt], device=DEV)
    vo = ko.clone()
    A.attn_paged_gather(c.k, c.v, c.table_d, i32(cu), n, dtype=T[dt], k_out=ko, v_out=vo, **c.kw())
    status_ok()
    for got, w in ((f64(ko), 0), (f64(vo), 1)):
        for b, t in enumerate(c.tokens(lengths)):
            x = t[w]
            if is8(kind):  # fp32 product of two exact factors, then the rows' type
                assert (np.abs(got[cu[b]:cu[b + 1]] - x) <= (U[dt] + 2.0 ** -24) * np.abs(x) + TINY[dt]).all()
            else:
                np.testing.assert_array_equal(got[cu[b]:cu[b + 1]], x)
        assert (got[:2] == 5).all() and (got[cu[-1]:] == 5).all()


def test_gather_bad_pages_read_as_zero():
    c = Cache("bf16", "e4m3", [60, 20], 2, 64, 16, seed=4)
    c.fill([60, 20], 4)
    c.table[0, 1], c.table[1, 0] = -7, c.k.shape[0]
    k, v = A.attn_paged_gather(c.k, c.v, i32(c.table), i32([0, 60, 80]), 80, dtype=torch.bfloat16, **c.kw())
    expect_flag()
    for x, w in ((f64(k), 0), (f64(v), 1)):
        assert (x[16:32] == 0).all() and (x[60:76] == 0).all()
        assert (x[:16] != 0).any() and (x[32:60] != 0).any() and (x[76:80] != 0).any()
    # more tokens than the table has room for, prefix sums that decrease
    A.attn_paged_gather(c.k, c.v, i32(c.table), i32([0, 75, 80]), 80, dtype=torch.bfloat16, **c.kw())
    expect_flag()
    A.attn_paged_gather(c.k, c.v, i32(c.table), i32([0, 90, 80]), 80, dtype=torch.bfloat16, **c.kw())
    expect_flag()


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("dt,kind", [("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e5m2")])
def test_a_serving_run(dt, kind):
    """Prompts appended, steps of one and of three tokens attended as they arrive, then the next
    chunk of one prompt over its cached tokens read back."""
    H, Hkv, hd, page, theta = 8, 2, 128, 16, 10000.0
    upto = [[37, 64, 5], [38, 65, 6], [41, 68, 9], [42, 69, 10]]
    c = Cache(dt, kind, [200, 69, 10], Hkv, hd, page, seed=30)
    g = torch.Generator().manual_seed(31)
    at, hist = [0, 0, 0], [([], []), ([], []), ([], [])]
    for lengths in upto:
        new = [u - a for u, a in zip(lengths, at)]
        cu = np.cumsum([0] + new)
        rows = torch.randn((int(cu[-1]), (H + 2 * Hkv) * hd), generator=g).to(T[dt]).to(DEV)
        q, k, v = rows[:, :H * hd], rows[:, H * hd:-Hkv * hd], rows[:, -Hkv * hd:]
        ld = i32(lengths)
        qr = A.attn_paged_append(k, v, c.k, c.v, c.table_d, ld, i32(cu), H=H, q=q, rope_theta=theta, **c.kw())
        for b in range(3):
            pos = np.arange(at[b], lengths[b])
            hist[b][0].append(oracle.turn_rows(f64(k[cu[b]:cu[b + 1]]), pos, hd, theta))
            hist[b][1].append(f64(v[cu[b]:cu[b + 1]]))
        if max(new) == min(new) <= 16:
            Lq = new[0]
            o, lse = A.attn_paged_decode(qr.view(3, Lq, H * hd), c.k, c.v, c.table_d, ld, H=H, **c.kw())
            status_ok()
            check_decode(c, qr.view(3, Lq, H * hd), lengths, o, lse)
            # and against attention on what went in: the cache's own rounding is all that is between
            tok = [tuple(np.concatenate(x) for x in h) for h in hist]
            qt = np.stack([oracle.turn_rows(f64(q[cu[b]:cu[b + 1]]), np.arange(at[b], lengths[b]), hd, theta) for b in range(3)])
            ro, _ = oracle.paged_decode(qt, tok, lengths, H=H, Hkv=Hkv, scale=1 / math.sqrt(hd))
            assert np.linalg.norm(f64(o) - ro) <= 3 * U[kind] * np.linalg.norm(ro)
        at = lengths
    # the first prompt goes on: 100 more tokens, attended by the prefill kernel over the pages read back
    lengths, n = [142, 69, 10], 100
    rows = torch.randn((n, (H + 2 * Hkv) * hd), generator=g).to(T[dt]).to(DEV)
    q, k, v = rows[:, :H * hd], rows[:, H * hd:-Hkv * hd], rows[:, -Hkv * hd:]
    qr = A.attn_paged_append(k, v, c.k, c.v, c.table_d, i32(lengths), i32([0, n, n, n]), H=H, q=q, rope_theta=theta, **c.kw())
    kk, vv = A.attn_paged_gather(c.k, c.v, c.table_d[:1], i32([0, 142]), 142, dtype=T[dt], **c.kw())
    o, lse = A.attn_fwd(qr[None].contiguous(), kk[None], vv[None], H=H, Hkv=Hkv, causal=True, q_offset=42)
    status_ok()
    tok = c.tokens(lengths)[0]
    ro, rl = oracle.fwd(f64(qr)[None], tok[0][None], tok[1][None], H=H, Hkv=Hkv, scale=1 / math.sqrt(hd), causal=True, q_offset=42)
    assert np.abs(f64(o) - ro).max() <= 2e-2 and np.abs(f64(lse) - rl).max() <= 2e-2  # the prefill tests' O; the keys' 16-bit rounding on LSE


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_captured_step_is_replayed_as_the_cache_grows(kind):
    """One graph of append and decode; lengths, page table, rows and pages change between replays."""
    B, H, Hkv, hd, page = 4, 4, 2, 64, 16
    full = [50, 33, 20, 0]
    c = Cache("bf16", kind, full, Hkv, hd, page, seed=17, most=6)
    c.fill([14, 31, 2, 0], 17)
    rows = torch.zeros((B, (H + 2 * Hkv) * hd), dtype=torch.bfloat16, device=DEV)
    lengths, cu, table = i32([0] * B), i32(range(B + 1)), torch.full_like(c.table_d, -1)
    ws = torch.empty(A.attn_paged_decode_workspace_size(B, 1, H, Hkv, hd), dtype=torch.uint8, device=DEV)

    def step():
        q, k, v = rows[:, :H * hd], rows[:, H * hd:-Hkv * hd], rows[:, -Hkv * hd:]
        qr = A.attn_paged_append(k, v, c.k, c.v, table, lengths, cu, H=H, q=q, rope_theta=1000.0, **c.kw())
        return qr, *A.attn_paged_decode(qr.view(B, 1, -1), c.k, c.v, table, lengths, H=H, workspace=ws, **c.kw())

    step()  # an empty batch
    status_ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, o, lse = step()
    at = [14, 31, 2, 0]
    table.copy_(c.table_d)
    for i in range(5):
        at = [a + 1 if b < 3 else 0 for b, a in enumerate(at)]
        if i == 3:
            at[2] = 0  # its slot runs empty
        rows.copy_(torch.randn(rows.shape, generator=torch.Generator().manual_seed(i)).to(rows.dtype))
        lengths.copy_(i32(at))
        host = c.host()
        graph.replay()
        status_ok()
        q = rows[:, :H * hd]
        k, v = rows[:, H * hd:-Hkv * hd], rows[:, -Hkv * hd:]
        want = oracle.paged_append(f64(k), f64(v), *host, c.table, at, range(B + 1), Hkv=Hkv, kind=kind if is8(kind) else None,
                                   theta=1000.0)
        np.testing.assert_array_equal(c.host()[1], want[1])
        x = oracle.turn_rows(f64(q), np.array(at) - 1, hd, 1000.0)
        live = [b for b in range(B) if at[b]]
        close(f64(qr)[live].reshape(-1, H, hd), x[live].reshape(-1, H, hd), "bf16")
        check_decode(c, qr.view(B, 1, -1)[live], [at[b] for b in live], o[live], lse[live], tokens=[c.tokens(at)[b] for b in live])
        for b in range(B):
            if not at[b]:
                assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()


def test_calls_on_another_stream():
    """The stream argument: the call runs there, and so is its own memory given back there."""
    lengths = [300, 77]
    c = Cache("bf16", "e4m3", lengths, 2, 128, 32, seed=19)
    c.fill(lengths, 19)
    q = torch.randn((2, 1, 8 * 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    ld = i32(lengths)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for handle in (side, side.cuda_stream):
        torch.cuda._sleep(20000000)  # the current stream is busy; nothing waits for it
        o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, ld, H=8, stream=handle, **c.kw())
        side.synchronize()
        got.append((o, lse))
    torch.cuda.synchronize()
    status_ok()
    for o, lse in got:
        check_decode(c, q, lengths, o, lse)
    k = torch.ones((2, 256), dtype=torch.bfloat16, device=DEV)
    one, cu = i32([0, 1, 2]), i32([0, 300, 377])
    torch.cuda.synchronize()
    qo = A.attn_paged_append(k, k, c.k, c.v, c.table_d, ld, one, H=8, q=q[:, 0], rope_theta=10.0, stream=side, **c.kw())
    kk, vv = A.attn_paged_gather(c.k, c.v, c.table_d, cu, 377, dtype=torch.bfloat16, stream=side, **c.kw())
    side.synchronize()
    status_ok()
    # a block that holds earlier tokens keeps its scale: 1 is rounded to e4m3 in it, and to bf16
    assert (np.abs(f64(vv)[[299, 376]] - 1) <= U["e4m3"] + 2 * U["bf16"]).all() and torch.isfinite(qo.float()).all()


def test_calls_on_the_default_stream_by_its_handle():
    """A handle of 0 is the default stream, whatever the current one is: the call waits for the lengths."""
    c = Cache("f16", "f16", [90], 2, 64, 16, seed=20)
    c.fill([90], 20)
    q = torch.randn((1, 2, 4 * 64), generator=torch.Generator().manual_seed(2)).to(torch.float16).to(DEV)
    ld, new = i32([0]), i32([90])
    torch.cuda.synchronize()
    torch.cuda._sleep(20000000)
    ld.copy_(new)
    with torch.cuda.stream(torch.cuda.Stream()):
        o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, ld, H=4, stream=0, **c.kw())
    torch.cuda.synchronize()
    status_ok()
    check_decode(c, q, [90], o, lse)


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
        k, v = c.k, c.v
        c.k = torch.zeros((P, Hkv, page, hd), dtype=torch.uint8 if is8(kind) else T[kind], device=DEV).view(T[kind])
        c.v = torch.zeros((P, Hkv, page, hd), dtype=torch.uint8 if is8(kind) else T[kind], device=DEV).view(T[kind])
        if is8(kind):
            c.ks, c.vs = torch.ones((P, Hkv), device=DEV), torch.ones((P, Hkv), device=DEV)
        c.table[0] = [P - 1, P - 2]
        c.table_d = i32(c.table)
        g = torch.Generator().manual_seed(2)
        x, y = (torch.randn((100, Hkv * hd), generator=g).to(T[dt]).to(DEV) for _ in range(2))
        A.attn_paged_append(x, y, c.k, c.v, c.table_d, i32([100]), i32([0, 100]), H=Hkv, **c.kw())
        ko, vo = A.attn_paged_gather(c.k, c.v, c.table_d, i32([0, 100]), 100, dtype=T[dt], **c.kw())
        q = torch.randn((1, 2, Hkv * hd), generator=g).to(T[dt]).to(DEV)
        o, lse = A.attn_paged_decode(q, c.k, c.v, c.table_d, i32([100]), H=Hkv, **c.kw())
        status_ok()
        assert (np.abs(f64(vo) - f64(y)) <= (U[kind] + U[dt]) * np.abs(f64(y)) + 2.0 ** -7 * np.abs(f64(y)).max()).all()
        check_decode(c, q, [100], o, lse, tokens=[(f64(ko), f64(vo))])
        assert not bits(c.k[:2]).any()
        del c, k, v
        torch.cuda.empty_cache()
