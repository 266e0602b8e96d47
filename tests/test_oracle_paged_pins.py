"""Pins for the oracle's paged cache: the 8-bit types against torch's, the row turn against
rope(), the append against its own reading back, the decode against the dense oracle."""
import numpy as np
import pytest
import torch

T8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_values_and_rounding_of_the_8_bit_types(oracle, kind):
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(T8[kind]).float().numpy()
    np.testing.assert_array_equal(oracle.f8_values(kind), want.astype(np.float64))
    g = np.random.default_rng(3)
    x = np.concatenate([g.standard_normal(4000) * 10.0 ** g.uniform(-7, 2, 4000), want[np.isfinite(want)]])
    pos = np.sort(want[np.isfinite(want) & (want >= 0)]).astype(np.float64)
    x = np.concatenate([x, (pos[1:] + pos[:-1]) / 2, -(pos[1:] + pos[:-1]) / 2])  # ties
    x = x[np.abs(x) <= oracle.F8_TOP[kind]].astype(np.float32)
    got = oracle.f8_values(kind)[oracle.f8_round(x, kind)]
    np.testing.assert_array_equal(got, torch.from_numpy(x).to(T8[kind]).double().numpy())
    top = oracle.F8_TOP[kind]
    got = oracle.f8_values(kind)[oracle.f8_round([top * 3, -top * 3, np.inf, -np.inf, np.nan], kind)]
    np.testing.assert_array_equal(got[:4], [top, -top, top, -top])
    assert np.isnan(got[4])


def test_row_turn_is_rope(oracle):
    x = np.random.default_rng(5).standard_normal((7, 3 * 16))
    np.testing.assert_allclose(oracle.turn_rows(x, range(11, 18), 16, 700.0),
                               oracle.rope(x[None], head_dim=16, pos=11, theta=700.0)[0], atol=1e-13)


def test_append_in_steps_reads_back_what_went_in(oracle):
    g = np.random.default_rng(7)
    page, Hkv, hd = 4, 2, 8
    lengths = [9, 0, 6]
    table = np.array([[5, 1, 3], [-1, -1, -1], [0, 6, -1]])
    kv = [(g.standard_normal((n, Hkv * hd)), g.standard_normal((n, Hkv * hd))) for n in lengths]
    kc, vc = np.full((7, Hkv, page, hd), np.nan), np.full((7, Hkv, page, hd), np.nan)
    for done, upto in (([0, 0, 0], [3, 0, 6]), ([3, 0, 6], [9, 0, 6])):
        cu = np.cumsum([0] + [u - d for d, u in zip(done, upto)])
        k, v = (np.concatenate([kv[b][w][done[b]:upto[b]] for b in range(3)]) for w in range(2))
        kc, vc, _, _, _ = oracle.paged_append(k, v, kc, vc, None, None, table, upto, cu, Hkv=Hkv)
    for b, n in enumerate(lengths):
        np.testing.assert_array_equal(oracle.paged_tokens(kc, None, table[b], n), kv[b][0])
        np.testing.assert_array_equal(oracle.paged_tokens(vc, None, table[b], n), kv[b][1])
    assert np.isnan(kc[[2, 4]]).all() and np.isnan(kc[3, :, 1:]).all() and np.isnan(kc[6, :, 2:]).all()


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_a_block_takes_the_smallest_power_of_two_that_fits(oracle, kind):
    page, Hkv, hd = 4, 1, 8
    top = oracle.F8_TOP[kind]
    code = np.zeros((1, Hkv, page, hd), np.uint8)
    ones = np.ones((1, Hkv))
    table = np.array([[0]])
    rows = np.full((1, hd), 1.0)
    for first, want in ((top, 1.0), (np.nextafter(top, 1e9), 2.0), (top / 2, 0.5), (0.0, 2.0 ** -64)):
        x = rows * first
        kc, vc, ks, _, _ = oracle.paged_append(x, x, code, code, ones, ones, table, [1], [0, 1], Hkv=1, kind=kind)
        assert ks[0, 0] == want
    # a second token of four times the size: the first one's codes move down by two binades
    kc, vc, ks, vs, _ = oracle.paged_append(rows, rows, code, code, ones, ones, table, [1], [0, 1], Hkv=1, kind=kind)
    kc2, _, ks2, _, _ = oracle.paged_append(rows * 4, rows, kc, vc, ks, vs, table, [2], [0, 1], Hkv=1, kind=kind)
    assert ks2[0, 0] == 4 * ks[0, 0]
    np.testing.assert_array_equal(oracle.paged_tokens(kc2, ks2, table[0], 2, kind), [[1.0] * hd, [4.0] * hd])
    # a smaller one leaves the scale
    _, _, ks3, _, _ = oracle.paged_append(rows / 9, rows, kc2, vc, ks2, vs, table, [3], [0, 1], Hkv=1, kind=kind)
    assert ks3[0, 0] == ks2[0, 0]


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_a_block_keeps_a_large_scale_of_either_sign(oracle, kind):
    page, hd = 4, 8
    code = np.full((1, 1, page, hd), oracle.f8_round(2.0, kind), np.uint8)
    table, rows = np.array([[0]]), np.full((1, hd), 1.0)
    for old, want in ((-4.0, -4.0), (-2.0 ** -30, 1.0), (0.0, 1.0)):
        sc = np.full((1, 1), old)
        x = rows * oracle.F8_TOP[kind]
        kc, _, ks, _, _ = oracle.paged_append(x, x, code, code, sc, sc, table, [2], [0, 1], Hkv=1, kind=kind)
        assert ks[0, 0] == want
        got = oracle.paged_tokens(kc, ks, table[0], 2, kind)
        np.testing.assert_array_equal(got[1], x[0])
        np.testing.assert_allclose(got[0], 2.0 * old, atol=2.0 ** -9 * abs(want) if old != want else 0)


def test_decode_is_the_dense_oracle_on_the_gathered_tokens(oracle):
    g = np.random.default_rng(11)
    H, Hkv, hd, Lq = 4, 2, 8, 3
    lengths = [10, 3, 2, 0]
    tokens = [(g.standard_normal((n, Hkv * hd)), g.standard_normal((n, Hkv * hd))) for n in lengths]
    q = g.standard_normal((4, Lq, H * hd))
    for kw in (dict(causal=True), dict(causal=True, window=4, softcap=2.0), dict(causal=False, window=3)):
        o, lse = oracle.paged_decode(q, tokens, lengths, H=H, Hkv=Hkv, scale=0.3, **kw)
        for b in (0, 1):
            ro, rl = oracle.fwd(q[b:b + 1], tokens[b][0][None], tokens[b][1][None], H=H, Hkv=Hkv, scale=0.3,
                                q_offset=lengths[b] - Lq, **kw)
            np.testing.assert_allclose(o[b], ro[0], atol=1e-13)
            np.testing.assert_allclose(lse[b], rl[0], atol=1e-13)
        # two tokens: the rows sit at -1, 0, 1, the last two are the dense rows 0 and 1
        ro, rl = oracle.fwd(q[2:3, 1:], tokens[2][0][None], tokens[2][1][None], H=H, Hkv=Hkv, scale=0.3, **kw)
        np.testing.assert_allclose(o[2, 1:], ro[0], atol=1e-13)
        if kw["causal"]:
            assert (o[2, 0] == 0).all() and np.isneginf(lse[2, :, 0]).all()
        assert (o[3] == 0).all() and np.isneginf(lse[3]).all()
