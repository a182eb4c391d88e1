"""Pins of the oracle's position rotation, 4-bit cache and windowed attention (CPU)."""

import numpy as np
import pytest

from oracle import paged


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 64, 128])
def test_rope_depends_on_the_distance_alone(rotary, interleaved):
    r = np.random.default_rng(1)
    q, k = r.standard_normal((1, 1, 128)), r.standard_normal((1, 1, 128))

    def dot(p, d):
        def turn(x, at):
            a = paged.rope_angles([at], rotary, 1e4)
            return paged.rope(x, np.cos(a), np.sin(a), interleaved)
        return float((turn(q, p + d) * turn(k, p)).sum())

    assert abs(dot(0, 5) - dot(77, 5)) < 1e-10
    assert abs(dot(0, 0) - float((q * k).sum())) < 1e-12
    if rotary:
        assert abs(dot(0, 5) - dot(0, 6)) > 1e-3


def test_rope_pairs_by_hand():
    x = np.zeros((1, 1, 128))
    x[0, 0, 0] = 1.0
    c, s = np.zeros((1, 64)), np.ones((1, 64))  # a quarter turn
    assert np.argmax(paged.rope(x, c, s, False)[0, 0]) == 64
    assert np.argmax(paged.rope(x, c, s, True)[0, 0]) == 1
    assert np.argmax(paged.rope(x, c[:, :32], s[:, :32], False)[0, 0]) == 32
    x[0, 0, 0], x[0, 0, 100] = 0.0, 1.0
    assert np.array_equal(paged.rope(x, c[:, :32], s[:, :32], True), x)  # beyond the rotated channels


def test_every_nibble_of_a_tile_is_used_once():
    u, j = np.meshgrid(np.arange(16), np.arange(128), indexing="ij")
    for place, lo, hi in ((paged.k_place, 0, 1024), (paged.v_place, 1024, 2048)):
        byte, nib = place(u, j)
        assert byte.min() == lo and byte.max() == hi - 1
        assert len(set(zip(byte.ravel().tolist(), nib.ravel().tolist()))) == 2048
        # no byte holds two tokens
        owner = {}
        for b, t in zip(byte.ravel().tolist(), u.ravel().tolist()):
            assert owner.setdefault(b, t) == t


def test_block_round_trip():
    r = np.random.default_rng(2)
    kc, vc = r.integers(0, 16, (2, 64, 128)).astype(np.uint8)
    ks, vs = r.random((2, 64, 2)).astype(np.float16)
    got = paged.unpack_block(paged.pack_block(kc, ks, vc, vs))
    for a, b in zip(got, (kc, ks, vc, vs)):
        assert np.array_equal(a, b)


def test_quantiser_on_crafted_rows():
    x = np.zeros((1, 128))
    x[0, :64] = np.linspace(-7.5, 7.5, 64)
    x[0, 64] = 1e9  # above what the largest scale reaches
    c, s, _ = paged.quantise(x)
    assert s[0, 0] == 1.0 and c[0, 0] == 0 and c[0, 63] == 15
    assert s[0, 1] == np.float16(65504.0) and c[0, 64] == 15 and c[0, 65] == 8
    c, s, _ = paged.quantise(np.zeros((1, 128)))
    assert (s == 0).all() and (c == 8).all() and (paged.levels(c, s) == 0).all()
    x = np.full((1, 128), 0.5)
    x[0, 0], x[0, 64] = 7.5, 7.5
    x[0, 1:4] = [-1.0, 0.0, 1.0]  # decision points belong to the upper bin
    c, s, _ = paged.quantise(x)
    assert c[0, 1:4].tolist() == [7, 8, 9]


@pytest.mark.parametrize("seed", range(4))
def test_levels_are_the_nearest_ones(seed):
    x = paged.to_rotated(np.random.default_rng(seed).standard_normal((5, 128)))
    c, s, _ = paged.quantise(x)
    err = np.abs(paged.levels(c, s) - x).reshape(5, 2, 64)
    assert (err <= 0.5 * s.astype(np.float64)[..., None] * (1 + 2.0 ** -6)).all()
    y = paged.from_rotated(paged.levels(c, s))
    assert np.linalg.norm(y - paged.from_rotated(x)) < 0.15 * np.linalg.norm(x)


def test_attend_against_brute_force():
    r = np.random.default_rng(3)
    k, v, q = r.standard_normal((20, 128)), r.standard_normal((20, 128)), r.standard_normal(128)
    for p, window, sinks, want in ((9, 4, 2, [0, 1, 6, 7, 8, 9]), (9, -1, 0, list(range(10))), (9, 0, 3, [0, 1, 2]),
                                   (25, 4, 0, []), (22, 4, 0, [19]), (1, 4, 8, [0, 1]), (9, 0, 0, [])):
        got = paged.attend(q, k, v, p, window, sinks, 0.1)[0]
        e = [np.exp(0.1 * float(q @ k[j])) for j in want]
        ref = sum((w * v[j] for w, j in zip(e, want)), np.zeros(128)) / sum(e) if want else np.zeros(128)
        assert np.allclose(got, ref, atol=1e-12)
