"""The block-sparse oracle against closed forms and scalar brute force (no GPU)."""

import math

import numpy as np
import pytest

from oracle import attention, sparse


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,D", [(16, 64), (64, 64), (32, 128)])
def test_rotation_is_a_complex_product(rot, D, interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, D))
    ang = rng.uniform(-9, 9, (5, rot // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = sparse.rotate(x, cs, interleaved)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, rot // 2 + i)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang[:, None, i])
        assert np.allclose(y[..., a], z.real, atol=1e-14) and np.allclose(y[..., b], z.imag, atol=1e-14)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    x32, cs32 = x.astype(np.float32), cs.astype(np.float32)
    err = np.abs(sparse.rotate(x32, cs32, interleaved, np.float32)
                 - sparse.rotate(x32, cs32, interleaved))
    assert (err <= sparse.rotation_error(x32, cs32, interleaved)).all() and err.max() > 0


def test_rotated_logits_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 64))
    freq = 10000.0 ** (-np.arange(32) / 32)

    def at(x, p):
        return sparse.rotate(x, np.concatenate([np.cos(p * freq), np.sin(p * freq)])[None], False)

    z = [float((at(q, p + 17) * at(k, p)).sum()) for p in (0, 5, 1000)]
    assert np.allclose(z, z[0], atol=1e-10)


def _paged(seed, lens, bs, Hkv, D):
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm = rng.permutation(nb)
    tables = np.full((len(lens), max(need + [1])), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    return rng, tables, rng.standard_normal((nb, Hkv, bs, D)), rng.standard_normal((nb, Hkv, bs, D))


@pytest.mark.parametrize("new", [None, [0, 1, 3, 20]])
def test_bounds_by_brute_force(new):
    lens = [0, 5, 16, 23]
    _, tables, k, _ = _paged(3, lens, 8, 2, 4)
    before = np.full((k.shape[0], 2, 2, 4), 7.5)
    got = sparse.key_bounds(before, k, tables, lens, new)
    want = before.copy()
    for s, n in enumerate(lens):
        for lb in range(-(-n // 8)):
            tokens = [t for t in range(lb * 8, min(n, lb * 8 + 8))]
            if new is not None and not any(t >= n - new[s] for t in tokens):
                continue
            for h in range(2):
                for d in range(4):
                    col = [k[tables[s, lb], h, t % 8, d] for t in tokens]
                    want[tables[s, lb], h, 0, d], want[tables[s, lb], h, 1, d] = max(col), min(col)
    assert np.array_equal(got, want)


def test_scores_bound_the_logits_and_selection_keeps_the_best():
    lens = [100, 40, 0, 7]
    rng, tables, k, _ = _paged(4, lens, 8, 2, 16)
    q = rng.standard_normal((4, 6, 16))
    bounds = sparse.key_bounds(np.zeros((k.shape[0], 2, 2, 16)), k, tables, lens)
    score = sparse.block_scores(q[0], bounds, tables[0], 13)
    for h in range(2):
        for b in range(13):
            keys = k[tables[0, b], h, :min(8, 100 - 8 * b)]
            logits = (q[0, 3 * h:3 * h + 3] @ keys.T).sum(0)
            assert (logits <= score[h, b] + 1e-12).all()
            hi, lo = bounds[tables[0, b], h]
            larger = sum(max(q[0, 3 * h + g, d] * hi[d], q[0, 3 * h + g, d] * lo[d])
                         for g in range(3) for d in range(16))
            assert math.isclose(larger, score[h, b], rel_tol=1e-12)
    sel = sparse.select_blocks(q, bounds, tables, lens, 8, 6, 1, 2)
    for h in range(2):
        kept = sel[0, h].tolist()
        assert kept == sorted(kept) and {0, 11, 12} <= set(kept)
        middle = [b for b in kept if b not in (0, 11, 12)]
        worst = min(score[h, b] for b in middle)
        assert all(score[h, b] <= worst for b in range(1, 11) if b not in middle)
    assert sel[1].tolist() == [[0, 1, 2, 3, 4, -1]] * 2
    assert (sel[2] == -1).all() and sel[3].tolist() == [[0] + [-1] * 5] * 2


def test_equal_scores_keep_the_lowest_blocks():
    bounds = np.ones((10, 1, 2, 4))
    q = np.ones((1, 1, 4))
    sel = sparse.select_blocks(q, bounds, np.arange(10)[None], [80], 8, 5, 1, 1)
    assert sel.tolist() == [[[0, 1, 2, 3, 9]]]


def test_attention_over_every_block_is_the_paged_decode():
    lens = [0, 1, 33, 64]
    rng, tables, k, v = _paged(5, lens, 8, 2, 16)
    q = rng.standard_normal((4, 4, 16))
    full = np.full((4, 2, 9), -1, np.int32)
    for s, n in enumerate(lens):
        b = -(-n // 8)
        full[s, :, :b] = rng.permutation(b)
    want = attention.paged_decode(q, k, v, tables, lens, 0.25, 8)
    assert np.allclose(sparse.decode_sparse(q, k, v, tables, lens, full, 0.25), want, atol=1e-13)
    # a block listed twice counts twice
    one = np.array([[[0, 0, 1]]], np.int32)
    twice = sparse.decode_sparse(q[2:3, :2], k[:, :1], v[:, :1], tables[2:3], [16], one, 0.25)
    K, V = (np.concatenate([x[tables[2, b], 0] for b in (0, 0, 1)]) for x in (k, v))
    assert np.allclose(twice[0], attention.attend(q[2, :2], K, V, 0.25), atol=1e-13)


def test_a_nan_score_is_kept_before_an_infinite_one():
    bounds = np.ones((6, 1, 2, 4))
    bounds[1:5, 0, 0, 0] = np.inf
    bounds[4, 0, 1, 1] = np.nan
    sel = sparse.select_blocks(np.ones((1, 1, 4)), bounds, np.arange(6)[None], [48], 8, 2, 0, 0)
    assert sel.tolist() == [[[1, 4]]]
