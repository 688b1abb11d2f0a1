"""Pins of the cache calls' oracle: torch's softmax in float64, hand cases, and the rotation's own laws (CPU)."""
import numpy as np
import pytest
import torch

from oracle import cache as oc


def _batch(rng, chunks, cached, page, hkv, D):
    need = [-(-(t + c) // page) for t, c in zip(chunks, cached)]
    table = np.full((len(chunks), max(need) + 1), -1, dtype=np.int32)
    order = rng.permutation(sum(need) + 2)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    offs = np.concatenate([[0], np.cumsum(np.array(chunks) - 1)]).astype(np.int32)
    pages = rng.normal(size=(2, sum(need) + 2, page, hkv, D))
    return table, offs, pages[0], pages[1]


@pytest.mark.parametrize("window", [0, 1, 4])
def test_attend_matches_dense_softmax(window):
    rng = np.random.default_rng(1)
    chunks, cached, page, hkv, G, D = [3, 1, 5], [0, 7, 10], 8, 2, 3, 16
    table, offs, k, v = _batch(rng, chunks, cached, page, hkv, D)
    q = rng.normal(size=(sum(chunks), hkv * G, D))
    out, lse, mean, big, _ = oc.attend(q, k, v, table, offs, None, cached, 0.3, window)
    r = 0
    for b, (T, c) in enumerate(zip(chunks, cached)):
        slot = np.arange(c + T)
        K = torch.from_numpy(k[table[b][slot // page], slot % page])
        V = torch.from_numpy(v[table[b][slot // page], slot % page])
        for j in range(T):
            lo = max(0, c + j - window + 1) if window else 0
            for g in range(hkv * G):
                z = 0.3 * (K[lo:c + j + 1, g // G] @ torch.from_numpy(q[r + j, g]))
                w = torch.softmax(z, 0)
                # a sum of n rounded products is off by at most n 2^-53 sum |w v|, on either side
                assert (abs(out[r + j, g] - (w @ V[lo:c + j + 1, g // G]).numpy()) <= 1e-13 * mean[r + j, g]).all()
                np.testing.assert_allclose(lse[r + j, g], torch.logsumexp(z, 0).item(), rtol=1e-12)
                assert (mean[r + j, g] >= np.abs(out[r + j, g]) - 1e-12).all() and big[r + j, g] >= abs(z).max()
        r += T


def test_tree_masks_by_hand():
    # node 1 and 2 under the root, 3 under 1, 4 under 3, 5 under 2
    par = [0, 0, 1, 3, 2]
    assert oc.depths(par).tolist() == [0, 1, 1, 2, 3, 2]
    assert oc.lineage(par)[4].tolist() == [True, True, False, True, True, False]
    assert oc.lineage(par)[5].tolist() == [True, False, True, False, False, True]
    # a chain of parents is the causal triangle
    assert np.array_equal(oc.lineage([0, 1, 2]), np.tril(np.ones((4, 4), dtype=bool)))


def test_tree_path_attends_like_the_chain_of_its_nodes():
    rng = np.random.default_rng(2)
    par, page, D = [0, 0, 1, 3, 2], 8, 8
    table, offs, k, v = _batch(rng, [6], [5], page, 1, D)
    q = rng.normal(size=(6, 1, D))
    out, lse, mean, *_ = oc.attend(q, k, v, table, offs, np.array(par), [5], 0.5)
    slot = np.array([0, 1, 2, 3, 4, 5, 6, 8, 9])  # the cached tokens, then nodes 0, 1, 3, 4
    K, V = k[table[0][slot // page], slot % page, 0], v[table[0][slot // page], slot % page, 0]
    w = torch.softmax(torch.from_numpy(0.5 * K @ q[4, 0]), 0).numpy()
    assert (abs(out[4, 0] - w @ V) <= 1e-13 * mean[4, 0]).all()


def test_masked_places_are_not_read_and_empty_rows_are_zero():
    rng = np.random.default_rng(3)
    table, offs, k, v = _batch(rng, [2], [9], 8, 1, 8)
    want = oc.attend(np.ones((2, 1, 8)), k, v, table, offs, None, [9], 1.0, window=3)
    k2, v2 = k.copy(), v.copy()
    used = {(int(table[0][s // 8]), s % 8) for s in range(7, 11)}
    for p in range(k.shape[0]):
        for t in range(8):
            if (p, t) not in used:
                k2[p, t] = v2[p, t] = np.nan
    got = oc.attend(np.ones((2, 1, 8)), k2, v2, table, offs, None, [9], 1.0, window=3)
    assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])
    table[:] = -1
    out, lse, *_ = oc.attend(np.ones((2, 1, 8)), k, v, table, offs, None, [9], 1.0)
    assert not out.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_the_distance_only(interleaved):
    rng = np.random.default_rng(4)
    freq = 100.0 ** (-np.arange(4) / 4)
    x, y = rng.normal(size=12), rng.normal(size=12)
    dots = [oc.rotate(x, (p + 3) * freq, interleaved) @ oc.rotate(y, p * freq, interleaved) for p in (0, 5, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    np.testing.assert_allclose(np.linalg.norm(oc.rotate(x, freq, interleaved)), np.linalg.norm(x))
    assert np.array_equal(oc.rotate(x, freq, interleaved)[8:], x[8:])
    one = oc.rotate(np.array([1.0, 0.0]), np.array([np.pi / 2]), interleaved)
    np.testing.assert_allclose(one, [0.0, 1.0], atol=1e-15)


def test_append_places_and_positions():
    q = np.ones((6, 1, 2)); k = np.ones((6, 1, 2))
    par = np.array([0, 0, 1], dtype=np.int32)
    _, kk, slots, seq = oc.append(q, k, None, np.array([0, 3, 4]), np.concatenate([par, [0]]), [10, 2], freq=[0.1])
    assert slots.tolist() == [10, 11, 12, 13, 2, 3] and seq.tolist() == [0, 0, 0, 0, 1, 1]
    ang = [1.0, 1.1, 1.1, 1.2, 0.2, 0.3]
    np.testing.assert_allclose(kk[:, 0, 0], np.cos(ang) - np.sin(ang))


def test_compact_by_hand():
    x = np.arange(2 * 8, dtype=np.float64).reshape(2, 8, 1, 1)
    table = np.array([[1, 0]])
    # cached 6: chunk slots 6 (root), 7, 8, 9, 10; the accepted path is nodes 2, 3, 4
    y, now = oc.compact(x, table, np.array([0, 4]), np.array([6]), np.array([3]), np.array([2, 3, 4, -1]))
    seq = np.concatenate([y[1, :, 0, 0], y[0, :, 0, 0]])
    old = np.concatenate([x[1, :, 0, 0], x[0, :, 0, 0]])
    assert seq[7:10].tolist() == old[8:11].tolist() and seq[:7].tolist() == old[:7].tolist()
    assert seq[10:].tolist() == old[10:].tolist() and now.tolist() == [10]
    y, now = oc.compact(x, table, np.array([0, 4]), np.array([6]), np.array([-1]), np.array([2, 3, 4, -1]))
    assert np.array_equal(x, y) and now.tolist() == [6]
