"""Pins of the oracle's norms, gathered weights and eviction (CPU)."""

import math

import numpy as np
import pytest

import oracle


def test_rms_norm_by_hand():
    # mean square of (3, 4) is 12.5
    np.testing.assert_allclose(oracle.rms_norm([3.0, 4.0], [2.0, 0.5], 0.0),
                               [6 / math.sqrt(12.5), 2 / math.sqrt(12.5)], rtol=1e-15)
    np.testing.assert_array_equal(oracle.rms_norm([3.0, 4.0], None, 1.0), [3.0, 4.0])
    assert np.all(oracle.rms_norm(np.zeros(5), np.ones(5), 1e-6) == 0)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 64))
    n = oracle.rms_norm(x, np.ones(64), 0.0)
    np.testing.assert_allclose((n * n).mean(-1), 1.0, rtol=1e-14)
    np.testing.assert_allclose(oracle.rms_norm(7 * x, np.ones(64), 0.0), n, rtol=1e-14)


def test_norm_rope_splits_the_row():
    rng = np.random.default_rng(1)
    H, dn, dr, dc, T = 3, 4, 6, 10, 5
    y = rng.standard_normal((T, H * (dn + dr) + dc + dr))
    wq, wc, wk = rng.standard_normal(dn + dr), rng.standard_normal(dc), rng.standard_normal(dr)
    pos = np.array([0, 1, 7, 1000, 131071])
    q, ckr = oracle.norm_rope(y, H, dn, dr, dc, wq, wc, wk, 1e-6, pos)
    for t in range(T):
        for h in range(H):
            x = y[t, h * 10:(h + 1) * 10]
            n = [v / math.sqrt(sum(u * u for u in x) / 10 + 1e-6) * g for v, g in zip(x, wq)]
            np.testing.assert_allclose(q[t, h, :dn], n[:dn], rtol=1e-13)
            for k in range(dr // 2):
                z = complex(n[dn + 2 * k], n[dn + 2 * k + 1])
                a = float(pos[t]) * 10000.0 ** (-2 * k / dr)
                z *= complex(math.cos(a), math.sin(a))
                np.testing.assert_allclose(q[t, h, dn + 2 * k:dn + 2 * k + 2], [z.real, z.imag],
                                           atol=1e-9)
        np.testing.assert_allclose(ckr[t, :dc], oracle.rms_norm(y[t, 30:40], wc, 1e-6), rtol=1e-13)
    np.testing.assert_allclose(ckr[0, dc:], oracle.rms_norm(y[0, 40:], wk, 1e-6), rtol=1e-13)


def test_attention_weights_of_a_true_softmax_sum_to_its_rows():
    rng = np.random.default_rng(2)
    S_q, H, L, dc, dr = 3, 4, 9, 6, 2
    q, rows = rng.standard_normal((S_q, H, dc + dr)), rng.standard_normal((L, dc + dr))
    att = oracle.latent_attention(q, rows[:, :dc], rows[:, dc:], 0.3)
    w = oracle.attention_weights(q, rows, att["lse"], 0.3)
    assert w.sum() == pytest.approx(S_q * H, rel=1e-13)
    # the last token is seen by the last query alone
    s = 0.3 * q[-1] @ rows[-1]
    assert w[-1] == pytest.approx(np.exp(s - att["lse"][-1]).sum(), rel=1e-13)
    # a query that saw nothing gives nothing
    lse = att["lse"].copy()
    lse[1] = -np.inf
    assert oracle.attention_weights(q, rows, lse, 0.3).sum() == pytest.approx(2 * H, rel=1e-13)


def test_evict_by_hand():
    # slots      0    1    2    3    4    5    6    7
    w = [9.0, 0.1, 5.0, 0.1, 0.2, 7.0, 0.0, 8.0]
    # one sink, one recent: slots 1..6 are free; 0.0 (6), then the lower 0.1 (1), leave
    assert oracle.evict(w, list(range(8)), 6, 1, 1) == ([(1, 7)], 6)
    # three more than are free: six leave, the two protected stay
    assert oracle.evict(w, list(range(8)), 0, 1, 1) == ([(1, 7)], 2)
    assert oracle.evict(w, list(range(8)), 8, 0, 0) == ([], 8)
    assert oracle.evict(w, list(range(8)), 100, 0, 0) == ([], 8)
    assert oracle.evict([], [], 3, 0, 0) == ([], 0)
    # positions out of slot order: position 7 sits in slot 0 and is recent
    assert oracle.evict([0.0, 1.0, 2.0], [7, 3, 5], 2, 0, 1) == ([(1, 2)], 2)
    nan = float("nan")
    assert oracle.evict([nan, float("inf"), -0.0, 0.0], [0, 1, 2, 3], 1, 0, 0) == ([], 1)
    assert oracle.evict([-0.0, 0.0, nan, 0.0], [0, 1, 2, 3], 3, 0, 0) == ([(0, 3)], 3)


def test_dims_copy_and_pickle_after_their_first_call():
    import copy
    import pickle

    from mla_latent_kv_35_b200 import binding, build
    build.build()
    d = binding.MLADims(8, 128, 512, 64, 128, 256, 64, 0.1, 10000.0, "bf16")
    size = binding.mla_chunk_attention_workspace_size(d, 2, 8, 4)
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d))):
        assert e == d
        assert binding.mla_chunk_attention_workspace_size(e, 2, 8, 4) == size


@pytest.mark.parametrize("seed", range(20))
def test_evict_keeps_the_heaviest_and_moves_the_fewest(seed):
    rng = np.random.default_rng(seed)
    L = int(rng.integers(1, 60))
    w = rng.integers(0, 6, L).astype(float)          # many ties
    pos = rng.permutation(L * 2)[:L]
    budget, ns, nr = int(rng.integers(0, L + 3)), int(rng.integers(0, 4)), int(rng.integers(0, 6))
    pairs, new = oracle.evict(w, list(pos), budget, ns, nr)
    slots = list(range(new))
    for to, frm in pairs:
        assert to < new <= frm < L
        slots[to] = frm
    kept = set(slots)
    assert len(kept) == new
    end = pos.max() + 1
    prot = {t for t in range(L) if pos[t] < ns or pos[t] >= end - nr}
    assert prot <= kept
    gone = set(range(L)) - kept
    assert new == budget or budget >= L or kept == prot
    for g in gone:
        for k in kept - prot:
            assert (w[g], g) < (w[k], k)
    # a kept slot before the end never moves
    assert all(slots[t] == t for t in range(new) if t not in {a for a, _ in pairs})
