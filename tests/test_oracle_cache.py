"""The cache operators' oracle pinned on the CPU against other code: dense
softmax matrices, the decode oracle with the drafted path put into the cache,
brute force and invariants."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle import cache as OC
from oracle import decode as OD
from oracle import layouts as OL

PATS = [(OL.BAND_GLOBAL, 1, dict(window=1, global_first=1)), (OL.DYADIC, 1, dict(window=0, global_first=0, dyadic_kmin=1)),
        (OL.RANDOM, 4, dict(density=0.3, seed=5))]


@pytest.mark.parametrize("kind,L,pat", PATS)
def test_prompt_weights_are_column_sums_of_the_dense_softmax(kind, L, pat):
    n, B, H, G, d = 70, 8, 4, 2, 4
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((H, n, d)), rng.standard_normal((G, n, d)), rng.standard_normal((G, n, d))
    sets = OL.kept_sets(kind, n, B, L, **pat)
    _, lse = OA.forward_sparse(q, k, v, sets, B, 0.5)
    got = OC.prompt_weights(q, k, lse, sets, B, 0.5)
    want = np.zeros((G, n))
    for f in range(H):
        s = np.where(OA.token_mask(sets[f % L], n, B), 0.5 * q[f] @ k[f // 2].T, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        want[f // 2] += (e / e.sum(1, keepdims=True)).sum(0)
    np.testing.assert_allclose(got, want, rtol=1e-12)
    assert got.sum() == pytest.approx(H * n)           # every row gives one in all


@pytest.mark.parametrize("kind,L,pat", PATS)
def test_tree_rows_are_decode_steps_with_the_path_in_the_cache(kind, L, pat):
    n, B, batch, H, G, d, T = 64, 8, 2, 4, 2, 4, 12
    rng = np.random.default_rng(1)
    sets = OL.kept_sets(kind, n, B, L, **pat)
    k, v = rng.standard_normal((batch * G, n, d)), rng.standard_normal((batch * G, n, d))
    order = rng.permutation(batch * 8)
    lengths = [29, 47]
    par = np.array([[-1, 0, 1, 2, 3, 4, 5, 1, 7, -1, 9, 10], [-1, -1, 0, 1, 2, 2, 5, 6, 7, 8, -2, -2]])
    q = rng.standard_normal((batch * H, T, d))
    kt, vt = rng.standard_normal((batch * G, T, d)), rng.standard_normal((batch * G, T, d))
    kc, vc, table = OD.pages_from_sequences(k, v, batch, B, order)
    o, lse = OC.tree(q, kt, vt, kc, vc, table, lengths, par, sets, B, 0.7)
    for b in range(batch):
        for i in range(T):
            if par[b, i] == -2:
                assert np.isnan(lse[b * H:(b + 1) * H, i]).all()
                continue
            path, x = [], i
            while x != -1:
                path.append(x)
                x = par[b, x]
            k2, v2 = k.copy(), v.copy()
            for e, x in enumerate(reversed(path)):
                k2[b * G:(b + 1) * G, lengths[b] + e] = kt[b * G:(b + 1) * G, x]
                v2[b * G:(b + 1) * G, lengths[b] + e] = vt[b * G:(b + 1) * G, x]
            kc2, vc2, _ = OD.pages_from_sequences(k2, v2, batch, B, order)
            pos = [lengths[b] + len(path) - 1] * batch
            o2, lse2 = OD.decode_step(q[:, i], kc2, vc2, table, pos, sets, B, 0.7)
            np.testing.assert_allclose(o[b * H:(b + 1) * H, i], o2[b * H:(b + 1) * H], rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(lse[b * H:(b + 1) * H, i], lse2[b * H:(b + 1) * H], rtol=1e-12)


def test_step_weights_sum_to_one_per_query_row_and_match_the_last_prompt_row():
    n, B, H, G, d = 40, 8, 4, 2, 4
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((H, n, d)), rng.standard_normal((G, n, d)), rng.standard_normal((G, n, d))
    sets = OL.kept_sets(OL.RANDOM, n, B, 2, density=0.4, seed=3)
    kc, vc, table = OD.pages_from_sequences(k, v, 1, B, rng.permutation(5))
    t = 37
    o, lse = OD.decode_step(q[:, t], kc, vc, table, [t], sets, B, 0.5)
    w = OC.step_weights(q[:, t], kc, table, [t], lse, sets, B, 0.5, n)
    assert w.sum() == pytest.approx(H)
    full = np.full((H, n), -np.inf)
    full[:, t] = lse
    np.testing.assert_allclose(w, OC.prompt_weights(q, k, full, sets, B, 0.5), rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (7, 3), (19, 19), (20, 4), (50, 0)])
def test_evict_keeps_the_right_tokens_and_moves_them_whole(ids, budget, recent):
    n, B, batch, G, d = 40, 8, 3, 2, 4
    rng = np.random.default_rng(4)
    kc, vc = rng.standard_normal((batch * 5, G, B, d)), rng.standard_normal((batch * 5, G, B, d))
    table = rng.permutation(batch * 5).reshape(batch, 5)
    w = np.round(np.exp(rng.standard_normal((batch * G, n))), 1).astype(np.float32)     # with ties
    w[0, :6] = np.nan
    tok = np.stack([rng.permutation(n) * 3 for _ in range(batch * G)]) if ids else None
    lengths = [40, 20, 0]
    kc2, vc2, w2, t2, l2 = OC.evict(kc, vc, table, lengths, w, tok, n, budget, recent)

    def read(c, r, length):
        return np.stack([c[table[r // G][s // B], r % G, s % B] for s in range(length)]) if length else np.zeros((0, d))

    for r in range(batch * G):
        length, kept = lengths[r // G], min(lengths[r // G], budget)
        assert l2[r // G] == kept
        was = tok[r] if ids else np.arange(n)
        by_token = {int(was[s]): s for s in range(length)}
        # each kept slot holds one of the sequence's tokens, whole, at most once
        held = t2[r, :kept].tolist()
        assert len(set(held)) == kept and set(held) <= set(by_token)
        src = [by_token[t] for t in held]
        np.testing.assert_array_equal(read(kc2, r, kept), read(kc, r, length)[src])
        np.testing.assert_array_equal(read(vc2, r, kept), read(vc, r, length)[src])
        np.testing.assert_array_equal(w2[r, :kept], w[r, src])
        # nothing left out would have come before something kept
        new = max(by_token) if by_token else -1
        rank = [(was[s] > new - recent, np.inf if was[s] > new - recent else (-np.inf if np.isnan(w[r, s]) else w[r, s]),
                 -s) for s in range(length)]
        out = [rank[s] for s in range(length) if s not in src]
        assert not out or min(rank[s] for s in src) > max(out)
        # a kept token below the new length has not moved
        assert all(s == x for x, s in enumerate(src) if x in src)
        np.testing.assert_array_equal(t2[r, kept:], new + 1 + np.arange(n - kept))
        assert (w2[r, kept:] == 0).all()


def test_planted_mistakes_are_seen():
    """A tree oracle that let a sibling in, or a cut that took the highest slot at a tie, would differ."""
    n, B, d = 32, 8, 4
    rng = np.random.default_rng(6)
    sets = OL.kept_sets(OL.BAND_GLOBAL, n, B, 1, window=4, global_first=0)
    kc, vc = rng.standard_normal((4, 1, B, d)), rng.standard_normal((4, 1, B, d))
    table = np.arange(4)[None]
    q, kt, vt = (rng.standard_normal((1, 3, d)) for _ in range(3))
    a = OC.tree(q, kt, vt, kc, vc, table, [9], [[-1, 0, 0]], sets, B, 1.0)[0]
    b = OC.tree(q, kt, vt, kc, vc, table, [9], [[-1, 0, 1]], sets, B, 1.0)[0]
    np.testing.assert_array_equal(a[:, :2], b[:, :2])
    assert np.abs(a[:, 2] - b[:, 2]).max() > 1e-3
    w = np.array([[1.0, 5.0, 1.0, 1.0]], dtype=np.float32)
    t2 = OC.evict(kc, vc, table, [4], w, None, 4, 2, 0)[3]
    assert t2[0, :2].tolist() == [0, 1]
