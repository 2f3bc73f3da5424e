"""Pins of the fp64 oracle of the passes around attention: invariants, differences, brute force."""
import numpy as np
import pytest

from oracle import attention_fp64 as ora
from oracle import operators_fp64 as ops


def rope_case(seed=0, B=2, H=3, N=5, d=16, rd=8, axes=2):
    g = np.random.default_rng(seed)
    x, w = g.standard_normal((B, H, N, d)), 1 + 0.2 * g.standard_normal(d)
    pos = g.integers(0, 1000, (axes, B, N))
    freq = 10000.0 ** (-2 * np.arange(rd // 2) / rd)
    return x, w, pos, freq, ((1, rd // 2 - 1) if axes == 2 else (rd // 2,))


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_scores_depend_on_the_distance(inter):
    x, _, _, freq, _ = rope_case(rd=16)
    y = ops.norm_rope(x, None, np.full((1, 2, 5), 77), freq, (8,), inter, 1e-6)
    assert np.allclose((y**2).sum(-1), (x**2).sum(-1), rtol=1e-13)
    # <R_m a, R_n b> depends on m - n alone
    a, b = x[:1, :1, :1], x[1:, :1, :1]
    dots = []
    for m, n in ((10, 3), (1010, 1003)):
        ra = ops.norm_rope(a, None, np.full((1, 1, 1), m), freq, (8,), inter, 1e-6)
        rb = ops.norm_rope(b, None, np.full((1, 1, 1), n), freq, (8,), inter, 1e-6)
        dots.append((ra * rb).sum())
    assert abs(dots[0] - dots[1]) < 1e-10


def test_norm_and_axes():
    x, w, pos, freq, sec = rope_case()
    y = ops.norm_rope(x, np.ones(16), np.zeros((2, 2, 5), int), freq, sec, False, 1e-12)
    assert np.allclose((y**2).mean(-1), 1.0)
    # a pair of the first section follows axis 0 only
    a = ops.norm_rope(x, w, pos, freq, sec, False, 1e-6)
    moved = pos.copy()
    moved[1] += 5
    b = ops.norm_rope(x, w, moved, freq, sec, False, 1e-6)
    assert np.array_equal(a[..., [0, 4]], b[..., [0, 4]]) and not np.allclose(a[..., [1, 5]], b[..., [1, 5]])
    assert np.array_equal(a[..., 8:], b[..., 8:])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradients_by_differences(inter):
    x, w, pos, freq, sec = rope_case(seed=3)
    g = np.random.default_rng(9)
    dy = g.standard_normal(x.shape)
    dx, dw = ops.norm_rope_bwd(dy, x, w, pos, freq, sec, inter, 1e-3)

    def f(x, w):
        return (ops.norm_rope(x, w, pos, freq, sec, inter, 1e-3) * dy).sum()

    for _ in range(20):
        i, j = tuple(g.integers(0, n) for n in x.shape), g.integers(0, 16)
        e, u = np.zeros_like(x), np.zeros_like(w)
        e[i], u[j] = 1e-6, 1e-6
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-6 - dx[i]) < 1e-7
        assert abs((f(x, w + u) - f(x, w - u)) / 2e-6 - dw[j]) < 1e-6
    assert np.allclose(ops.norm_rope_bwd(dy, x, None, pos, freq, sec, inter, 1e-3)[0],
                       ops._turn(dy, -ops._angles(pos, freq, sec), inter))


def cache(R=3, Hkv=2, d=8, bs=4, maxb=5, seed=1):
    g = np.random.default_rng(seed)
    blocks = R * maxb + 6
    table = g.permutation(blocks)
    kc, vc = g.standard_normal((2, blocks, Hkv, bs, d))
    return kc, vc, table[: R * maxb].reshape(R, maxb), table[R * maxb :], g


def test_shared_prefix_equals_one_table():
    kc, vc, table, extra, g = cache()
    q = g.standard_normal((3, 4, 8))
    ctx = np.array([8, 4, 0])
    o, lse = ops.decode_shared(q, kc, vc, extra[:3], 12, table, ctx, 4, 0.3)
    joined = np.concatenate([np.tile(extra[:3], (3, 1)), table], 1)  # 12 tokens fill three blocks
    O, L = ora.paged_decode(q, kc, vc, joined, ctx + 12, 4, 0.3)
    assert np.allclose(o, O, atol=1e-13) and np.allclose(lse, L, atol=1e-13)
    o, lse = ops.decode_shared(q, kc, vc, extra[:3], 0, table, ctx, 4, 0.3)
    assert (o[2] == 0).all() and (lse[2] == -np.inf).all()


def test_scored_weights_sum_to_the_heads_and_leave_the_rest():
    kc, vc, table, _, g = cache()
    q, w0 = g.standard_normal((3, 6, 8)), g.random((3, 2, 20))
    ctx = np.array([20, 7, 0])
    o, lse, w = ops.decode_scored(q, kc, vc, table, ctx, w0, 4, 0.3)
    O, L = ora.paged_decode(q[:2], kc, vc, table[:2], ctx[:2], 4, 0.3)
    assert np.allclose(o[:2], O) and np.allclose(lse[:2], L)
    assert np.allclose((w - w0).sum(-1), [[3, 3], [3, 3], [0, 0]])
    assert np.array_equal(w[1, :, 7:], w0[1, :, 7:])


def test_eviction_keeps_the_recent_and_the_heavy():
    kc, vc, table, _, g = cache()
    ctx, seq, keep, recent = np.array([18, 9, 5]), np.array([30, 9, 5]), 8, 3
    w = np.where(np.arange(20) < ctx[:, None, None], g.random((3, 2, 20)), 0.0)
    sp = np.full((3, 2, 20), -1)
    sp[0, :, :10] = [g.permutation(22)[:10] for _ in range(2)]  # of positions below 30 - (18 - 10)
    k2, v2, n2, w2, p2 = ops.evict(kc, vc, table, ctx, seq, w, sp, keep, recent, 4)
    assert n2.tolist() == [8, 8, 5]
    for r in range(3):
        for h in range(2):
            old = [sp[r, h, s] if sp[r, h, s] >= 0 else seq[r] - ctx[r] + s for s in range(ctx[r])]
            rows = {p: (ora.depage(kc, table[r], ctx[r], h, 4)[s], w[r, h, s]) for s, p in enumerate(old)}
            kept = p2[r, h, : n2[r]].tolist()
            now = ora.depage(k2, table[r], n2[r], h, 4)
            assert len(set(kept)) == n2[r] and set(range(seq[r] - min(recent, ctx[r]), seq[r])) <= set(kept)
            for i, p in enumerate(kept):  # every kept position carries its own row and weight
                assert np.array_equal(rows[p][0], now[i]) and rows[p][1] == w2[r, h, i]
            dropped = [rows[p][1] for p in rows if p not in kept]
            heavy = [rows[p][1] for p in kept if p < seq[r] - recent]
            assert not dropped or not heavy or max(dropped) <= min(heavy)
            assert (p2[r, h, n2[r] :] == -1).all() and (w2[r, h, n2[r] :] == 0).all()
    # a second call with nothing appended changes nothing
    again = ops.evict(k2, v2, table, n2, seq, w2, p2, keep, recent, 4)
    assert all(np.array_equal(a, b) for a, b in zip(again, (k2, v2, n2, w2, p2)))


def test_turn_by_hand():
    """A quarter turn takes (1, 0) to (0, 1) and (0, 1) to (-1, 0); where the pair lies is all that differs."""
    for inter, pair in ((False, (1, 5)), (True, (2, 3))):  # pair 1 of a rotary width of 8
        x = np.zeros((1, 1, 2, 10))
        x[0, 0, 0, pair[0]], x[0, 0, 1, pair[1]], x[..., 9] = 1, 1, 7
        freq = np.array([0.1, np.pi / 6, 0.2, 0.3])
        y = ops.norm_rope(x, None, np.full((1, 1, 2), 3), freq, (4,), inter, 1e-6)
        want = np.zeros_like(x)
        want[0, 0, 0, pair[1]], want[0, 0, 1, pair[0]], want[..., 9] = 1, -1, 7
        assert np.allclose(y, want, atol=1e-15)


def test_append_is_the_norm_then_one_cache_write_a_token():
    kc, vc, table, _, g = cache(d=16)
    q, k, v = g.standard_normal((3, 4, 3, 16)), *g.standard_normal((2, 3, 2, 3, 16))
    w, pos, freq = 1 + 0.1 * g.standard_normal((2, 16)), g.integers(0, 99, (1, 3, 3)), 0.3 ** np.arange(8)
    ctx, ql, out = np.array([20, 6, 4]), np.array([3, 2, 0]), np.full(q.shape, 9.0)
    Q, K, V = ops.norm_rope_append(q, k, v, *w, pos, freq, (8,), False, 1e-6, kc, vc, table, ctx, ql, out, 4)
    qn, kn = (ops.norm_rope(x, u, pos, freq, (8,), False, 1e-6) for x, u in zip((q, k), w))
    k2, v2 = kc, vc
    for r in range(3):
        for i in range(ql[r]):
            k2, v2 = ora.paged_append(k2, v2, table[r : r + 1], ctx[r : r + 1] - ql[r] + i, kn[r : r + 1, :, i],
                                      v[r : r + 1, :, i], 4)
        assert np.array_equal(Q[r, :, : ql[r]], qn[r, :, : ql[r]]) and (Q[r, :, ql[r] :] == 9).all()
    assert np.array_equal(K, k2) and np.array_equal(V, v2)


def test_attention_after_an_eviction_is_that_of_the_kept_tokens():
    kc, vc, table, _, g = cache()
    ctx, w, sp = np.array([18, 9, 5]), g.random((3, 2, 20)), np.full((3, 2, 20), -1)
    k2, v2, n2, _, p2 = ops.evict(kc, vc, table, ctx, ctx, w, sp, 8, 3, 4)
    q = g.standard_normal((3, 2, 8))
    o, lse = ora.paged_decode(q, k2, v2, table, n2, 4, 0.3)
    for r in range(3):
        for h in range(2):
            kept = sorted(p2[r, h, : n2[r]])  # in their old order; a first eviction: positions are slots
            k, v = (ora.depage(c, table[r], ctx[r], h, 4)[kept] for c in (kc, vc))
            s = 0.3 * k @ q[r, h]
            p = np.exp(s - s.max())
            assert np.allclose(o[r, h], p @ v / p.sum()) and np.isclose(lse[r, h], np.log(p.sum()) + s.max())
