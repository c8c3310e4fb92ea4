"""Pins of the float64 readings of the per-head norms, the scored attention and
the sampled acceptance: hand-computed cases and identities with the other
oracle functions."""
import math

import numpy as np
import pytest

import workloads as W


def _bf16(orc, x):
    return orc.round_bf16(np.asarray(x, np.float64))


def test_sample_row_by_hand(orc):
    # weights 1, 1/2, 1/4, 1/4 in the order of tokens 2, 0, 1, 3
    l = np.log(np.array([0.5, 0.25, 1.0, 0.25]))
    # vocabulary order 0, 1, 2, 3: inclusive sums 0.5, 0.75, 1.75, 2 (a sum equal to u * S is not above it)
    assert [orc.sample_row(l, u)[0] for u in (0.0, 0.24, 0.26, 0.37, 0.38, 0.87, 0.88, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    tok, lp, kept = orc.sample_row(l, 0.9, top_k=3)  # the tie of 1 and 3 keeps the lower index
    assert kept == [2, 0, 1] and tok == 2 and lp == pytest.approx(math.log(1 / 1.75))
    assert orc.sample_row(l, 0.1, top_p=0.5)[2] == [2]  # nothing is before the first token, 1.0 is before the next
    assert orc.sample_row(l, 0.1, top_p=0.51)[2] == [2, 0]
    assert orc.sample_row(l, 0.1, top_p=0.0)[2] == [2]
    assert orc.sample_row(l, 0.1, min_p=0.4)[2] == [2, 0]
    assert orc.sample_row(l, 0.1, top_k=3, top_p=0.6)[2] == [2, 0]  # 0.6 of the top three's 1.75
    assert orc.sample_row(l, 0.1, T=0.0)[:2] == (2, 0.0)
    assert orc.sample_row(l, 1.0)[0] == 3
    assert orc.sample_row(np.full(4, -np.inf), 0.3)[0] == -1
    assert orc.sample_row(np.array([np.nan, -np.inf, 1.0]), 0.7)[0] == 2
    assert orc.sample_row(np.array([np.inf, 3.0, np.inf]), 0.7)[0] == 2


def test_sample_row_frequencies(orc):
    rng = np.random.default_rng(3)
    l = rng.normal(size=6)
    p = np.exp(l / 0.7)
    p /= p.sum()
    n = 20000
    draws = np.bincount([orc.sample_row(l, (i + 0.5) / n, T=0.7)[0] for i in range(n)], minlength=6) / n
    # a stratified u hits each cell within two strata of its width
    assert np.abs(draws - p).max() <= 2.0 / n


def test_greedy_sampling_is_tree_accept(orc):
    rng = np.random.default_rng(5)
    parent = np.stack([W.tree_uniform_depth(9, 4, rng) for _ in range(3)]).astype(np.int32)
    logits = rng.normal(size=(3, 10, 12)).astype(np.float32)
    draft = rng.integers(0, 12, size=(3, 10)).astype(np.int32)
    top = logits.argmax(-1)
    for b in range(3):
        for i in range(1, 10):
            if rng.random() < 0.7:
                draft[b, i] = top[b, parent[b, i]]
    st = np.zeros(3, np.int32)
    tok, _, al, path, bonus = orc.tree_accept_sample(logits, np.zeros((3, 10)), np.zeros(3), draft, parent, st, 4)
    am, al2, path2, bonus2 = orc.tree_accept(logits, draft, parent, st, 4)
    for a, b in ((tok, am), (al, al2), (path, path2), (bonus, bonus2)):
        np.testing.assert_array_equal(a, b)


def test_scored_attention_without_scores_is_tree_attention(orc):
    rng = np.random.default_rng(6)
    B, M, Hq, Hkv, D, S = 2, 6, 4, 2, 64, 40
    parent = np.stack([W.tree_uniform_depth(M, 3, rng) for _ in range(B)]).astype(np.int32)
    q = _bf16(orc, rng.normal(size=(B, M + 1, Hq, D)))
    k, v = (_bf16(orc, rng.normal(size=(B, Hkv, S, D))) for _ in range(2))
    ks, kl, st = np.array([3, 0]), np.array([20, 0]), np.zeros(B, np.int32)
    got, _ = orc.tree_attention_scored(q, k, v, ks, kl, parent, st, Hkv)
    ref = orc.tree_attention(q, k, v, ks, kl, parent, st, Hkv)
    np.testing.assert_allclose(got, ref, rtol=0, atol=1e-5)  # the C oracle sums in fp32
    wide, _ = orc.tree_attention_scored(q, k, v, ks, kl, parent, st, Hkv, softcap=1e6, window=1000,
                                        slopes=np.zeros(Hq))
    np.testing.assert_allclose(wide, got, atol=1e-9)
    one, _ = orc.tree_attention_scored(q, k, v, ks, kl, parent, st, Hkv, window=1)
    for b in range(B):  # a window of one position leaves each node itself
        c = ks[b] + kl[b]
        own = orc.bf16_to_f64(v)[b, :, c:c + M + 1]
        np.testing.assert_allclose(one[b], np.repeat(own.transpose(1, 0, 2), Hq // Hkv, 1), atol=1e-12)


def test_norm_rope_by_hand(orc):
    D, Hq, Hkv = 64, 1, 1
    x = np.zeros((1, 1, 3, D))
    x[0, 0, 0, 0], x[0, 0, 0, 32] = 3.0, 4.0  # mean square 25 / 64
    x[0, 0, 1, 5] = -2.0
    x[0, 0, 2] = np.arange(D)
    k = np.zeros((1, 1, 8, D), np.uint16)
    w = _bf16(orc, np.full(D, 0.5))
    q, kc, vc, _, _ = orc.tree_qk_norm_rope(_bf16(orc, x), w, None, 1.0, 0.0, k, k, np.array([1]), np.array([2]),
                                            np.array([[0]]), Hq, Hkv, D, 100.0)
    s = 1.5 * 8 / 5
    assert q[0, 0, 0, 0] == pytest.approx(s * (3 * math.cos(2) - 4 * math.sin(2)))
    assert q[0, 0, 0, 32] == pytest.approx(s * (4 * math.cos(2) + 3 * math.sin(2)))
    ang = 2 * 100.0 ** (-10 / 64)
    assert kc[0, 0, 3, 5] == pytest.approx(-8 * math.cos(ang)) and kc[0, 0, 3, 37] == pytest.approx(-8 * math.sin(ang))
    np.testing.assert_array_equal(vc[0, 0, 3], np.arange(D))
    assert not kc[0, 0, [0, 1, 2, 4]].any()
    part, _, _, _, _ = orc.tree_qk_norm_rope(_bf16(orc, x), None, None, 1.0, 0.0, k, k, np.array([1]), np.array([2]),
                                             np.array([[0]]), Hq, Hkv, 0, 100.0)
    assert part[0, 0, 0, 0] == pytest.approx(3 * 8 / 5) and part[0, 0, 0, 32] == pytest.approx(4 * 8 / 5)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=3.0, window=9), dict(slopes=True), dict(slopes=True, window=2, softcap=50.0)])
def test_vectorised_reference_is_the_oracle(orc, kw):
    """The float64 reference of the GPU tests against the oracle's loops."""
    import torch

    from operator_helpers import attention_ref

    rng = np.random.default_rng(8)
    B, M, Hq, Hkv, D, S = 3, 7, 4, 2, 64, 50
    parent = np.stack([W.tree_uniform_depth(M, 4, rng) for _ in range(B)]).astype(np.int32)
    q = _bf16(orc, rng.normal(size=(B, M + 1, Hq, D)))
    k, v = (_bf16(orc, rng.normal(size=(4, Hkv, S, D))) for _ in range(2))
    ks, kl, st, slots = np.array([3, 0, 1, 0]), np.array([20, 0, 41, 50]), np.array([0, 0, 4]), [2, 1, 0]
    if "slopes" in kw:
        kw = dict(kw, slopes=np.array([0.5, 0.1, 0.0, -0.2], np.float32))
    a, am = orc.tree_attention_scored(q, k, v, ks, kl, parent, st, Hkv, slots=slots, **kw)
    t = lambda x: torch.as_tensor(orc.bf16_to_f64(x))  # noqa: E731
    if "slopes" in kw:
        kw["slopes"] = torch.as_tensor(kw["slopes"])
    b, bm = attention_ref(t(q), t(k), t(v), ks, kl, parent, st, slots=slots, **kw)
    np.testing.assert_allclose(a, b.numpy(), atol=1e-12)
    np.testing.assert_allclose(am, bm.numpy(), atol=1e-12)
