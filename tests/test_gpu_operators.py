"""GPU parity of tree_qk_norm_rope, tree_attention_scored and tree_accept_sample
against float64 references, at the sizes and masks where they can go wrong, and
a run of the three together with kv_commit_realign."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_04_b200 as tv
import workloads as W
from gpu_helpers import dev, gpu_accept, gpu_mask, i32
from operator_helpers import attention_ref, attention_tolerance, parents, rope_tolerance

pytestmark = pytest.mark.gpu


def _poison(t):
    if t is not None:
        t.view(torch.uint8).fill_(0xFF)
    return t


# ----------------------------------------------------------------------------- norms and rotation

def _norm_case(B, M, Hq, Hkv, D, lens, seed, pad=0, slots=None, left=True, S_extra=3):
    rng = np.random.default_rng(seed)
    g = W.torch_generator(seed, dev())
    lens = np.broadcast_to(np.asarray(lens, np.int32), (B,)).copy()
    S_cap = int(lens.max()) + M + 1 + S_extra
    NS = B if slots is None else max(slots) + 2
    ks, kl = np.zeros(NS, np.int32), np.zeros(NS, np.int32)
    rows = np.arange(B) if slots is None else np.asarray(slots)
    ks[rows] = (lens.max() - lens) if left else 0
    kl[rows] = lens
    par = parents(B, M, 9, rng)
    wide = W.randn_bf16((B, M + 1, (Hq + 2 * Hkv) * D + pad), g, dev())
    qkv = wide[..., :(Hq + 2 * Hkv) * D].unflatten(-1, (Hq + 2 * Hkv, D))
    k, v = (W.randn_bf16((NS, Hkv, S_cap, D), g, dev()) for _ in range(2))
    wq, wk = (W.randn_bf16((D,), g, dev()) for _ in range(2))
    return qkv, wq, wk, k, v, ks, kl, par


@pytest.mark.parametrize(
    "B,M,Hq,Hkv,D,R,lens,pad,slots,offset,weights",
    [
        (1, 0, 4, 4, 64, 64, 0, 0, None, 0.0, "qk"),  # one token, no prefix
        (1, 0, 32, 8, 128, 128, 2000, 0, None, 0.0, "qk"),
        (2, 16, 6, 2, 128, 64, [5, 40], 8, None, 1.0, "qk"),  # half rotated, padded rows, weights around zero
        (3, 5, 8, 1, 64, 16, [0, 1, 33], 64, [4, 0, 2], 0.0, "q"),  # pool slots, no key weight
        (1, 255, 2, 1, 64, 0, 7, 0, None, 0.0, ""),  # the largest tree, no rotation, no weights
        (2, 3, 14, 2, 128, 112, 100000, 0, None, 0.0, "k"),  # far positions, R not a power of two
        (2, 2, 5, 5, 64, 48, 9, 24, [1, 3], 0.5, "qk"),
    ],
)
def test_qk_norm_rope(orc, B, M, Hq, Hkv, D, R, lens, pad, slots, offset, weights):
    qkv, wq, wk, k, v, ks, kl, par = _norm_case(B, M, Hq, Hkv, D, lens, 31 * B + M, pad, slots)
    wq, wk = wq if "q" in weights else None, wk if "k" in weights else None
    _, anc, depth, status = gpu_mask(par, 1000)
    qo = torch.full((B, M + 1, Hq, D), 77.0, dtype=torch.bfloat16, device=dev())
    k2, v2 = k.clone(), v.clone()
    tv.tree_qk_norm_rope(qkv, wq, wk, qo, k2, v2, i32(ks), i32(kl), depth, eps=1e-5, weight_offset=offset,
                         rope_theta=5e5, rotary_dim=R, slot=None if slots is None else i32(slots))
    torch.cuda.synchronize()
    bits = lambda t: None if t is None else W.bf16_bits(t.contiguous())  # noqa: E731
    # the cache of the oracle: only the columns around the step's rows differ, so keep it small
    c0 = max(0, min(int(x) + int(y) for x, y in zip(ks, kl) if y or not np.any(kl)) - 2) if np.max(kl) > 1000 else 0
    rq, rk, rv, qmag, kmag = orc.tree_qk_norm_rope(
        bits(qkv), bits(wq), bits(wk), offset, 1e-5, bits(k[:, :, c0:]), bits(v[:, :, c0:]), ks - c0 if c0 else ks, kl,
        depth.cpu().numpy(), Hq, Hkv, R, 5e5, slots) if not c0 else _shifted(orc, bits, qkv, wq, wk, offset, k, v, ks,
                                                                            kl, depth, Hq, Hkv, R, slots, c0)
    got = qo.double().cpu().numpy()
    assert (np.abs(got - rq) <= rope_tolerance(rq, qmag)).all()
    gk, gv = k2[:, :, c0:].double().cpu().numpy(), v2[:, :, c0:].double().cpu().numpy()
    assert (np.abs(gk - rk) <= np.where(kmag > 0, rope_tolerance(rk, kmag), 0.0)).all()  # other cells untouched
    np.testing.assert_array_equal(gv, rv)
    assert torch.equal(k2[:, :, :c0], k[:, :, :c0]) and torch.equal(v2[:, :, :c0], v[:, :, :c0])


def _shifted(orc, bits, qkv, wq, wk, offset, k, v, ks, kl, depth, Hq, Hkv, R, slots, c0):
    """The oracle on the cache's last columns: the prefix is cut by c0 columns, and c0 is added to the depths, so that
    positions stay as they are."""
    assert (ks + kl >= c0).all()
    kl2, ks2 = np.minimum(kl, ks + kl - c0), np.maximum(ks - c0, 0)
    # columns kv_start + kv_len shift by c0, positions by kl - kl2
    assert ((ks2 + kl2) == ks + kl - c0).all()
    rows = np.arange(depth.shape[0]) if slots is None else np.asarray(slots)
    dep = depth.cpu().numpy() + (kl - kl2)[rows][:, None]
    return orc.tree_qk_norm_rope(bits(qkv), bits(wq), bits(wk), offset, 1e-5, bits(k[:, :, c0:]), bits(v[:, :, c0:]),
                                 ks2, kl2, dep, Hq, Hkv, R, 5e5, slots)


def test_qk_norm_rope_bad_sequences_are_untouched():
    qkv, wq, wk, k, v, ks, kl, par = _norm_case(4, 3, 4, 2, 64, [9, 9, 9, 9], 5, slots=[0, 9, 2, 3])
    kl[2], ks[3] = -1, 10  # a slot outside the pool (below), a negative length, a range behind the cache's end
    _, anc, depth, status = gpu_mask(par, 1000)
    qo = torch.full((4, 4, 4, 64), 77.0, dtype=torch.bfloat16, device=dev())
    k2, v2 = k.clone()[:9], v.clone()[:9]
    tv.tree_qk_norm_rope(qkv, wq, wk, qo, k2, v2, i32(ks[:9]), i32(kl[:9]), depth, slot=i32([0, 9, 2, 3]))
    assert bool((qo[1:] == 77.0).all()) and not bool((qo[0] == 77.0).any())
    assert torch.equal(k2[1:], k[1:9]) and torch.equal(v2[1:], v[1:9])
    changed = (k2[0] != k[0]).any(-1).any(0).nonzero().flatten().tolist()
    assert changed and set(changed) <= set(range(int(ks[0] + kl[0]), int(ks[0] + kl[0]) + 4))


# ----------------------------------------------------------------------------- scored attention

def _attn_case(B, M, Hq, Hkv, D, lens, seed, left=True, slots=None, q_sigma=2.0, tree="uniform", slack=5):
    rng = np.random.default_rng(seed)
    g = W.torch_generator(seed, dev())
    lens = np.broadcast_to(np.asarray(lens, np.int32), (B,)).copy()
    S_cap = int(lens.max()) + M + 1 + slack
    NS = B if slots is None else max(slots) + 2
    ks, kl = np.zeros(NS, np.int32), np.zeros(NS, np.int32)
    rows = np.arange(B) if slots is None else np.asarray(slots)
    ks[rows] = (lens.max() - lens) if left else 0
    kl[rows] = lens
    par = parents(B, M, 9, rng, tree)
    q = W.randn_bf16((B, M + 1, Hq, D), g, dev()) * q_sigma
    k, v = (W.randn_bf16((NS, Hkv, S_cap, D), g, dev()) for _ in range(2))
    # whatever lies behind the step's rows and before the sequence is not used
    for s in range(NS):
        end = int(ks[s] + kl[s]) + M + 1
        k[s, :, end:], v[s, :, end:] = math.nan, math.inf
        k[s, :, :int(ks[s])], v[s, :, :int(ks[s])] = math.nan, math.nan
    return q, k, v, ks, kl, par


def _attend(q, k, v, ks, kl, par, status_override=None, slots=None, softcap=0.0, window=0, slopes=None, scale=None,
            stream=None):
    B, n, Hq, D = q.shape
    _, anc, depth, status = gpu_mask(par, 1000)
    if status_override is not None:
        status.copy_(i32(status_override))
    out = torch.full_like(q, math.nan)
    ws = _poison(tv.attention_scored_workspace(B, n - 1, Hq, k.shape[1], D, k.shape[2], window, q.device))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    tv.tree_attention_scored(q, k, v, i32(ks), i32(kl), anc, depth, status, out, ws, scale=scale, softcap=softcap,
                             window=window, alibi_slopes=slopes, slot=None if slots is None else i32(slots),
                             stream=stream)
    torch.cuda.synchronize()
    return out, status


def _check_attn(out, q, k, v, ks, kl, par, status=None, slots=None, **kw):
    st = np.zeros(q.shape[0], np.int32) if status is None else status
    ref, mean = attention_ref(q, k, v, ks, kl, par, st, slots=slots, **kw)
    err = (out.double() - ref).abs()
    bad = ~(err <= attention_tolerance(ref, mean))
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), float(err.nan_to_num(99).max()))


def _slopes(Hq):
    return (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().to(dev())


SHAPES = [
    (1, 0, 4, 4, 64, 0, None),  # one token, no prefix
    (1, 0, 2, 1, 128, 1, None),
    (1, 16, 4, 4, 64, 128, None),  # tiny
    (2, 5, 8, 2, 128, [0, 63], None),
    (3, 9, 6, 3, 64, [1, 100, 333], [3, 0, 5]),  # ragged, odd group, pool slots
    (2, 33, 8, 1, 128, [500, 127], None),  # two mask words, three query tiles
    (1, 255, 2, 1, 128, 200, None),  # the largest tree
    (4, 20, 12, 4, 128, [64, 65, 127, 129], None),  # tile edges
    (2, 85, 6, 2, 64, [70, 300], None),  # 258 query rows: a third tile of two rows
    (3, 0, 16, 2, 128, [3000, 1, 1777], None),  # split key ranges
    (2, 16, 14, 2, 64, [2500, 4097], [1, 0]),
]


@pytest.mark.parametrize("B,M,Hq,Hkv,D,lens,slots", SHAPES)
@pytest.mark.parametrize("softcap,window,bias", [(0.0, 0, False), (50.0, 0, False), (20.0, 40, False), (100.0, 0, False),
                                                 (0.0, 3, True), (0.0, 0, True), (30.0, 1000, True), (0.5, 7, False)])
def test_attention_scored(B, M, Hq, Hkv, D, lens, slots, softcap, window, bias):
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, D, lens, 100 * B + M, slots=slots)
    kw = dict(softcap=softcap, window=window, slopes=_slopes(Hq) if bias else None)
    out, status = _attend(q, k, v, ks, kl, par, slots=slots, **kw)
    assert int(status.abs().sum()) == 0
    _check_attn(out, q, k, v, ks, kl, par, slots=slots, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap,scale", [(5.0, 1.0), (30.0, 3.0), (58.0, 0.7), (200.0, 2.0)])
def test_attention_scored_saturating_scores(D, softcap, scale):
    """Scores far beyond the cap in both directions (a row whose scores are all near -cap included)."""
    q, k, v, ks, kl, par = _attn_case(2, 7, 8, 2, D, [300, 77], 9)
    k[:, :, :, 0].nan_to_num_(0.0)
    q[0, 3] = 0
    q[0, 3, :, 0] = 8.0
    k[0, :, int(ks[0]):int(ks[0] + kl[0]) + 8, 0] = -40.0  # row 3 of sequence 0: every score far below -cap
    kw = dict(softcap=softcap, scale=scale)
    out, _ = _attend(q, k, v, ks, kl, par, **kw)
    _check_attn(out, q, k, v, ks, kl, par, **kw)


@pytest.mark.parametrize("softcap", [0.0, 50.0])
@pytest.mark.parametrize("slope", [3.0, 1e-3, -0.05])
def test_attention_scored_steep_and_rising_bias(softcap, slope):
    q, k, v, ks, kl, par = _attn_case(1, 12, 4, 2, 128, 2000, 4)
    kw = dict(softcap=softcap, slopes=torch.full((4,), slope, device=dev()))
    out, _ = _attend(q, k, v, ks, kl, par, **kw)
    _check_attn(out, q, k, v, ks, kl, par, **kw)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_attention_scored_growing_maximum(softcap):
    """Scores that rise along the keys: the running maximum moves in every tile."""
    q, k, v, ks, kl, par = _attn_case(1, 4, 4, 1, 128, 1500, 6)
    ramp = torch.linspace(0, 1, 1500, device=dev()).to(torch.bfloat16)
    k[0, 0, int(ks[0]):int(ks[0]) + 1500] = ramp[:, None] * q[0, 0, 0].sign()
    out, _ = _attend(q, k, v, ks, kl, par, softcap=softcap, scale=0.5)
    _check_attn(out, q, k, v, ks, kl, par, softcap=softcap, scale=0.5)


def test_attention_scored_prefix_before_the_window_is_not_used():
    q, k, v, ks, kl, par = _attn_case(2, 5, 4, 2, 128, [900, 300], 12)
    for b in range(2):
        first = int(ks[b] + kl[b]) - 64 + 1
        k[b, :, :first], v[b, :, :first] = math.nan, math.inf
    out, _ = _attend(q, k, v, ks, kl, par, window=64, softcap=50.0)
    _check_attn(out, q, k, v, ks, kl, par, window=64, softcap=50.0)


def test_attention_scored_invalid_sequences_give_zero_rows():
    q, k, v, ks, kl, par = _attn_case(5, 4, 4, 2, 128, [300, 200, 100, 50, 700], 13)
    kl[1] = -5
    ks[2] = 100000
    out, status = _attend(q, k, v, ks, kl, par, status_override=[0, 0, 0, 4, 0], softcap=50.0, slots=[0, 1, 2, 3, 9])
    assert not bool(out[1:].float().abs().sum())
    _check_attn(out[:1], q[:1], k, v, ks, kl, par[:1], softcap=50.0)
    assert status.tolist() == [0, 0, 0, 4, tv.SEQ_BAD_GEOMETRY]


def test_attention_scored_large_batch_and_trees():
    """More units than CTAs that fit at once, ragged lengths, two to five query tiles a unit."""
    rng = np.random.default_rng(7)
    for B, M, Hq, Hkv, lens in ((24, 63, 32, 4, rng.integers(1, 900, 24)), (40, 2, 32, 16, rng.integers(1, 400, 40)),
                                (6, 128, 16, 4, rng.integers(100, 3000, 6))):
        q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, 128, lens, 17)
        out, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
        _check_attn(out, q, k, v, ks, kl, par, softcap=50.0)


@pytest.mark.parametrize("B,M,Hq,Hkv,D,lens,failed", [
    (3, 0, 8, 1, 128, [6000, 1, 2500], ()),                     # pieces of rows of very different lengths
    (5, 7, 8, 2, 64, [3000, 64, 65, 127, 800], (2,)),            # few rows: 32, and keys that end inside a chunk
    (2, 32, 2, 2, 128, [5000, 4100], ()),                        # one row more than few
    (120, 0, 12, 1, 128, [i * 13 % 1300 for i in range(120)], (3,)),        # few rows, shares by cost
    (9, 3, 32, 8, 64, [4000, 0, 977, 955, 2880, 1, 79, 80, 3999], (4,)),   # pieces or shares; an invalid row between
    (50, 1, 16, 4, 64, [1000 + 37 * i % 900 for i in range(50)], (0, 49)),  # more rows than CTAs, one query tile
    (30, 23, 64, 4, 128, [(i * 331) % 1500 for i in range(30)], (7,)),      # three query tiles: pairs and lone ones
    (40, 16, 20, 1, 64, [0] * 20 + [2400] + [5] * 19, ()),     # one long row among rows of one tile
    (300, 2, 2, 1, 64, [i % 3 * 40 for i in range(300)], (5,)),             # rows too short to cut
])
def test_attention_scored_rows_cut_between_ctas(B, M, Hq, Hkv, D, lens, failed):
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, D, lens, 5 + B)
    status = [4 if b in failed else 0 for b in range(B)]
    for kw in (dict(softcap=30.0), dict(slopes=_slopes(Hq)), dict(window=1100)):
        out, _ = _attend(q, k, v, ks, kl, par, status_override=status, **kw)
        _check_attn(out, q, k, v, ks, kl, par, status=status, **kw)
        again, _ = _attend(q, k, v, ks, kl, par, status_override=status, **kw)
        assert torch.equal(out, again)


def test_attention_scored_repeats_exactly_and_on_another_stream():
    q, k, v, ks, kl, par = _attn_case(2, 16, 8, 2, 128, [4000, 2500], 21)
    a, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    b, _ = _attend(q, k, v, ks, kl, par, softcap=50.0, stream=torch.cuda.Stream())
    assert torch.equal(a, b)


# ----------------------------------------------------------------------------- sampled acceptance

def _sample(logits, u, T, par, draft, max_depth, k=None, p=None, m=None, status_override=None, ws=None):
    B, n, V = logits.shape
    parg, anc, depth, status = gpu_mask(par, max_depth)
    if status_override is not None:
        status.copy_(i32(status_override))
    f = lambda a: None if a is None else torch.as_tensor(np.asarray(a, np.float32), device=dev())  # noqa: E731
    tok = torch.full((B, n), -7, dtype=torch.int32, device=dev())
    lp = torch.full((B, n), math.nan, device=dev())
    al, bonus = (torch.full((B,), -7, dtype=torch.int32, device=dev()) for _ in range(2))
    path = torch.full((B, max_depth + 1), -7, dtype=torch.int32, device=dev())
    ws = _poison(tv.accept_sample_workspace(B, n - 1, V, dev())) if ws is None else ws
    tv.tree_accept_sample(logits, f(u), f(T), i32(draft), parg, depth, anc, status, max_depth, tok, al, path, bonus,
                          ws, top_k=None if k is None else i32(k), top_p=f(p), min_p=f(m), logprob=lp)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (tok, lp, al, path, bonus)] + [status]


def _check_sample(orc, logits, u, T, par, draft, max_depth, k=None, p=None, m=None, status=None, got=None):
    B = logits.shape[0]
    got = _sample(logits, u, T, par, draft, max_depth, k, p, m, status) if got is None else got
    as32 = lambda a: None if a is None else np.asarray(a, np.float32)  # noqa: E731
    ref = orc.tree_accept_sample(logits.float().cpu().numpy(), as32(u), as32(T), draft, par,
                                 np.zeros(B, np.int32) if status is None else np.asarray(status), max_depth, k, as32(p),
                                 as32(m))
    np.testing.assert_array_equal(got[0], ref[0])
    # fp32 rounding of the logarithm, and weights good to 2^-40
    fin = np.isfinite(ref[1])
    assert (np.isfinite(got[1]) == fin).all()
    assert (np.abs(got[1][fin] - ref[1][fin]) <= 2.0 ** -24 * np.abs(ref[1][fin]) + 2.0 ** -36).all()
    for a, b in zip(got[2:5], ref[2:5]):
        np.testing.assert_array_equal(a, b)


def _sample_case(B, M, V, seed, bf16=False, pad=0, sigma=2.0, offset=0):
    rng = np.random.default_rng(seed)
    par = parents(B, M, 9, rng)
    x = rng.normal(0, sigma, (B, M + 1, V))
    for _ in range(min(20, V)):
        np.put_along_axis(x, rng.integers(0, V, (B, M + 1, 1)), rng.random((B, M + 1, 1)) * 6 * sigma, 2)
    full = torch.zeros(offset + B * (M + 1) * (V + pad), dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    view = full[offset:].view(B, M + 1, V + pad)[..., :V]
    view.copy_(torch.as_tensor(x))
    u = rng.random((B, M + 1)).astype(np.float32)
    top = view.float().argmax(-1).cpu().numpy()
    draft = rng.integers(0, V, (B, M + 1)).astype(np.int32)
    for b in range(B):
        for i in range(1, M + 1):
            if rng.random() < 0.7:
                draft[b, i] = top[b, par[b, i]]
    return view, u, par, draft, rng


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,M,V,pad,offset", [(1, 0, 1, 0, 0), (2, 3, 2, 0, 0), (1, 7, 31, 1, 1), (3, 5, 1000, 0, 0),
                                              (2, 16, 1024, 8, 0), (2, 4, 4097, 3, 3), (1, 2, 32000, 0, 1),
                                              (8, 0, 20011, 5, 0), (1, 0, 262144, 0, 0)])
def test_accept_sample(orc, B, M, V, pad, offset, bf16):
    x, u, par, draft, rng = _sample_case(B, M, V, 7 * V + M, bf16, pad, offset=offset)
    T = 0.4 + rng.random(B)
    for k, p, m in ((None, None, None), ([1 + V // 3] * B, None, None), ([40] * B, None, None),
                    (None, [0.9] * B, None), (None, None, [0.05] * B), ([300] * B, [0.95] * B, [0.001] * B),
                    (None, [0.5] * B, [0.2] * B)):
        _check_sample(orc, x, u, T, par, draft, 9, k, p, m)


def test_accept_sample_settings_of_each_sequence(orc):
    B = 12
    x, u, par, draft, rng = _sample_case(B, 6, 9000, 3)
    T = np.array([0, 1, 0.7, 1.5, 1e-30, 1e30, np.inf, np.nan, -1, 1, 1, 1], np.float32)
    k = np.array([0, 5, 0, -3, 7, 9, 4, 0, 0, 9001, 1, 2 ** 31 - 1], np.int32)
    p = np.array([1, 0.8, 0.5, np.nan, 0.9, 2, 0.7, 0.1, 1, 0.0, 1, -1], np.float32)
    m = np.array([0, 0, 0.1, 0.02, np.nan, 0.5, 0, 0, 2, 0, 5, -1], np.float32)
    _check_sample(orc, x, u, T, par, draft, 9, k, p, m)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [5000, 140000])
def test_accept_sample_ties_and_flat_rows(orc, V, bf16):
    """Few distinct logits: every boundary falls among equal ones, and far more tokens are kept than fit a short list."""
    rng = np.random.default_rng(11)
    B, M = 2, 2
    par = parents(B, M, 9, rng)
    x = torch.as_tensor(rng.integers(-2, 3, (B, M + 1, V)).astype(np.float32), device=dev())
    x = x.to(torch.bfloat16) if bf16 else x
    u = rng.random((B, M + 1)).astype(np.float32)
    u[0, 0], u[0, 1] = 0.0, 1.0 - 2.0 ** -24
    draft = rng.integers(0, V, (B, M + 1)).astype(np.int32)
    for k, p, m in ((None, None, None), ([V // 2 + 1, 3], None, None), (None, [0.93, 0.2], None),
                    (None, None, [math.exp(-1.0 / 0.8) * 1.01, 1e-3]), ([V - 1, V // 10], [0.999, 0.4], None)):
        _check_sample(orc, x, u, [0.8, 1.3], par, draft, 9, k, p, m)


def test_accept_sample_infinities_and_nan(orc):
    rng = np.random.default_rng(12)
    B, M, V = 7, 1, 3000
    par = parents(B, M, 9, rng)
    x = rng.normal(size=(B, M + 1, V)).astype(np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 0, 5:2000:7] = np.inf
    x[3, :, ::2] = np.nan
    x[4] = -np.inf
    x[4, :, 2999] = -3e38
    x[5, 1] = -np.inf
    x[6, :, ::3], x[6, :, 1::3] = 0.0, -0.0
    u = rng.random((B, M + 1)).astype(np.float32)
    draft = np.zeros((B, M + 1), np.int32)
    draft[4, 1] = 2999
    draft[5, 1] = -1
    lx = torch.as_tensor(x, device=dev())
    for k, p, m in ((None, None, None), ([10] * B, [0.9] * B, None), (None, [0.6] * B, [0.3] * B)):
        _check_sample(orc, lx, u, [1.0] * B, par, draft, 9, k, p, m)
    _check_sample(orc, lx, u, [0.0] * B, par, draft, 9)


def test_accept_sample_status_and_greedy_like_tree_accept(orc):
    x, u, par, draft, rng = _sample_case(4, 9, 700, 8)
    _check_sample(orc, x, u, [1.0] * 4, par, draft, 9, status=[0, 4, 8, 0])
    got = _sample(x, u, [0.0] * 4, par, draft, 9)
    parg, anc, depth, status = gpu_mask(par, 9)
    ref = gpu_accept(x.contiguous(), draft, parg, depth, anc, status, 9)
    for a, b in zip((got[0], got[2], got[3], got[4]), ref):
        np.testing.assert_array_equal(a, b.cpu().numpy())


def test_accept_sample_many_rows(orc):
    x, u, par, draft, rng = _sample_case(12, 63, 3001, 14, True, 1)
    T = 0.3 + rng.random(12)
    _check_sample(orc, x, u, T, par, draft, 9, rng.integers(0, 90, 12), 0.5 + 0.6 * rng.random(12),
                  0.2 * rng.random(12) - 0.1)


# ----------------------------------------------------------------------------- together

def _teacher(seed, B=3, M=9, Hq=8, Hkv=2, D=64, V=3000, L=2, prefix=(150, 40, 97), window=(0, 60)):
    """A TreeVerifier of a teacher with normalised heads, capped scores, a local layer and sampled decoding, its
    packed projections and weights."""
    from tree_speculative_decoding_04_b200.verifier import TreeVerifier

    rng = np.random.default_rng(seed)
    g = W.torch_generator(seed, dev())
    S_cap = max(prefix) + 3 * (M + 1) + 8
    ver = TreeVerifier(B, M, Hq, Hkv, D, V, L, S_cap, max_depth=6, softcap=30.0, window=window, sampling=True)
    for layer in range(L):
        ver.k[layer].copy_(W.randn_bf16((B, Hkv, S_cap, D), g, dev()))
        ver.v[layer].copy_(W.randn_bf16((B, Hkv, S_cap, D), g, dev()))
    ver.kv_len.copy_(i32(np.array(prefix[:B])))
    ver.temperature.copy_(torch.tensor([0.8, 0.0, 1.2][:B]))
    ver.top_k.copy_(i32([0, 0, 50][:B]))
    ver.top_p.copy_(torch.tensor([0.9, 1.0, 0.95][:B]))
    wq, wk = (W.randn_bf16((D,), g, dev()) * 0.2 for _ in range(2))
    qkv = [W.randn_bf16((B, M + 1, Hq + 2 * Hkv, D), g, dev()) for _ in range(L)]
    return ver, qkv, wq, wk, rng


def _new_inputs(ver, qkv, rng, g):
    par = parents(ver.B, ver.M, 6, rng)
    ver.parent.copy_(i32(par))
    logits = torch.as_tensor(rng.normal(0, 2, ver.logits.shape).astype(np.float32))
    ver.logits.copy_(logits)
    top = logits.argmax(-1).numpy()
    draft = np.take_along_axis(top, par, 1).astype(np.int32)
    draft[:, ::4] = rng.integers(0, ver.V, draft[:, ::4].shape)
    ver.draft.copy_(i32(draft))
    ver.uniform.copy_(torch.as_tensor(rng.random((ver.B, ver.n)).astype(np.float32)))
    for t in qkv:
        t.copy_(W.randn_bf16(tuple(t.shape), g, dev()))
    return par, draft


def _step(ver, qkv, wq, wk):
    ver.build_mask()
    for layer in range(ver.L):
        ver.norm_rope(layer, qkv[layer], wq, wk, eps=1e-6, weight_offset=1.0, rope_theta=1e4, rotary_dim=ver.D // 2)
        ver.attention(layer)
    ver.accept()
    ver.commit()


def test_a_step_of_the_three_operators(orc):
    """norm_rope -> attention of a capped and of a local layer -> sampled acceptance -> commit, each against its
    reference on what the one before it left; two steps, so that the second works on the committed cache."""
    ver, qkv, wq, wk, rng = _teacher(1)
    g = W.torch_generator(2, dev())
    for _ in range(2):
        par, draft = _new_inputs(ver, qkv, rng, g)
        ks, kl = ver.kv_start.cpu().numpy(), ver.kv_len.cpu().numpy()
        before = [(k.clone(), v.clone()) for k, v in zip(ver.k, ver.v)]
        ver.build_mask()
        for layer in range(ver.L):
            ver.norm_rope(layer, qkv[layer], wq, wk, eps=1e-6, weight_offset=1.0, rope_theta=1e4, rotary_dim=32)
            ver.attention(layer)
            rq, rk, rv, qmag, kmag = orc.tree_qk_norm_rope(
                W.bf16_bits(qkv[layer]), W.bf16_bits(wq), W.bf16_bits(wk), 1.0, 1e-6, W.bf16_bits(before[layer][0]),
                W.bf16_bits(before[layer][1]), ks, kl, ver.depth.cpu().numpy(), ver.Hq, ver.Hkv, 32, 1e4)
            assert (np.abs(ver.q[layer].double().cpu().numpy() - rq) <= rope_tolerance(rq, qmag)).all()
            gk = ver.k[layer].double().cpu().numpy()
            assert (np.abs(gk - rk) <= np.where(kmag > 0, rope_tolerance(rk, kmag), 0.0)).all()
            np.testing.assert_array_equal(ver.v[layer].double().cpu().numpy(), rv)
            _check_attn(ver.out[layer], ver.q[layer], ver.k[layer], ver.v[layer], ks, kl, par, softcap=30.0,
                        window=ver.window[layer])
        ver.accept()
        torch.cuda.synchronize()
        got = [t.cpu().numpy() for t in (ver.argmax, ver.logprob, ver.accept_len, ver.path, ver.bonus)]
        _check_sample(orc, ver.logits, ver.uniform.cpu().numpy(), ver.temperature.cpu().numpy(), par, draft, 6,
                      ver.top_k.cpu().numpy(), ver.top_p.cpu().numpy(), ver.min_p.cpu().numpy(), got=got)
        ver.commit()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(ver.kv_len.cpu().numpy(), kl + 1 + got[2])


def test_a_captured_step_replays_on_new_inputs():
    ver, qkv, wq, wk, rng = _teacher(3)
    twin, qkv2, wq2, wk2, _ = _teacher(3)
    g = W.torch_generator(4, dev())
    _new_inputs(ver, qkv, rng, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in (*ver.k, *ver.v, ver.kv_len)]
    with torch.cuda.stream(side):
        _step(ver, qkv, wq, wk)  # warm-up
    torch.cuda.synchronize()
    for t, o in zip((*ver.k, *ver.v, ver.kv_len), keep):
        t.copy_(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(ver, qkv, wq, wk)
    for _ in range(3):
        _new_inputs(ver, qkv, rng, g)
        for a, b in ((twin.parent, ver.parent), (twin.logits, ver.logits), (twin.draft, ver.draft),
                     (twin.uniform, ver.uniform), *zip(qkv2, qkv)):
            a.copy_(b)
        graph.replay()
        _step(twin, qkv2, wq2, wk2)
        torch.cuda.synchronize()
        for a, b in ((ver.argmax, twin.argmax), (ver.path, twin.path), (ver.bonus, twin.bonus), (ver.kv_len, twin.kv_len),
                     (ver.logprob, twin.logprob), *zip(ver.out, twin.out), *zip(ver.k, twin.k), *zip(ver.v, twin.v)):
            assert torch.equal(a, b)


def test_step_from_host_with_a_sampling_teacher():
    from tree_speculative_decoding_04_b200.verifier import TreeVerifier

    rng = np.random.default_rng(6)
    a, b = (TreeVerifier(2, 5, 4, 2, 64, 500, 2, 120, 5, softcap=50.0, sampling=True) for _ in range(2))
    for ver in (a, b):
        ver.kv_len.copy_(i32([60, 33]))
        ver.top_k.fill_(20)
    h = a.pinned_inputs()
    par = parents(2, 5, 5, rng)
    h["parent"].copy_(torch.as_tensor(par))
    h["draft"].copy_(torch.as_tensor(rng.integers(0, 500, (2, 6)).astype(np.int32)))
    h["logits"].copy_(torch.as_tensor(rng.normal(size=(2, 6, 500)).astype(np.float32)))
    h["uniform"].copy_(torch.as_tensor(rng.random((2, 6)).astype(np.float32)))
    for name in ("q", "tree_k", "tree_v"):
        h[name].copy_(torch.as_tensor(rng.normal(size=tuple(h[name].shape))).to(torch.bfloat16))
    a.step_from_host()
    for name in ("parent", "draft", "logits", "tree_k", "tree_v"):
        getattr(b, name).copy_(h[name])
    b.uniform.copy_(h["uniform"])
    for layer in range(2):
        b.q[layer].copy_(h["q"][layer])
        b.write_tree_rows(layer)
    b.step()
    torch.cuda.synchronize()
    for x, y in ((a.argmax, b.argmax), (a.accept_len, b.accept_len), (a.path, b.path), *zip(a.out, b.out), *zip(a.k, b.k)):
        assert torch.equal(x, y)
    assert torch.equal(h["bonus"], b.bonus.cpu()) and a.h2d_bytes() == sum(
        h[k].numel() * h[k].element_size() for k in ("parent", "draft", "logits", "uniform", "q", "tree_k", "tree_v"))


def test_two_calls_at_once_on_two_streams():
    """Two attention and two sampling calls in flight together, each with a workspace of its own."""
    q, k, v, ks, kl, par = _attn_case(2, 16, 8, 2, 128, [4000, 2500], 31)
    ref, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    x, u, spar, draft, rng = _sample_case(4, 5, 30000, 32)
    sref = _sample(x, u, [1.0] * 4, spar, draft, 9, p=[0.9] * 4)
    _, anc, depth, status = gpu_mask(par, 1000)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.empty_like(q) for _ in streams], []
    ks, kl = i32(ks), i32(kl)
    torch.cuda.synchronize()
    for s, out in zip(streams, outs):
        wss.append(tv.attention_scored_workspace(2, 16, 8, 2, 128, k.shape[2], 0, q.device))
        for _ in range(5):
            tv.tree_attention_scored(q, k, v, ks, kl, anc, depth, status, out, wss[-1], softcap=50.0, stream=s)
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(_sample(x, u, [1.0] * 4, spar, draft, 9, p=[0.9] * 4))
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, ref)
    for g in got:
        for a, b in zip(g[:5], sref[:5]):
            np.testing.assert_array_equal(a, b)


def test_attention_scored_workspace_is_needed_where_ranges_split():
    q, k, v, ks, kl, par = _attn_case(1, 0, 4, 2, 64, 3000, 33)
    _, anc, depth, status = gpu_mask(par, 10)
    need = tv.attention_scored_workspace_size(1, 0, 4, 2, 64, k.shape[2], 0)
    assert need > 0 and tv.attention_scored_workspace_size(1, 0, 4, 2, 64, k.shape[2], 64) == 0
    for ws in (None, torch.empty(need - 16, dtype=torch.uint8, device=dev())):
        with pytest.raises(tv.TVError, match="INVALID_ARG"):
            tv.tree_attention_scored(q, k, v, i32(ks), i32(kl), anc, depth, status, torch.empty_like(q), ws)


def test_attention_scored_wait_limit():
    """Waits that give up at once: every sequence is either flagged, with rows that are zero or right, or right."""
    q, k, v, ks, kl, par = _attn_case(3, 40, 8, 2, 128, [2000, 900, 50], 34)
    ref, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    tv.set_wait_limit_ns(1)
    try:
        out, status = _attend(q, k, v, ks, kl, par, softcap=50.0)
    finally:
        tv.set_wait_limit_ns(0)
    for b in range(3):
        assert int(status[b]) in (0, tv.SEQ_TIMEOUT)
        same, zero = (out[b] == ref[b]).all(-1), (out[b] == 0).all(-1)
        assert bool((same | zero).all()) if int(status[b]) else bool(same.all())
    again, status = _attend(q, k, v, ks, kl, par, softcap=50.0)
    assert torch.equal(again, ref) and int(status.abs().sum()) == 0


@pytest.mark.parametrize("M,Hq,lens", [(0, 32, [3431, 583, 935, 3652, 609, 1846, 579, 3760]),
                                       (0, 32, [1431, 583, 935, 1652, 609, 1846, 579, 760]), (16, 64, [3000, 1500, 700]),
                                       (40, 16, [2500, 90])])
def test_attention_scored_thousands_of_launches(M, Hq, lens):
    """Lone and paired query tiles over split ranges, queued thousands deep: one answer, no sequence flagged.  (The
    two pipes of a lone tile run apart by as much as the ring of key tiles allows.)"""
    B = len(lens)
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, 8 if M == 0 else 2, 128, lens, 77)
    ref, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    _check_attn(ref, q, k, v, ks, kl, par, softcap=50.0)
    _, anc, depth, status = gpu_mask(par, 1000)
    ks, kl = i32(ks), i32(kl)
    ws = tv.attention_scored_workspace(B, M, Hq, k.shape[1], 128, k.shape[2], 0, q.device)
    out = torch.empty_like(q)
    for _ in range(6):
        for _ in range(3000):
            tv.tree_attention_scored(q, k, v, ks, kl, anc, depth, status, out, ws, softcap=50.0)
        assert int(status.abs().sum()) == 0 and torch.equal(out, ref)
