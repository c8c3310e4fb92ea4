"""GPU tests of the operators where their arithmetic comes to its limits:
temperatures near zero, masked vocabularies, waits that give up, calls in flight
together, many rows, rows of few keys."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_04_b200 as tv
from gpu_helpers import dev, gpu_mask, i32
from operator_helpers import parents
from test_gpu_operators import _attend, _attn_case, _check_attn, _check_sample, _norm_case, _sample, _slopes

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- temperatures and fills

TEMPERATURES = [1e-6, 1e-7, 1e-8, 5e-9, 1e-9, 1e-12, 1e-18, 1e-20, 1e-25, 1e-30, 1e-45, 1e-3]
FILTERS = [(None, None, None), (None, 0.9, None), (None, 0.5, 0.2), (None, None, 0.3), (40, 0.95, None)]


def _filters(B, k, p, m):
    return ([k] * B if k else None), ([p] * B if p else None), ([m] * B if m else None)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("k,p,m", FILTERS)
def test_accept_sample_near_zero_temperature(orc, k, p, m, bf16):
    """Row maxima from 1 to 100 and around zero, alone, with neighbours one float below, and shared by tokens of
    several chunks."""
    rng = np.random.default_rng(21)
    B, M, V = len(TEMPERATURES), 8, 5000
    par = parents(B, M, 9, rng)
    x = rng.normal(0, 2, (B, M + 1, V)).astype(np.float32)
    for r in range(M + 1):
        top = [1.0, 7.3, 24.7, 59.9, 100.0, 0.0, 3e-5, 12.5, 33.3][r]
        if r in (5, 6):
            x[:, r] = -np.abs(x[:, r])
        x[:, r] = np.minimum(x[:, r], np.float32(top) - np.float32(0.5))
        at = rng.permutation(V)[:8]
        x[:, r, at[0]] = top
        if r in (3, 4, 6, 7, 8):
            x[:, r, at[1:5]] = top
        if r in (2, 4, 8):
            x[:, r, at[5:8]] = np.nextafter(np.float32(top), np.float32(0))
    lx = torch.as_tensor(x, device=dev())
    lx = lx.to(torch.bfloat16) if bf16 else lx
    u = rng.random((B, M + 1)).astype(np.float32)
    u[:, 7], u[:, 8] = 0.0, 1.0 - 2.0 ** -24
    draft = lx.float().argmax(-1).cpu().numpy().astype(np.int32)
    draft = np.stack([draft[b, par[b]] for b in range(B)])
    got = _sample(lx, u, TEMPERATURES, par, draft, 9, *_filters(B, k, p, m))
    assert ((got[0] >= 0) & (got[0] < V)).all()
    _check_sample(orc, lx, u, TEMPERATURES, par, draft, 9, *_filters(B, k, p, m), got=got)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1e-3, 1e-8, 1e-20])
def test_accept_sample_near_zero_temperature_of_flat_rows(orc, T, bf16):
    """Thousands of equal maxima: more than a short list holds, and the borders of top-p and top-k among them."""
    rng = np.random.default_rng(22)
    B, M, V = 2, 1, 60000
    par = parents(B, M, 9, rng)
    x = torch.as_tensor(rng.integers(37, 39, (B, M + 1, V)).astype(np.float32), device=dev())
    x = x.to(torch.bfloat16) if bf16 else x
    u = rng.random((B, M + 1)).astype(np.float32)
    draft = np.zeros((B, M + 1), np.int32)
    for k, p, m in ((None, None, None), (None, 0.7, None), (20000, None, None), (20000, 0.3, 0.5)):
        _check_sample(orc, x, u, [T, T], par, draft, 9, *_filters(B, k, p, m))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fill", [-1e4, -1e18, -1e20, -1e25, -1e30, -3.3895314e38])
def test_accept_sample_masked_vocabulary(orc, fill, bf16):
    """Most of the vocabulary holds one large negative number: whole chunks of it, a chunk with one token left, a
    padded end, and a row that holds nothing else."""
    rng = np.random.default_rng(23)
    B, M, V = 10, 3, 6500
    par = parents(B, M, 9, rng)
    x = rng.normal(0, 3, (B, M + 1, V)).astype(np.float32)
    x[:, :, 1024:4096] = fill
    x[:, 1, 3500] = 4.0
    x[:, :, 5100:] = fill
    x[:, 3] = fill
    x[:5, 2, :1024] = fill  # the first live chunk is not the row's first
    lx = torch.as_tensor(x, device=dev())
    lx = lx.to(torch.bfloat16) if bf16 else lx
    u = rng.random((B, M + 1)).astype(np.float32)
    T = np.linspace(0.3, 1.5, B)
    draft = rng.integers(0, 1024, (B, M + 1)).astype(np.int32)
    for k, p, m in FILTERS:
        _check_sample(orc, lx, u, T, par, draft, 9, *_filters(B, k, p, m))


# ----------------------------------------------------------------------------- waits that give up

@pytest.mark.parametrize("B,M,Hq,Hkv,D,lens", [
    (60, 1, 8, 2, 128, [i * 53 % 1300 for i in range(60)]),  # few rows
    (12, 15, 8, 1, 64, [i * 531 % 6000 for i in range(12)]),  # a lone query tile
    (20, 40, 16, 2, 128, [i * 53 % 1900 for i in range(20)]),  # a pair and a lone tile of each kv head
])
def test_attention_scored_short_limits_leave_no_copies_behind(B, M, Hq, Hkv, D, lens):
    """Launches whose waits give up between launches that work in the shared memory they leave: the latter are right."""
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, D, lens, 40)
    ref, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    _check_attn(ref, q, k, v, ks, kl, par, softcap=50.0)
    _, anc, depth, status = gpu_mask(par, 1000)
    ks, kl = i32(ks), i32(kl)
    ws = tv.attention_scored_workspace(B, M, Hq, Hkv, D, k.shape[2], 0, q.device)
    flagged, outs = [], []
    try:
        for limit in (1, 500, 1000, 2000, 3000, 4000):
            for _ in range(25):
                for ns in (limit, 0):
                    tv.set_wait_limit_ns(ns)
                    out, st = torch.full_like(q, 7.0), torch.zeros_like(status)
                    tv.tree_attention_scored(q, k, v, ks, kl, anc, depth, st, out, ws, softcap=50.0)
                    if ns:
                        flagged.append(st)
                    else:
                        outs.append((out, st))
            assert all(torch.equal(out, ref) and int(st.abs().sum()) == 0 for out, st in outs)
            outs.clear()
    finally:
        tv.set_wait_limit_ns(0)
    assert any(int(st.sum()) > 0 for st in flagged)


@pytest.mark.parametrize("B,M,Hq,Hkv,D,lens", [
    (3, 3, 8, 1, 64, [700, 60, 250]),            # few rows, short keys: rows never cut
    (5, 1, 16, 4, 128, [900, 30, 700, 150, 880]),  # few rows, whole ones
    (2, 3, 8, 1, 128, [9000, 5000]),             # few rows, cut between CTAs
    (60, 9, 16, 2, 64, [i * 37 % 700 for i in range(60)]),  # a lone tile of 80 rows, several items to a CTA
    (2, 15, 8, 1, 128, [6000, 3100]),            # a lone tile, cut between CTAs
    (40, 40, 16, 2, 128, [i * 53 % 900 for i in range(40)]),  # a pair and a lone tile of each kv head
])
def test_attention_scored_rows_are_zero_or_complete_after_a_wait_ran_out(B, M, Hq, Hkv, D, lens):
    """Limits from nothing to a step's length, many launches: whichever warp gives up first, a flagged sequence has no
    row that lacks some of its keys, and the others are right."""
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, D, lens, 41)
    ref, _ = _attend(q, k, v, ks, kl, par, softcap=50.0)
    _check_attn(ref, q, k, v, ks, kl, par, softcap=50.0)
    _, anc, depth, clean = gpu_mask(par, 1000)
    ks, kl = i32(ks), i32(kl)
    ws = tv.attention_scored_workspace(B, M, Hq, Hkv, D, k.shape[2], 0, q.device)
    flagged = 0
    try:
        for limit in (1, 300, 1000, 2000, 4000):
            tv.set_wait_limit_ns(limit)
            for _ in range(40):
                out, status = torch.full_like(q, 7.0), torch.zeros_like(clean)
                tv.tree_attention_scored(q, k, v, ks, kl, anc, depth, status, out, ws, softcap=50.0)
                same, zero = (out == ref).all(-1), (out == 0).all(-1)
                assert bool((same | zero).all())
                assert bool(((status == 0) | (status == tv.SEQ_TIMEOUT)).all())
                assert bool(same.flatten(1).all(1)[status == 0].all())
                flagged += int((status != 0).sum())
    finally:
        tv.set_wait_limit_ns(0)
    assert flagged > 0
    out, status = torch.full_like(q, 7.0), torch.zeros_like(clean)
    tv.tree_attention_scored(q, k, v, ks, kl, anc, depth, status, out, ws, softcap=50.0)
    assert torch.equal(out, ref) and int(status.abs().sum()) == 0


# ----------------------------------------------------------------------------- calls in flight together

@pytest.mark.parametrize("bf16", [False, True])
def test_accept_sample_calls_in_flight_together(orc, bf16):
    """Calls queued on two streams with nothing between them, each stream with a workspace and outputs of its own;
    rows of every kind, those with a flat top-p through all launches."""
    rng = np.random.default_rng(51)
    B, M, V = 12, 9, 30000
    par = parents(B, M, 9, rng)
    x = [torch.as_tensor(rng.normal(0, s, (B, M + 1, V)).astype(np.float32), device=dev()) for s in (0.4, 0.7)]
    x = [t.to(torch.bfloat16) if bf16 else t for t in x]
    u = [rng.random((B, M + 1)).astype(np.float32) for _ in x]
    T = np.linspace(0.5, 1.4, B).astype(np.float32)
    k = [0, 0, 0, 40, 0, 0, 9000, 0, 0, 0, 1, 0]
    p = [0.95, 0.9, 1.0, 1.0, 0.99, 0.5, 0.9, 1.0, 0.999, 0.8, 0.3, 0.97]
    m = [0, 0, 0, 0, 0.01, 0, 0, 0.2, 0, 0.05, 0, 0]
    draft = rng.integers(0, V, (B, M + 1)).astype(np.int32)
    ref = [_sample(x[i], u[i], T, par, draft, 9, k, p, m) for i in range(2)]
    for i in range(2):
        _check_sample(orc, x[i], u[i], T, par, draft, 9, k, p, m, got=ref[i])
    parg, anc, depth, _ = gpu_mask(par, 9)
    f32 = lambda a: torch.as_tensor(np.asarray(a, np.float32), device=dev())  # noqa: E731
    settings = [f32(T), i32(k), f32(p), f32(m)]
    streams, calls = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        ws = tv.accept_sample_workspace(B, M, V, dev())
        e = lambda *s: torch.empty(s, dtype=torch.int32, device=dev())  # noqa: E731
        outs = [(e(B, M + 1), torch.empty((B, M + 1), device=dev()), e(B), e(B, 10), e(B)) for _ in range(30)]
        calls.append((ws, f32(u[i]), i32(draft), torch.zeros(B, dtype=torch.int32, device=dev()), outs))
    torch.cuda.synchronize()
    for r in range(30):
        for i, s in enumerate(streams):
            ws, ui, di, st, outs = calls[i]
            tok, lp, al, path, bonus = outs[r]
            tv.tree_accept_sample(x[i], ui, settings[0], di, parg, depth, anc, st, 9, tok, al, path, bonus, ws,
                                  top_k=settings[1], top_p=settings[2], min_p=settings[3], logprob=lp, stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        for outs in calls[i][4]:
            for got, want in zip(outs, ref[i][:5]):
                np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_qk_norm_rope_of_many_rows():
    """More rows than a GPU takes at once (fewer threads to a row), against the same rows a few at a time."""
    B, M, Hq, Hkv, D = 37, 20, 6, 2, 128
    qkv, wq, wk, k, v, ks, kl, par = _norm_case(B, M, Hq, Hkv, D, [7 * b for b in range(B)], 52, pad=8)
    _, anc, depth, status = gpu_mask(par, 1000)
    ks, kl = i32(ks), i32(kl)
    for R in (D, 32):
        got, want = [(torch.full((B, M + 1, Hq, D), 77.0, dtype=torch.bfloat16, device=dev()), k.clone(), v.clone())
                     for _ in range(2)]
        tv.tree_qk_norm_rope(qkv, wq, wk, *got, ks, kl, depth, eps=1e-5, rope_theta=5e5, rotary_dim=R)
        for b in range(B):
            tv.tree_qk_norm_rope(qkv[b:b + 1], wq, wk, want[0][b:b + 1], want[1][b:b + 1], want[2][b:b + 1],
                                 ks[b:b + 1], kl[b:b + 1], depth[b:b + 1], eps=1e-5, rope_theta=5e5, rotary_dim=R)
        for a, c in zip(got, want):
            assert torch.equal(a, c)


# ----------------------------------------------------------------------------- the weights' normaliser

@pytest.mark.parametrize("B,M,Hq,Hkv,D,lens,window", [
    (3, 3, 8, 2, 64, [40, 1, 9], 1),            # few rows, one key to a row
    (2, 40, 16, 2, 128, [300, 77], 1),          # paired tiles, one key to a row
    (4, 0, 4, 4, 128, [0, 1, 2, 3], 0),         # one to four keys
    (2, 20, 12, 2, 64, [3, 30], 0),
    (2, 0, 8, 1, 128, [5000, 70], 0),           # cut between CTAs
])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (20.0, False), (50.0, False), (70.0, False), (0.0, True),
                                          (30.0, True)])
def test_attention_scored_of_equal_values_is_that_value(B, M, Hq, Hkv, D, lens, window, softcap, bias):
    """Every row is a mean of the V rows it reads: with one V row, or equal ones, it is exactly that row.

    The products with the rounded weights are exact, and the fp32 sums of n <= 5001 of them and the normaliser's
    reciprocal are off by less than n 2^-24 + 2^-22 < 2^-11, which does not reach the half step 2^-9 of a bf16 value."""
    q, k, v, ks, kl, par = _attn_case(B, M, Hq, Hkv, D, lens, 61)
    if not window:
        for b in range(B):
            c0, end = int(ks[b]), int(ks[b] + kl[b]) + M + 1
            v[b, :, c0:end] = v[b, :, c0:c0 + 1].clone()
    out, _ = _attend(q, k, v, ks, kl, par, softcap=softcap, window=window, slopes=_slopes(Hq) if bias else None)
    for b in range(B):
        c0 = int(ks[b] + kl[b])
        want = v[b, :, c0:c0 + M + 1].transpose(0, 1).repeat_interleave(Hq // Hkv, 1)  # the row's own key
        assert torch.equal(out[b], want)
