"""Host-side refusals of tree_qk_norm_rope, tree_attention_scored and
tree_accept_sample: bad arguments are turned away before the device is touched."""
import ctypes

import pytest
import torch

import __graft_entry__
import tree_speculative_decoding_04_b200 as tv

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return tv.load()


P = ctypes.c_void_p
d, z = P(256), P(0)  # d is never dereferenced


def _norm(lib, **kw):
    a = dict(qkv=d, stride=8 * 64, wq=d, wk=d, off=0.0, eps=1e-6, q=d, k=d, v=d, S=64, ks=d, kl=d, depth=d, B=1, M=3,
             Hq=4, Hkv=2, D=64, R=64, theta=1e4, slot=z, ns=0, stream=z)
    assert set(kw) <= set(a)
    return lib.tree_qk_norm_rope(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(M=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(S=-1), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(off=float("inf")), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(M=256), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED), (dict(R=72), INVALID),
    (dict(R=24), UNSUPPORTED), (dict(R=-16), INVALID), (dict(theta=1.0), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(stride=8 * 64 - 8), INVALID), (dict(stride=8 * 64 + 4), INVALID), (dict(slot=d), INVALID),
    (dict(qkv=z), INVALID), (dict(depth=z), INVALID), (dict(q=P(264)), INVALID), (dict(wq=P(258)), INVALID),
    (dict(Hq=2 ** 30, stride=2 ** 40), UNSUPPORTED), (dict(B=0, qkv=z), 0),
])
def test_norm_refusals(lib, kw, rc):
    assert _norm(lib, **kw) == rc


def _attn(lib, **kw):
    a = dict(q=d, k=d, v=d, S=64, ks=d, kl=d, anc=d, depth=d, status=d, B=1, M=3, Hq=4, Hkv=2, D=64, scale=0.1,
             cap=50.0, window=0, slopes=z, out=d, ws=z, ws_bytes=0, slot=z, ns=0, stream=z)
    assert set(kw) <= set(a)
    return lib.tree_attention_scored(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(M=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(cap=-1.0), INVALID), (dict(cap=float("nan")), INVALID), (dict(cap=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(window=4, depth=z), INVALID), (dict(slopes=d, depth=z), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(M=256), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED), (dict(q=P(264)), INVALID),
    (dict(out=z), INVALID), (dict(slot=d), INVALID), (dict(status=z), INVALID), (dict(B=0, q=z), 0),
    (dict(B=4096, M=255, Hq=4096, Hkv=1, S=2 ** 20), UNSUPPORTED),  # 2^12 * 2^13 * 2^14 tiles
])
def test_attention_refusals(lib, kw, rc):
    assert _attn(lib, **kw) == rc


def _samp(lib, **kw):
    a = dict(logits=d, kind=0, stride=100, u=d, T=d, k=z, p=z, m=z, draft=d, parent=d, depth=d, anc=d, status=d, B=1,
             M=3, V=100, md=3, tok=d, lp=z, al=d, path=d, bonus=d, ws=d, ws_bytes=1 << 20, stream=z)
    assert set(kw) <= set(a)
    return lib.tree_accept_sample(*{**a, **kw}.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), INVALID), (dict(M=-1), INVALID), (dict(V=0), INVALID), (dict(md=-1), INVALID),
    (dict(stride=99), INVALID), (dict(kind=2), INVALID), (dict(M=256), UNSUPPORTED),
    (dict(V=262145, stride=262145), UNSUPPORTED), (dict(logits=P(257)), INVALID), (dict(logits=P(258)), INVALID),
    (dict(u=z), INVALID), (dict(T=z), INVALID), (dict(tok=z), INVALID), (dict(ws=z), INVALID),
    (dict(ws=P(264)), INVALID), (dict(ws_bytes=8), INVALID), (dict(B=0, logits=z), 0),
])
def test_sample_refusals(lib, kw, rc):
    assert _samp(lib, **kw) == rc


def test_binding_refuses_host_tensors_and_wrong_shapes():
    B, n, V = 2, 3, 10
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    args = dict(logits=f(B, n, V), uniform=f(B, n), temperature=f(B), draft=i(B, n), parent=i(B, n), depth=i(B, n),
                anc_mask=i(B, n, 1), status=i(B), max_depth=2, token=i(B, n), accept_len=i(B), path=i(B, 3), bonus=i(B),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(tv.TVError, match="GPU"):
        tv.tree_accept_sample(**args)
    for name, bad in (("logits", f(B, n, V).double()), ("uniform", f(B, n + 1)), ("top_p", f(B, 1)), ("token", f(B, n)),
                      ("logits", f(B, n, 2 * V)[..., ::2]), ("logits", f(B, 2 * n, V)[:, :n]),
                      ("logits", f(1, 1, V).expand(B, n, V))):
        with pytest.raises(tv.TVError, match=name):
            tv.tree_accept_sample(**{**args, name: bad})
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    attn = dict(q=b16(1, 3, 4, 64), k=b16(1, 2, 9, 64), v=b16(1, 2, 9, 64), kv_start=i(1), kv_len=i(1),
                anc_mask=i(1, 3, 1), depth=i(1, 3), status=i(1), out=b16(1, 3, 4, 64))
    with pytest.raises(tv.TVError, match="GPU"):
        tv.tree_attention_scored(**attn)
    for name, bad in (("alibi_slopes", f(2)), ("k", b16(2, 2, 9, 64)), ("q", f(1, 3, 4, 64)), ("slot", i(2))):
        with pytest.raises(tv.TVError, match=name):
            tv.tree_attention_scored(**{**attn, name: bad})
    norm = dict(qkv=b16(1, 3, 8, 64), q_weight=None, k_weight=None, q_out=b16(1, 3, 4, 64), k=b16(1, 2, 9, 64),
                v=b16(1, 2, 9, 64), kv_start=i(1), kv_len=i(1), depth=i(1, 3))
    with pytest.raises(tv.TVError, match="GPU"):
        tv.tree_qk_norm_rope(**norm)
    for name, bad in (("qkv", b16(1, 3, 7, 64)), ("q_weight", b16(128)), ("depth", i(1, 4)),
                      ("qkv", b16(1, 3, 8, 128)[..., ::2])):
        with pytest.raises(tv.TVError, match=name):
            tv.tree_qk_norm_rope(**{**norm, name: bad})
