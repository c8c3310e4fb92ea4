"""The verification-step operators beside plain greedy ones, as cases to measure.

Three operators of one step: ``norm_rope`` (per-head norms of queries and keys,
rotation to the tree positions, the cache append), ``attention`` (tree attention
with capped scores, a sliding window or a bias that falls with distance) and
``sample`` (sampled acceptance: temperature, top-k, top-p, min-p).  ``run``
computes each in elementary torch operations, or through the package's calls
where ``own`` is true.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1e6
EPS = 1e-6

# Token counts, head layouts and vocabularies are those of the repository's own
# workloads (tiny, mha7b, eqspec, b32gqa, stress) or generic.
_LISTED = [
    # one new token of one sequence, the latency case of plain decoding
    dict(name="norm_rope token", op="norm_rope", B=1, M=0, Hq=32, Hkv=8, D=128, R=128, lo=2048, hi=2048, left=False,
         spare=0, pad=0),
    # a 64-node tree, as many key heads as query heads (mha7b)
    dict(name="norm_rope mha tree", op="norm_rope", B=1, M=64, Hq=32, Hkv=32, D=128, R=128, lo=2048, hi=2048,
         left=False, spare=0, pad=0),
    # chains of five drafts in a pool with free slots, half of each head rotated, padded projection rows
    dict(name="norm_rope pool chains", op="norm_rope", B=8, M=5, Hq=32, Hkv=8, D=64, R=32, lo=512, hi=4096,
         left=False, spare=5, pad=64),
    # the largest trees and batch (stress)
    dict(name="norm_rope large", op="norm_rope", B=16, M=128, Hq=64, Hkv=8, D=128, R=128, lo=512, hi=4096, left=True,
         spare=0, pad=0),
    # the smallest tree step: a short prefix, head dim 64, capped scores (tiny)
    dict(name="attention tiny capped", op="attention", B=1, M=16, Hq=4, Hkv=4, D=64, lo=128, hi=128, cap=30.0,
         window=0, alibi=False, depth=10, left=False, spare=0),
    # plain decoding of a ragged batch, one token each, capped scores
    dict(name="attention token capped", op="attention", B=8, M=0, Hq=32, Hkv=8, D=128, lo=512, hi=4096, cap=50.0,
         window=0, alibi=False, depth=0, left=True, spare=0),
    # a local layer over long prefixes: only the window's keys count
    dict(name="attention long window", op="attention", B=8, M=5, Hq=32, Hkv=8, D=128, lo=4096, hi=32768, cap=50.0,
         window=4096, alibi=False, depth=5, left=False, spare=3),
    # a large batch of small trees, bias by distance (b32gqa)
    dict(name="attention batch bias", op="attention", B=32, M=16, Hq=32, Hkv=2, D=128, lo=8192, hi=8192, cap=0.0,
         window=0, alibi=True, depth=10, left=False, spare=0),
    # large trees over long prefixes, capped scores, bound by the tensor cores (half of stress)
    dict(name="attention large capped", op="attention", B=8, M=128, Hq=64, Hkv=8, D=128, lo=4096, hi=16384, cap=50.0,
         window=0, alibi=False, depth=12, left=True, spare=0),
    # plain decoding: one token for each of eight users with settings of their own
    dict(name="sample token", op="sample", B=8, M=0, V=151936, bf16=False, rule="mixed", sigma=2.0, depth=0, pad=0),
    # a 64-node tree of one sequence, bf16 logits, nucleus sampling
    dict(name="sample tree nucleus", op="sample", B=1, M=64, V=32000, bf16=True, rule="top_p", sigma=2.0, depth=6,
         pad=0),
    # the largest trees, batch and logits (stress), users with settings of their own
    dict(name="sample large", op="sample", B=16, M=128, V=128256, bf16=False, rule="mixed", sigma=2.0, depth=12,
         pad=0),
]

_RULES = ("temperature", "top_k", "top_p", "min_p", "top_k top_p", "mixed")


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "attention", "sample"))
    M = rng.choice((0, _log(rng, 1, 128)))
    B = _log(rng, 1, 32)
    if op == "sample":
        V = _log(rng, 1000, 151936)
        while B * (M + 1) * V > 2064 * 128256:
            B, M = max(1, B // 2), M // 2
        return dict(op=op, B=B, M=M, V=V, bf16=rng.random() < 0.5, rule=rng.choice(_RULES),
                    sigma=rng.choice((1.0, 2.0, 3.0)), depth=min(M, rng.randint(4, 12)),
                    pad=rng.choice((0, rng.randint(1, 64))))
    D = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8, 32))
    Hq = Hkv * rng.choice((1, 2, 4, 7, 8, 16) if Hkv < 8 else (1, 2, 4))
    if op == "norm_rope":
        lo = _log(rng, 16, 4096)
        while B * (M + 1) * Hq > 2064 * 64:
            B = max(1, B // 2)
        while B * Hkv * (lo + 200) > 32 * 8 * 4096:
            lo //= 2
        return dict(op=op, B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, R=rng.choice((D, D, D // 2)), lo=max(1, lo // 2), hi=lo,
                    left=rng.random() < 0.5, spare=rng.choice((0, 3)), pad=rng.choice((0, 8, 64)))
    hi = _log(rng, 16, 32768)
    while B > 1 and (B * Hkv * hi * D > 8 * 8 * 32768 * 128 or B * (M + 1) * Hq * (hi + M) > 8 * 129 * 64 * 16384):
        B //= 2
    while B * (M + 1) * Hq * (hi + M) > 8 * 129 * 64 * 16384:
        hi //= 2
    return dict(op=op, B=B, M=M, Hq=Hq, Hkv=Hkv, D=D, lo=max(1, hi // 4), hi=hi, cap=rng.choice((0.0, 20.0, 50.0)),
                window=rng.choice((0, _log(rng, 1, 4096))), alibi=rng.random() < 0.4, depth=min(M, rng.randint(4, 12)),
                left=rng.random() < 0.5, spare=rng.choice((0, 3)))


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _tree(B, M, depth, g_cpu):
    """Random trees of M nodes and at most the given depth, one for each sequence: parent, node depths, and which
    rows are ancestors (itself included), as truth values and as 32-bit words."""
    n = M + 1
    parent = torch.zeros((B, n), dtype=torch.int64)
    dep = torch.zeros((B, n), dtype=torch.int64)
    anc = torch.zeros((B, n, n), dtype=torch.bool)
    anc[:, 0, 0] = True
    pick = torch.rand((B, n), generator=g_cpu)
    rows = torch.arange(B)
    for i in range(1, n):
        ok = dep[:, :i] < depth
        # the pick-th of the rows that may have a child
        want = (pick[:, i] * ok.sum(1)).long()
        p = ((ok.cumsum(1) - 1 == want[:, None]) & ok).long().argmax(1)
        parent[:, i] = p
        dep[:, i] = dep[rows, p] + 1
        anc[:, i] = anc[rows, p]
        anc[:, i, i] = True
    W = (n + 31) // 32
    words = torch.zeros((B, n, W * 32), dtype=torch.int64)
    words[:, :, :n] = anc
    words = (words.view(B, n, W, 32) << torch.arange(32)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    i32 = torch.int32
    return dict(parent=parent.to(DEV, i32), depth=dep.to(DEV, i32), anc=anc.to(DEV), anc_words=words.to(DEV, i32))


def _geometry(c, g_cpu):
    """Where each sequence's prefix lies, and the cache slots of the batch (None: slot = row)."""
    B, M = c["B"], c["M"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=g_cpu)
    S = (c["hi"] + M + 1 + 7) // 8 * 8
    start = (lens.max() - lens) if c["left"] else torch.zeros_like(lens)
    n_slots = B + c["spare"]
    slot = torch.randperm(n_slots, generator=g_cpu)[:B] if c["spare"] else None
    ks, kl = torch.zeros(n_slots, dtype=torch.int64), torch.zeros(n_slots, dtype=torch.int64)
    rows = torch.arange(B) if slot is None else slot
    ks[rows], kl[rows] = start, lens
    i32 = torch.int32
    return dict(S=S, n_slots=n_slots, slot=None if slot is None else slot.to(DEV, i32), rows=rows.to(DEV),
                kv_start=ks.to(DEV, i32), kv_len=kl.to(DEV, i32))


def prepare(case, seed):
    c = case
    g, h = _gen(seed), torch.Generator().manual_seed(int(seed) + 1)
    B, n = c["B"], c["M"] + 1
    bf, i32 = torch.bfloat16, torch.int32
    s = dict(c)
    if c["op"] == "sample":
        V = c["V"]
        s.update(_tree(B, c["M"], max(1, c["depth"]), h))
        # teacher logits: a bulk, and in each row a few dozen tokens that stand out, by different amounts
        full = torch.empty((B, n, V + c["pad"]), dtype=torch.float32, device=DEV).normal_(0, c["sigma"], generator=g)
        hot = torch.randint(0, V, (B, n, 48), generator=g, device=DEV)
        up = torch.rand((B, n, 48), generator=g, device=DEV).square() * (5.0 * c["sigma"]) + 2.0 * c["sigma"]
        full.scatter_add_(2, hot, up)
        s["logits"] = (full.to(bf) if c["bf16"] else full)[..., :V]
        s["uniform"] = torch.rand((B, n), generator=g, device=DEV)
        # settings for each sequence
        kind = torch.randint(0, 6, (B,), generator=h) if c["rule"] == "mixed" else \
            torch.full((B,), _RULES.index(c["rule"]))
        r = torch.rand((B, 4), generator=h)
        T = 0.5 + r[:, 0]
        if c["rule"] == "mixed":
            T[kind == 5] = 0.0  # a greedy user
        has_k, has_p, has_m = (kind == 1) | (kind == 4), (kind == 2) | (kind == 4), kind == 3
        s["temperature"] = T.to(DEV)
        s["top_k"] = torch.where(has_k, (r[:, 1] * 99).long() + 2, 0).to(DEV, i32)
        s["top_p"] = torch.where(has_p, 0.8 + 0.19 * r[:, 2], 1.0).to(DEV)
        s["min_p"] = torch.where(has_m, 0.02 + 0.1 * r[:, 3], 0.0).to(DEV)
        # drafts: what a draft model close to the teacher would propose
        top = s["logits"].float().topk(2, -1).indices.to(i32)
        at = s["parent"].long()[..., None].expand(-1, -1, 2)
        coin = torch.rand((B, n, 1), generator=g, device=DEV) < 0.7
        s["draft"] = torch.where(coin, top.gather(1, at)[..., :1], top.gather(1, at)[..., 1:])[..., 0].contiguous()
        s["draft"][:, 0] = 0
        D1 = max(1, c["depth"]) + 1
        e = lambda *shape, t=i32: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
        s.update(status=torch.zeros(B, dtype=i32, device=DEV), token=e(B, n), logprob=e(B, n, t=torch.float32),
                 accept_len=e(B), path=e(B, D1), bonus=e(B), max_depth=D1 - 1)
        return s
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    s.update(_geometry(c, h))
    s.update(_tree(B, c["M"], max(1, c.get("depth", 10)), h))

    def randn(*shape, sigma=1.0):
        x = torch.empty(shape, dtype=bf, device=DEV)
        flat = x.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            part = flat[i:i + (1 << 28)]
            part.copy_(torch.empty(part.shape, dtype=torch.float32, device=DEV).normal_(0, sigma, generator=g))
        return x

    s["k"], s["v"] = randn(s["n_slots"], Hkv, s["S"], D), randn(s["n_slots"], Hkv, s["S"], D)
    if c["op"] == "norm_rope":
        width = (Hq + 2 * Hkv) * D
        rows = randn(B, n, width + c["pad"], sigma=1.5)
        s["qkv"] = rows[..., :width].unflatten(-1, (Hq + 2 * Hkv, D))
        s["q_weight"] = (1 + 0.2 * randn(D).float()).to(bf)
        s["k_weight"] = (1 + 0.2 * randn(D).float()).to(bf)
        s["q_out"] = torch.empty((B, n, Hq, D), dtype=bf, device=DEV)
        return s
    # queries that match some keys well: scores up to about the cap's size
    s["q"] = randn(B, n, Hq, D, sigma=2.0)
    s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().to(DEV) if c["alibi"] else None
    s["status"] = torch.zeros(B, dtype=i32, device=DEV)
    s["out"] = torch.empty((B, n, Hq, D), dtype=bf, device=DEV)
    return s


# ----------------------------------------------------------------------------- the operators

def run(state):
    s = state
    if own:
        import tree_speculative_decoding_04_b200 as tv

        if s["op"] == "norm_rope":
            tv.tree_qk_norm_rope(s["qkv"], s["q_weight"], s["k_weight"], s["q_out"], s["k"], s["v"], s["kv_start"],
                                 s["kv_len"], s["depth"], eps=EPS, rope_theta=THETA, rotary_dim=s["R"], slot=s["slot"])
            return s["q_out"], s["k"], s["v"]
        if s["op"] == "attention":
            if "workspace" not in s:  # kept by the user's program from call to call
                s["workspace"] = tv.attention_scored_workspace(s["B"], s["M"], s["Hq"], s["Hkv"], s["D"], s["S"],
                                                               s["window"], s["q"].device)
            tv.tree_attention_scored(s["q"], s["k"], s["v"], s["kv_start"], s["kv_len"], s["anc_words"], s["depth"],
                                     s["status"], s["out"], s["workspace"], softcap=s["cap"], window=s["window"],
                                     alibi_slopes=s["slopes"], slot=s["slot"])
            return s["out"]
        if "workspace" not in s:
            s["workspace"] = tv.accept_sample_workspace(s["B"], s["M"], s["V"], s["logits"].device)
        tv.tree_accept_sample(s["logits"], s["uniform"], s["temperature"], s["draft"], s["parent"], s["depth"],
                              s["anc_words"], s["status"], s["max_depth"], s["token"], s["accept_len"], s["path"],
                              s["bonus"], s["workspace"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                              logprob=s["logprob"])
        return s["token"], s["logprob"], s["accept_len"], s["path"], s["bonus"]
    return {"norm_rope": _norm_rope, "attention": _attention, "sample": _sample}[s["op"]](s)


def _norm_rope(s):
    Hq, Hkv, R = s["Hq"], s["Hkv"], s["R"]
    B, n = s["B"], s["M"] + 1
    x = s["qkv"][:, :, :Hq + Hkv].float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    w = torch.cat([s["q_weight"].float().expand(Hq, -1), s["k_weight"].float().expand(Hkv, -1)])
    x = x * w
    pos = s["kv_len"][s["rows"]][:, None] + s["depth"]
    freq = THETA ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    angle = pos.double()[..., None] * freq
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    a, b, rest = x[..., :R // 2], x[..., R // 2:R], x[..., R:]
    x = torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1).to(torch.bfloat16)
    col = (s["kv_start"] + s["kv_len"])[s["rows"]][:, None] + torch.arange(n, device=DEV)
    at = (s["rows"][:, None, None], torch.arange(Hkv, device=DEV)[None, None], col[:, :, None].long())
    s["k"][at] = x[:, :, Hq:]
    s["v"][at] = s["qkv"][:, :, Hq + Hkv:]
    return x[:, :, :Hq].contiguous(), s["k"], s["v"]


def _attention(s):
    Hq, Hkv, D, n, B = s["Hq"], s["Hkv"], s["D"], s["M"] + 1, s["B"]
    G = Hq // Hkv
    start, length = s["kv_start"][s["rows"]].long(), s["kv_len"][s["rows"]].long()
    N = s["S"]
    j = torch.arange(N, device=DEV)
    at = (start[:, None] + j).clamp(max=N - 1)[:, None, :, None].expand(-1, Hkv, -1, D)
    K = s["k"][s["rows"]].gather(2, at).float()
    V = s["v"][s["rows"]].gather(2, at).float()
    q = s["q"].view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D).float()
    x = (q @ K.mT).mul_(D ** -0.5).view(B, Hkv, n, G, N)
    if s["cap"]:
        x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
    # position of each key, and which keys each node may read
    r = (j - length[:, None]).clamp(0, n - 1)
    in_tree = (j >= length[:, None]) & (j < length[:, None] + n)
    kpos = torch.where(in_tree, length[:, None] + s["depth"].long().gather(1, r), j)
    qpos = length[:, None] + s["depth"]
    dist = qpos[:, :, None] - kpos[:, None]
    ok = (j < length[:, None])[:, None] | (in_tree[:, None] & s["anc"].gather(2, r[:, None].expand(-1, n, -1)))
    if s["window"]:
        ok &= dist < s["window"]
    if s["slopes"] is not None:
        x.sub_(s["slopes"].view(1, Hkv, 1, G, 1) * dist[:, None, :, None].float())
    x.masked_fill_(~ok[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (x.view(B, Hkv, n * G, N) @ V).view(B, Hkv, n, G, D) / x.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(torch.bfloat16)


def _sample(s):
    x = s["logits"].float()
    B, n, V = x.shape
    T = s["temperature"].double()
    greedy = T <= 0
    T = torch.where(greedy, 1.0, T)[:, None, None]
    k = torch.where(greedy, 1, torch.where(s["top_k"] > 0, s["top_k"], V))[:, None, None]
    vals, order = torch.sort(x, dim=-1, descending=True, stable=True)
    w = ((vals.double() - vals[..., :1].double()) / T).exp_()
    rank = torch.arange(V, device=DEV)
    w = torch.where(rank < k, w, 0.0)
    total = w.sum(-1, keepdim=True)
    before = w.cumsum(-1).sub_(w)
    p = s["top_p"].double()[:, None, None]
    keep = (before < p * total) | (p >= 1)
    keep &= w >= s["min_p"].double()[:, None, None]
    keep |= rank == 0
    w = torch.where(keep, w, 0.0)
    total = w.sum(-1, keepdim=True)
    del before, keep, vals
    w = torch.zeros_like(w).scatter_(2, order, w)
    below = w.cumsum(-1) <= s["uniform"].double()[..., None] * total
    last = (w > 0).long().mul_(rank).amax(-1)
    token = torch.minimum(below.sum(-1), last)
    lw = (x.gather(2, token[..., None]).double() - x.amax(-1, keepdim=True).double()) / T
    logprob = (lw - total.log())[..., 0].float()
    # the longest path whose drafts are the drawn tokens
    match = s["draft"] == token.gather(1, s["parent"].long())
    match[:, 0] = True
    good = (match[:, None] | ~s["anc"]).all(-1)
    row = torch.arange(n, device=DEV)
    end = torch.where(good, s["depth"] * 1024 - row, -(1 << 30)).argmax(-1)
    on = s["anc"][torch.arange(B, device=DEV), end]
    path = torch.zeros((B, s["max_depth"] + 2), dtype=torch.int64, device=DEV)
    path.scatter_(1, torch.where(on, s["depth"].long(), s["max_depth"] + 1), row.expand(B, -1))
    i32 = torch.int32
    return (token.to(i32), logprob, s["depth"].gather(1, end[:, None])[:, 0], path[:, :-1].to(i32).contiguous(),
            token.gather(1, end[:, None])[:, 0].to(i32))


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    n = c["M"] + 1
    rows = c["B"] * n
    if c["op"] == "sample":
        el = rows * c["V"]
        return {"bytes": el * (2 if c["bf16"] else 4) + 40 * rows, "flops": 4 * el}
    if c["op"] == "norm_rope":
        el = rows * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 4 * el + 4 * rows, "flops": 10 * el}
    keys = (c["lo"] + c["hi"]) / 2
    if c["window"]:
        keys = min(keys, c["window"])
    kv = c["B"] * c["Hkv"] * (keys + n) * c["D"] * 4
    # a node reads its own ancestors only: about half the tree's depth
    pairs = rows * c["Hq"] * (keys + 1 + c["depth"] / 2)
    return {"bytes": kv + rows * c["Hq"] * c["D"] * 4, "flops": 4 * c["D"] * pairs}


# ----------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](s)


def _exact_norm_rope(s):
    Hq, Hkv, R, n, D = s["Hq"], s["Hkv"], s["R"], s["M"] + 1, s["D"]
    k, v = s["k"].double(), s["v"].double()
    q = torch.empty((s["B"], n, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(s["B"]):
        sl = int(s["rows"][b])
        c0, length = int(s["kv_start"][sl] + s["kv_len"][sl]), int(s["kv_len"][sl])
        x = s["qkv"][b].double()
        v[sl, :, c0:c0 + n] = x[:, Hq + Hkv:].transpose(0, 1)
        for part, weight in (("q", s["q_weight"]), ("k", s["k_weight"])):
            y = x[:, :Hq] if part == "q" else x[:, Hq:Hq + Hkv]
            y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
            ang = (length + s["depth"][b].double())[:, None, None] / THETA ** (
                torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)
            z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * torch.polar(
                torch.ones_like(ang), ang)
            y = torch.cat([z.real, z.imag, y[..., R:]], -1)
            if part == "q":
                q[b] = y
            else:
                k[sl, :, c0:c0 + n] = y.transpose(0, 1)
    return q, k, v


def _exact_attention(s):
    Hq, Hkv, D, n, B = s["Hq"], s["Hkv"], s["D"], s["M"] + 1, s["B"]
    G = Hq // Hkv
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        sl = int(s["rows"][b])
        c0, length = int(s["kv_start"][sl]), int(s["kv_len"][sl])
        N = length + n
        dep = s["depth"][b].double()
        kpos = torch.cat([torch.arange(length, device=DEV, dtype=torch.float64), length + dep])
        dist = (length + dep)[:, None] - kpos
        ok = torch.cat([torch.ones((n, length), dtype=torch.bool, device=DEV), s["anc"][b]], 1)
        if s["window"]:
            ok = ok & (dist < s["window"])
        for h in range(Hkv):
            K, V = s["k"][sl, h, c0:c0 + N].double(), s["v"][sl, h, c0:c0 + N].double()
            a = torch.einsum("ngd,sd->gns", s["q"][b, :, h * G:(h + 1) * G].double(), K) / math.sqrt(D)
            if s["cap"]:
                a = torch.tanh(a / s["cap"]) * s["cap"]
            if s["slopes"] is not None:
                a = a - s["slopes"][h * G:(h + 1) * G].double()[:, None, None] * dist
            a = torch.where(ok, a, -math.inf)
            a = torch.exp(a - torch.logsumexp(a, -1, keepdim=True))
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gns,sd->ngd", a, V)
    return out


def _exact_sample(s):
    """The log probability of each row's drawn token; the drawn tokens and the walk are whole numbers."""
    x = s["logits"]
    B, n, V = x.shape
    got = torch.zeros((B, n), dtype=torch.float64, device=DEV)
    for b in range(B):
        T, k, p, m = (float(s[f][b]) for f in ("temperature", "top_k", "top_p", "min_p"))
        if T <= 0:
            continue
        for u0 in range(0, n, 16):
            l = x[b, u0:u0 + 16].double()
            order = torch.argsort(-l, dim=-1, stable=True)
            prob = torch.softmax(l / T, -1).gather(1, order)
            if 0 < k < V:
                prob[:, int(k):] = 0
                prob = prob / prob.sum(-1, keepdim=True)
            keep = torch.ones_like(prob, dtype=torch.bool)
            if p < 1:
                keep[:, 1:] &= (prob.cumsum(-1) < p)[:, :-1]
            if m > 0:
                keep[:, 1:] &= (prob >= m * prob[:, :1])[:, 1:]
            prob = prob * keep
            prob = prob / prob.sum(-1, keepdim=True)
            flat = torch.zeros_like(prob).scatter_(1, order, prob)
            cum = flat.cumsum(-1)
            t = torch.searchsorted(cum, s["uniform"][b, u0:u0 + 16].double()[:, None] * cum[:, -1:], right=True)
            got[b, u0:u0 + 16] = flat.gather(1, t.clamp(max=V - 1)).log()[:, 0]
    return None, got, None, None, None
