"""Inputs, a vectorised float64 reference and calls for the tests of
tree_qk_norm_rope, tree_attention_scored and tree_accept_sample."""
import math

import numpy as np
import torch

import workloads as W


def tree_tables(parent):
    """parent [B][n] -> (depth [B][n], anc bool [B][n][n]) by walking the pointers."""
    B, n = parent.shape
    depth = np.zeros((B, n), np.int64)
    anc = np.zeros((B, n, n), bool)
    for b in range(B):
        anc[b, 0, 0] = True
        for u in range(1, n):
            p = parent[b, u]
            depth[b, u] = depth[b, p] + 1
            anc[b, u] = anc[b, p]
            anc[b, u, u] = True
    return depth, anc


def attention_ref(q, k, v, kv_start, kv_len, parent, status, scale=None, softcap=0.0, window=0, slopes=None,
                  slots=None):
    """(out, mean) float64 like q: softmax(scores) v, and the same weights over |v|."""
    B, n, Hq, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    depth, anc = tree_tables(parent)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mean = torch.zeros_like(out)
    for b in range(B):
        sl = b if slots is None else int(slots[b])
        if status[b] != 0 or not 0 <= sl < k.shape[0]:
            continue
        ks, L = int(kv_start[sl]), int(kv_len[sl])
        if ks < 0 or L < 0 or ks + L + n > S_cap:
            continue
        dep = torch.as_tensor(depth[b], dtype=torch.float64, device=q.device)
        kpos = torch.cat([torch.arange(L, dtype=torch.float64, device=q.device), L + dep])
        dist = (L + dep)[:, None] - kpos[None]
        ok = torch.cat([torch.ones((n, L), dtype=torch.bool, device=q.device),
                        torch.as_tensor(anc[b], device=q.device)], 1)
        if window > 0:
            ok &= dist < window
        for h in range(Hkv):
            K, V = k[sl, h, ks:ks + L + n].double(), v[sl, h, ks:ks + L + n].double()
            V = torch.where(ok.any(0)[:, None], V, 0.0)
            K = torch.where(ok.any(0)[:, None], K, 0.0)
            s = torch.einsum("ugd,xd->ugx", q[b, :, h * G:(h + 1) * G].double(), K) * scale
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[h * G:(h + 1) * G].double()[None, :, None] * dist[:, None]
            p = torch.softmax(s.masked_fill(~ok[:, None], -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = p @ V
            mean[b, :, h * G:(h + 1) * G] = p @ V.abs()
    return out, mean


# Errors of one output of the scored attention, with u = 2^-8 the largest relative
# error of a rounding to bf16: the output itself is rounded (u |out|), and so is
# every softmax weight (u times the weighted mean of |v|; as the normaliser sums the
# rounded weights, a single output may reach u times the weighted mean of |v - out|
# instead, for a row of few keys whose heaviest has the smallest v: up to |out| more,
# which none of the tests' inputs comes to).  What is left are errors of the fp32 scores: a score of size
# |s| <= 100 off by a few fp32 roundings of itself and of the sum of |q k| terms
# (100 * 2^-20 < 2^-13 in the exponent), and the exponential's 2^-22: together
# below 2^-12 of the weighted mean.
def attention_tolerance(out, mean):
    return 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -11) * mean + 1e-30


# Errors of one output of the norm and rotation: the rounding to bf16, and fp32
# arithmetic on the two elements of the pair (a sum of squares of at most 128
# terms, a reciprocal square root, five products, sine and cosine off by at most
# 2^-20): below 2^-17 of |a| + |b|.
def rope_tolerance(out, mag):
    return 2.0 ** -8 * np.abs(out) + 2.0 ** -17 * mag + 1e-30


def parents(B, M, max_depth, rng, tree="uniform"):
    if tree == "chain":
        return np.stack([W.tree_chain(M)] * B).astype(np.int32)
    return np.stack([W.tree_uniform_depth(M, max_depth, rng) for _ in range(B)]).astype(np.int32)
