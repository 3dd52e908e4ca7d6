"""Single-exit LM-head operators where they can go wrong: peaked rows whose gradient is a small
difference, magnitudes near the ends of the type, logits that are not numbers, alternatives that differ in the last bits."""
import functools

import numpy as np
import pytest
import torch

from lm_head_loss_junction_b200 import token_logprobs, token_logprobs_bwd, topk_distill_bwd, topk_distill_fwd
from oracle import head as oh
from tests.head_helpers import Bounds, check_grads, check_top, half_step, make, within
from tests.test_parity_head import gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- gradients of peaked rows
@functools.lru_cache(maxsize=None)
def peaked(T, D, V, dtype=BF, seed=0):
    """Rows that are nearly certain of one token: q_y from 0.99 to 0.9997, and W with a mean row as long as its
    spread, so that what is lost of a row's small probabilities does not average out."""
    rng = np.random.Generator(np.random.PCG64(seed))
    W = rng.normal(size=(V, D)) * 2.0 / np.sqrt(D)
    mean = rng.normal(size=D) * 2.0 / np.sqrt(D)
    W = torch.from_numpy((W + mean).astype(np.float32)).to(dtype)
    Wd = W.double().numpy()
    y = rng.choice(V, size=T, replace=False).astype(np.int32)
    h, to = rng.normal(size=(T, D)) * 0.5, Wd[y] - mean
    base, lean = h @ Wd.T, to @ Wd.T
    target = np.resize([0.99, 0.995, 0.9975, 0.999, 0.9997], T)
    lo, hi = np.zeros(T), np.full(T, 60.0)
    for _ in range(24):
        mid = (lo + hi) / 2
        logq, _ = oh.log_softmax(base + mid[:, None] * lean)
        low = np.exp(logq[np.arange(T), y]) < target
        lo, hi = np.where(low, mid, lo), np.where(low, hi, mid)
    return torch.from_numpy((h + lo[:, None] * to).astype(np.float32)).to(dtype), W, y


def check_peaked(b, y, s, dh, dW):
    """Gradients of s_t (log q_y) of peaked rows: every token's dh and every untouched token's dW row keep their own
    relative precision.

    Bound of an entry of G, dl the error of a logit: an entry of a small probability is off by 2 dl (its logit and its
    row's log-sum-exp) + 2^-19 (exp, log) of itself, and 2^-11 (fp16; fp32 path: 2^-22); what is lost below fp16's
    smallest number is 2^-25 of a row stored between 2^13 and 2^15 times its largest coefficient: 2^-38 s.  The
    target's own entry is formed from its logit in 64 bits and the fp32 log-sum-exp (rounded, exp and log: 2^-24 |lse|
    and 2^-20 of s), in which the others' terms are off as above.  fp32 inputs: the log-sum-exp comes from fp32 logits
    but for the target's, which is as exact."""
    T, V = b.h.shape[0], b.W.shape[0]
    rows = np.arange(T)
    logq, lse = oh.log_softmax(b.h @ b.W.T)
    assert 0.985 < np.exp(logq[rows, y]).min() and np.exp(logq[rows, y]).max() < 0.9999
    G = np.exp(logq) * s
    G[rows, y] = 0.0
    G[rows, y] = -G.sum(axis=1)
    rel = 2 * b.dl + 2.0 ** -19 + (2.0 ** -11 if b.bf16 else 2.0 ** -22)
    e = rel[:, None] * np.abs(G) + (2.0 ** -38 * s if b.bf16 else 0.0)
    e[rows, y] += s * (2.0 ** -24 * np.abs(lse) + 2.0 ** -20)
    aG = np.abs(G)
    exp = G @ b.W
    within(dh, exp, e @ np.abs(b.W) + b._sum(V) * (aG @ np.abs(b.W)) + half_step(dh.dtype) * np.abs(exp), "dh")
    rare = np.setdiff1d(np.arange(V), y)
    exp = G.T[rare] @ b.h
    # h is copied to fp16 over at most twice its largest value: 2^-38 of that below fp16's normal range
    copy = 2.0 ** -37 * np.abs(b.h).max() * aG.T[rare].sum(axis=1, keepdims=True) if b.bf16 else 0.0
    within(dW[torch.from_numpy(rare).cuda()], exp, e.T[rare] @ np.abs(b.h) + copy + b._sum(T) * (aG.T[rare] @ np.abs(b.h)) +
           half_step(F32) * np.abs(exp), "dW of other tokens")


def peaked_step(op, y, h, W, **kw):
    """dh and dW of the mean of -log q_y."""
    T = y.shape[0]
    if op == "score":
        _, stats, _, _ = token_logprobs(y, h, W, **kw)
        return token_logprobs_bwd(y, h, W, stats, torch.full((T,), -1.0 / T, device="cuda"))
    z, ids = torch.zeros(T, 1, device="cuda"), y[:, None].contiguous()
    _, stats = topk_distill_fwd(y, ids, z, h, W)
    return topk_distill_bwd(y, ids, z, h, W, stats)


@pytest.mark.parametrize("T,D,V", [(150, 128, 49152), (520, 192, 33001), (200, 128, 131072)])
@pytest.mark.parametrize("op", ["score", "distill"])
def test_gradients_of_peaked_rows(T, D, V, op):
    h, W, y = peaked(T, D, V)
    check_peaked(Bounds(h, W), y, 1.0 / T, *peaked_step(op, *gpu(y, h, W)))


@pytest.mark.parametrize("op,T,D,V,dtype,top_k", [
    ("score", 20, 128, 49152, BF, 0), ("distill", 20, 128, 49152, BF, 0), ("score", 100, 1024, 9000, BF, 0),
    ("distill", 60, 2304, 6001, BF, 0), ("score", 20, 4352, 6001, BF, 0), ("score", 150, 2304, 6001, BF, 8),
    ("score", 520, 640, 6001, BF, 1), ("score", 100, 1024, 9000, BF, 33), ("score", 140, 192, 4001, F32, 0),
    ("distill", 140, 192, 4001, F32, 0), ("score", 140, 192, 4001, F32, 5)])
def test_peaked_rows_whatever_made_their_statistics(op, T, D, V, dtype, top_k):
    """Few tokens and alternatives have their log-sum-exp from other sums than the gradient's logits."""
    h, W, y = peaked(T, D, V, dtype)
    kw = dict(top_k=top_k) if top_k else {}
    check_peaked(Bounds(h, W), y, 1.0 / T, *peaked_step(op, *gpu(y, h, W), **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_of_some_rows_of_a_batch(dtype):
    """The statistics of a long batch, the gradients of a few of its rows."""
    h, W, y = peaked(300, 512, 6001, dtype)
    hg, Wg, yg = gpu(h, W, y)
    _, stats, _, _ = token_logprobs(yg, hg, Wg)
    for a, b in ((0, 40), (40, 300)):
        n = b - a
        dh, dW = token_logprobs_bwd(yg[a:b], hg[a:b], Wg, stats[:, a:b].contiguous(),
                                    torch.full((n,), -1.0 / n, device="cuda"))
        check_peaked(Bounds(h[a:b], W), y[a:b], 1.0 / n, dh, dW)


def test_heavy_entries_named_twice():
    """A token that holds its row, named in several places of its list and among the teacher's: its terms count once
    in the log-sum-exp, its coefficients all of them in the gradient."""
    T, D, V, K = 40, 1024, 5000, 64
    h, W, y = peaked(T, D, V)
    rng = np.random.Generator(np.random.PCG64(2))
    ids = rng.integers(0, V, size=(T, K)).astype(np.int32)
    for j in (0, 5, 31, 32, 40, 63):
        ids[:, j] = np.where(rng.random(T) < 0.7, y, ids[:, j])
    g = rng.normal(size=(T, K)).astype(np.float32)
    hg, Wg, ig, gg, yg = gpu(h, W, ids, g, y)
    b = Bounds(h, W)
    r = oh.token_logprobs(ids, h, W)
    logp, stats, _, _ = token_logprobs(ig, hg, Wg)
    within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
    within(logp, r["logp"], b.logp(r["lse"])[:, None] * np.ones((1, K)), "logp")
    once, stats1, _, _ = token_logprobs(yg, hg, Wg)
    named = torch.from_numpy((ids == y[:, None]).any(axis=1)).cuda()
    assert torch.equal(stats[:, named], stats1[:, named])
    dh, dW = token_logprobs_bwd(ig, hg, Wg, stats, gg)
    s = np.maximum(np.abs(g.astype(np.float64).sum(1)), np.abs(g).max(1))
    check_grads(b, oh.token_logprobs_grad(ids, h, W, g), s, dh, dW)
    z = rng.normal(size=(T, K)).astype(np.float32)
    losses, dstats = topk_distill_fwd(yg, ig, gpu(z)[0], hg, Wg, 0.4)
    d = oh.topk_distill(y, ids, z, h, W, 0.4)
    within(dstats[1], d["stats"][1], b.logp(r["lse"]), "ce")
    within(dstats[2], d["stats"][2], b.logp(r["lse"]) + 2.0 ** -20 * np.abs(d["stats"][2]), "kd")
    check_grads(b, d["G"], np.full(T, 1.0 / T), *topk_distill_bwd(yg, ig, gpu(z)[0], hg, Wg, dstats, 0.4))


@pytest.mark.parametrize("T", [40, 150])
@pytest.mark.parametrize("D", [640, 4352])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top_k", [0, 8])
def test_peaked_rows_whose_sums_are_exact(T, D, dtype, top_k):
    """One entry a row in h, the target at 64 and every other token at 46 or 45: no sum is truncated, so a tensor-core
    logit is off by what is given back, dl = D 2^-30 of it, and nothing else (fp32: not at all).  Gradients of the log
    probability, and of the entropy, whose own difference is that of log q_y and minus the entropy.

    Bound of an entry of G = s (g (1_y - q) - e q (log q + H)), with z = sum e^(l - l_y) near 1: after the target's term
    come up to 64 of its block of columns (a thread's share of 128, 40 tokens) and 16 merges, each rounding z by 2^-24:
    2^-17.6, and so much of its logarithm, in log-sum-exp and entropy.  The log-sum-exp is rounded to fp32 (2^-24 |lse|);
    the others' part of the entropy is off by 2 dl, their logits and log-sum-exp by 2 dl of themselves.  fp16: 2^-11, and
    2^-36 s below its range (the row's bound is at most 9 s)."""
    V, s = 5000, 1.0 / T
    rng = np.random.Generator(np.random.PCG64(28))
    y = rng.choice(V, size=T, replace=False).astype(np.int32)
    h = torch.zeros(T, D)
    h[:, 0] = 32.0
    W = torch.from_numpy(rng.integers(0, 9, size=(V, D)) / 4.0).float()
    W[:, 0] = torch.from_numpy(np.where(rng.random(V) < 0.5, 46.0, 45.0) / 32).float()
    # each token its own head column, so that only its target is large
    own = 1 + np.arange(T)
    h[torch.arange(T), torch.from_numpy(own)] = 8.0
    W[:, 1:T + 1] = 0.0
    W[torch.from_numpy(y.astype(np.int64)), torch.from_numpy(own)] = (64.0 - 32 * W[torch.from_numpy(y.astype(np.int64)), 0]) / 8
    h, W = h.to(dtype), W.to(dtype)
    b = Bounds(h, W)
    rows = np.arange(T)
    logq, lse = oh.log_softmax(b.h @ b.W.T)
    q = np.exp(logq)
    assert (np.abs(b.h @ b.W.T)[rows, y] == 64).all() and 0.9998 < q[rows, y].min() and q[rows, y].max() < 0.99999
    H = -np.sum(q * logq, axis=1)
    hg, Wg, yg = gpu(h, W, y)
    _, stats, _, _ = token_logprobs(yg, hg, Wg, top_k=top_k)
    dl = D * 2.0 ** -30 * 64 if b.bf16 else 0.0
    eH = 2 * dl * 20 * (1 - q[rows, y]) + 2.0 ** -17.6
    elq = 2.0 ** -24 * np.abs(lse) + 2.0 ** -17.6
    within(stats[1], H, eH, "entropy")
    for g, e in ((s, 0.0), (0.0, s), (s, 0.01 * s)):
        G = oh.token_logprobs_grad(y[:, None], b.h, b.W, np.full((T, 1), g), np.full(T, e))
        off = q * (g * (2 * dl + 2.0 ** -19) + e * (2 * dl * (np.abs(logq) + 1) + 2.0 ** -19 * (1 + np.abs(logq)) + eH[:, None]))
        off[rows, y] = g * elq + e * (elq + eH)
        off += 2.0 ** -11 * np.abs(G) + 2.0 ** -36 * s if b.bf16 else 2.0 ** -22 * np.abs(G)
        dh, dW = token_logprobs_bwd(yg, hg, Wg, stats, torch.full((T,), g, device="cuda"),
                                    torch.full((T,), e, device="cuda") if e else None)
        exp = G @ b.W
        within(dh, exp, off @ np.abs(b.W) + b._sum(V) * (np.abs(G) @ np.abs(b.W)) + half_step(dh.dtype) * np.abs(exp), "dh")


# ---------------------------------------------------------------- magnitudes
class Tiny(Bounds):
    """With what is lost below the smallest normal number: half of the output's smallest number, and of fp32's for
    each part of a sum (at most 74, and the copies')."""

    def dh(self, G, s, out):
        return super().dh(G, s, out) + torch.finfo(out).smallest_normal * torch.finfo(out).eps / 2 + 80 * 2.0 ** -150

    def dW(self, G, s, out):
        return super().dW(G, s, out) + torch.finfo(out).smallest_normal * torch.finfo(out).eps / 2 + 80 * 2.0 ** -150


@pytest.mark.parametrize("T", [20, 600])
@pytest.mark.parametrize("shift", [-114, -100, 114, 118])
def test_magnitudes_near_the_ends_of_bf16(T, shift):
    """W times 2^shift and h times 2^-shift; gradients within the bounds of any magnitude."""
    _, h, W, y = make(T, 64, 700, BF, seed=14)
    h, W = torch.ldexp(h.float(), torch.tensor(-shift)).to(BF), torch.ldexp(W.float(), torch.tensor(shift)).to(BF)
    yg, hg, Wg = gpu(y, h, W)
    _, stats, _, _ = token_logprobs(yg, hg, Wg)
    for g in (1.0, 2.0 ** -20):
        dh, dW = token_logprobs_bwd(yg, hg, Wg, stats, torch.full((T,), g, device="cuda"))
        assert torch.isfinite(dh).all() and torch.isfinite(dW).all()
        check_grads(Tiny(h, W), oh.token_logprobs_grad(y[:, None], h, W, np.full((T, 1), g)), np.full(T, g), dh, dW)


# ---------------------------------------------------------------- rows that are not numbers
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("V", [5, 128, 1024])
def test_rows_that_are_not_numbers_have_no_statistics(dtype, T, V):
    """NaN, not minus infinity, whether or not the vocabulary fills its last block of columns."""
    _, h, W, y = make(T, 64, V, dtype, seed=26)
    h[T // 2] = float("nan")
    hg, Wg, yg = gpu(h, W, y)
    for K in (0, 3):
        logp, stats, _, _ = token_logprobs(yg, hg, Wg, top_k=K)
        assert torch.isnan(stats[:, T // 2]).all() and torch.isnan(logp[T // 2])
        assert torch.isfinite(stats).sum() == 2 * (T - 1) and torch.isfinite(logp).sum() == T - 1
    _, stats = topk_distill_fwd(yg, yg[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), hg, Wg)
    assert torch.isnan(stats[:, T // 2]).all()


# ---------------------------------------------------------------- alternatives
@pytest.mark.parametrize("T", [1, 70, 200])
@pytest.mark.parametrize("spread", [1.0, 2.0, 3.0, 8.0])
def test_alternatives_of_rows_of_every_spread(T, spread):
    """From flat rows to rows of which only a handful of logits lie within 16 of the largest."""
    rng, h, W, y = make(T, 128, 6000, BF, seed=22)
    h = (h.float() * spread).to(BF)
    ids = np.stack([y, rng.integers(0, 6000, size=T)], axis=1).astype(np.int32)
    hg, Wg, ig = gpu(h, W, ids)
    b = Bounds(h, W)
    r = oh.token_logprobs(ids, h, W)
    for K in (2, 64):
        logp, stats, top, top_logp = token_logprobs(ig, hg, Wg, top_k=K)
        check_top(top, top_logp, h, W, K, b)
        within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
        within(stats[1], r["entropy"], b.entropy(r["entropy"]), "entropy")
        within(logp, r["logp"], b.logp(r["lse"])[:, None] * np.ones((1, 2)) + 2.0 ** -22 * np.abs(r["logp"]), "logp")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("V,K", [(5, 5), (90, 64), (3000, 20), (3000, 64), (130, 64)])
@pytest.mark.parametrize("spread", [1.0, 8.0])
def test_logits_that_are_not_numbers_are_no_alternatives(dtype, T, V, K, spread):
    """The K largest of those that are, then -1 and NaN."""
    rng, h, W, _ = make(T, 64, V, dtype, seed=23)
    h = (h.float() * spread).to(dtype)
    gone = np.zeros(V, dtype=bool)
    gone[rng.choice(V, size=3 if V < 3000 else 400, replace=False)] = True
    if V == 130:
        gone[5:120] = True
    if V == 3000:
        gone[256:512] = True                              # whole splits
    W[torch.from_numpy(gone)] = float("nan")
    hg, Wg = gpu(h, W)
    hg = torch.cat([hg, torch.full_like(hg[:1], float("nan"))])
    _, stats, top, top_logp = token_logprobs(None, hg, Wg, top_k=K)
    l = oh.head_logits(h, W)
    l[:, gone] = -np.inf
    order = np.argsort(-l, axis=1, kind="stable")[:, :K]
    have = min(K, int((~gone).sum()))
    order[:, have:] = -1
    np.testing.assert_array_equal(top.cpu().numpy()[:T], order)
    assert (top[T] == -1).all()                           # a row that is no number has none
    assert torch.isnan(top_logp).all() and torch.isnan(stats).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_alternatives_that_differ_in_the_last_bits(dtype, T):
    """More near-equal logits about the K-th than the fp32 sums can tell apart: the order is that of the products in
    64 bits, lower ids first where those are equal."""
    rng = np.random.Generator(np.random.PCG64(21))
    D, V, n = 512, 5000, 60
    W = rng.normal(size=(V, D)) * 0.05
    ids = rng.choice(V, size=n, replace=False)
    W = torch.from_numpy(W.astype(np.float32)).to(BF)
    # the same values in other orders: with equal entries of h the sums are equal, the fp32 ones hardly ever
    row = (np.abs(rng.normal(size=D)) * 2.0 ** rng.uniform(-14, 1, size=D)).astype(np.float32)
    W[ids] = torch.from_numpy(np.stack([rng.permutation(row) for _ in range(n)])).to(BF)
    h = torch.from_numpy(np.outer(1.0 + np.arange(T) % 3, np.ones(D)).astype(np.float32)).to(BF)
    # of one row in two, three entries are a bit off: so are the sums, by the values that meet them
    h[1::2, :3] = 2.0 ** -7 + h[1::2, :3]
    h, W = h.to(dtype), W.to(dtype)
    hg, Wg = gpu(h, W)
    b, r = Bounds(h, W), oh.token_logprobs(None, h, W)
    for K in (1, 7, 33, 60, 64):
        _, stats, top, logp = token_logprobs(None, hg, Wg, top_k=K)
        check_top(top, logp, h, W, K, b)
        within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
        within(stats[1], r["entropy"], b.entropy(r["entropy"]), "entropy")


def test_more_logits_in_doubt_than_are_ranked_again():
    """Equal rows of W past the 640 that are: their fp32 sums are equal too, so the lower ids come first all the same."""
    rng = np.random.Generator(np.random.PCG64(27))
    _, h, W, _ = make(50, 128, 3000, BF, seed=27)
    W[torch.from_numpy(rng.choice(3000, size=900, replace=False))] = (h.float().mean(0) * 2).to(BF)
    hg, Wg = gpu(h, W)
    for K in (1, 64):
        _, _, top, logp = token_logprobs(None, hg, Wg, top_k=K)
        check_top(top, logp, h, W, K, Bounds(h, W))


# ---------------------------------------------------------------- logits as low as a mask's
def masked(T, D, V, dtype, value, seed=31):
    """A column of h that is 1 and, in W, 0 or `value`: the vocabulary's entries that a program masks in this way."""
    rng, h, W, y = make(T, D, V, dtype, seed=seed)
    gone = np.zeros(V, dtype=bool)
    gone[32:64] = gone[300:512] = gone[V - 50:] = True
    gone[rng.choice(V, size=V // 10, replace=False)] = True
    y = np.where(gone[y], np.flatnonzero(~gone)[rng.integers(0, (~gone).sum(), size=T)], y).astype(np.int32)
    h[:, -1] = 1.0
    W[:, -1] = torch.from_numpy(np.where(gone, value, 0.0).astype(np.float32)).to(dtype)
    return rng, h, W, y, gone


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 60, 140])
@pytest.mark.parametrize("value", [-1e4, -1e30, -1e37, float(torch.finfo(BF).min), -np.inf])
def test_masked_vocabulary(dtype, T, value):
    D, V, K = 64, 900, 20
    rng, h, W, y, gone = masked(T, D, V, dtype, value)
    hg, Wg, yg = gpu(h, W, y)
    keep = np.flatnonzero(~gone)
    at = np.searchsorted(keep, y)
    small = W[torch.from_numpy(keep)]
    b = Bounds(h, small)
    r = oh.token_logprobs(at[:, None], h, small, top_k=K)
    for k in (0, K):
        logp, stats, top, tlp = token_logprobs(yg, hg, Wg, top_k=k)
        within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
        within(stats[1], r["entropy"], b.entropy(r["entropy"]), "entropy")
        within(logp[:, None], r["logp"], b.logp(r["lse"])[:, None], "logp")
        if k:
            np.testing.assert_array_equal(top.cpu().numpy(), keep[r["top_ids"]])
    dh, dW = token_logprobs_bwd(yg, hg, Wg, stats, torch.ones(T, device="cuda"), torch.full((T,), 0.1, device="cuda"))
    assert not torch.isnan(dW).any()
    assert not dW[torch.from_numpy(gone).cuda()].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 60, 140])
@pytest.mark.parametrize("value", [-1e4, -1e37, float(torch.finfo(BF).min), -np.inf])
def test_masked_tokens_named(dtype, T, value):
    """A masked token among the given ones: no probability, so its entry of the gradient is its coefficient, with an
    entropy's gradient too."""
    rng, h, W, y, gone = masked(T, 64, 900, dtype, value)
    keep = np.flatnonzero(~gone)
    at = np.searchsorted(keep, y)
    small = W[torch.from_numpy(keep)]
    out = np.flatnonzero(gone)[rng.integers(0, gone.sum(), size=T)].astype(np.int32)
    ids = np.stack([y, out], axis=1)
    g = rng.normal(size=(T, 2)).astype(np.float32)
    e = np.full(T, 0.1, dtype=np.float32)
    hg, Wg, ig, gg, eg = gpu(h, W, ids, g, e)
    logp, stats, _, _ = token_logprobs(ig, hg, Wg)
    assert (logp[:, 1] < -9e3).all()
    b = Bounds(h, small)
    G = oh.token_logprobs_grad(at[:, None], h, small, g[:, :1], e)
    G -= np.exp(oh.log_softmax(b.h @ b.W.T)[0]) * g[:, 1:].astype(np.float64)
    s = np.maximum(np.abs(g).max(1), np.abs(g.astype(np.float64).sum(1)))
    _, dW = token_logprobs_bwd(ig, hg, Wg, stats, gg, eg)
    check_grads(b, G, s, None, dW[torch.from_numpy(keep).cuda()])
    exp = np.zeros(W.shape)
    np.add.at(exp, out, g[:, 1:].astype(np.float64) * b.h)
    size = np.zeros(W.shape)
    np.add.at(size, out, np.abs(g[:, 1:].astype(np.float64) * b.h))
    # the coefficient in fp16, h's copy, the sums
    within(dW[torch.from_numpy(gone).cuda()], exp[gone], (size * (2.0 ** -11 + 2.0 ** -24 + b._sum(T)))[gone] +
           2.0 ** -37 * s.max() * np.abs(b.h).max() * T, "dW of masked tokens")


# ---------------------------------------------------------------- widths and exact rows
@pytest.mark.parametrize("D", [2304, 4352, 8192])
@pytest.mark.parametrize("T", [1, 70, 150])
def test_the_widths_of_the_larger_exits(D, T):
    rng, h, W, y = make(T, D, 2000, BF, seed=24)
    hg, Wg, yg = gpu(h, W, y)
    b = Bounds(h, W)
    r = oh.token_logprobs(y[:, None], h, W)
    logp, stats, _, _ = token_logprobs(yg, hg, Wg)
    within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
    within(stats[1], r["entropy"], b.entropy(r["entropy"]), "entropy")
    within(logp[:, None], r["logp"], b.logp(r["lse"])[:, None], "logp")
    _, _, top, top_logp = token_logprobs(None, hg, Wg, top_k=20)
    check_top(top, top_logp, h, W, 20, b)
    g = rng.normal(size=(T, 1)).astype(np.float32)
    dh, dW = token_logprobs_bwd(yg, hg, Wg, stats, gpu(g)[0][:, 0].contiguous())
    check_grads(b, oh.token_logprobs_grad(y[:, None], h, W, g), np.abs(g[:, 0]), dh, dW)


@pytest.mark.parametrize("D", [64, 2304, 4352, 65536])
@pytest.mark.parametrize("T", [1, 128, 129])
def test_rows_whose_sums_are_exact(D, T):
    """h with one entry a row, and h and W of small whole numbers: no addition rounds or truncates, so what is left
    is the correction for truncation that did not happen: D 2^-30 of a logit (the fp32 log-sum-exp and the exponentials:
    2^-20 as everywhere)."""
    rng = np.random.Generator(np.random.PCG64(25))
    V = 300
    for kind in ("one", "whole"):
        W = rng.integers(-8, 9, size=(V, D)) / 4.0
        h = np.zeros((T, D))
        if kind == "one":
            h[np.arange(T), rng.integers(0, D, size=T)] = rng.integers(1, 33, size=T)
        else:
            at = rng.integers(0, D, size=(T, 6))
            h[np.arange(T)[:, None], at] = rng.integers(-3, 4, size=(T, 6))
        h, W = torch.from_numpy(h).to(BF), torch.from_numpy(W).to(BF)
        l = oh.head_logits(h, W)
        logq, lse = oh.log_softmax(l)
        ids = np.argsort(-l, axis=1, kind="stable")[:, [0, V // 2]].astype(np.int32)
        hg, Wg, ig = gpu(h, W, ids)
        logp, stats, _, _ = token_logprobs(ig, hg, Wg)
        off = D * 2.0 ** -30 * np.abs(l).max(axis=1) + 2.0 ** -20 * (1 + np.abs(lse))
        within(stats[0], lse, off, kind + " lse")
        exp = np.take_along_axis(logq, ids, axis=1)
        within(logp, exp, (2 * off)[:, None] + 2.0 ** -22 * np.abs(exp), kind + " logp")


# ---------------------------------------------------------------- refusals
def test_empty_status_is_refused():
    _, h, W, y = make(4, 64, 100, BF)
    hg, Wg, yg = gpu(h, W, y)
    ids, z = yg[:, None].contiguous(), torch.zeros(4, 1, device="cuda")
    logp, stats, _, _ = token_logprobs(yg, hg, Wg)
    _, dstats = topk_distill_fwd(yg, ids, z, hg, Wg)
    words = torch.zeros(4, dtype=torch.int32, device="cuda")
    for status in (words[1:1], torch.zeros(0, dtype=torch.int32, device="cuda")):
        for call in (lambda: token_logprobs(yg, hg, Wg, status=status),
                     lambda: token_logprobs_bwd(yg, hg, Wg, stats, logp, status=status),
                     lambda: topk_distill_fwd(yg, ids, z, hg, Wg, status=status),
                     lambda: topk_distill_bwd(yg, ids, z, hg, Wg, dstats, status=status)):
            with pytest.raises(ValueError):
                call()
