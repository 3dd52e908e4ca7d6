"""Inputs and error bounds for the single-exit LM-head operators.

Bounds (derived, not fitted), with n = D / 16 sequential adds of a tensor-core
accumulation whose additions may truncate (one unit in the last place, 2^-23,
of a partial sum each; a partial sum is at most sum_i |h_i w_i|):
  logits     dl_t = (n + 32) 2^-23 max_v sum_i |h_ti W_vi|  (+32: the products
             of one step among themselves); the CUDA-core path adds D times with
             half that error each: (D / 2 + 32) 2^-23
  lse        dl_t + 2^-20 (1 + |lse|): exp and log to a few units in the last
             place, sums of V terms in a tree of 128-wide pieces
  logp       2 dl_t + the same
  entropy    its derivative is -q (log q + H): 2 (H + 1) dl_t + 2^-18 (1 + H)
  gradients  with s_t the row's largest coefficient, G_tv = s_t (q (A + B log q) + entries)
             where |A| <= 12 and |B| <= 1 (12: 1 + the largest entropy here).
             The dense term is off by the errors of l and exp, 2 dl_t + 2^-19,
             on s_t (12 q + q |log q|): on its own size, not on that of its
             difference to the entries, which can cancel.  G' is rounded to fp16:
             2^-11 relative, 2^-25 s_t below fp16's normal range (fp32 path: a
             few units, 2^-22 s_t (12 q + q |log q|), instead).
             W and h are copied to fp16: exact but for values below fp16's normal
             range, off by 2^-25 of the copy, whose largest value M lies in
             [2^-6, 2^15) or is brought to [2^13, 2^14) (then 2^-38 of it is
             that).  For W that is on sum_v |G_tv|.  h is copied times
             2^14 s_t / b, with b at most twice the largest s_t |h_ti|, and meets
             G / s_t, with the kernel's s_t more than half the one here:
             2 2^-39 2 s_max max |h| on sum_t |G_tv| / s_t.
             Summed over k = V or T terms
             (k / 16 + 32) 2^-23; the outputs rounded by half a unit (2^-8 bf16,
             2^-24 fp32).
"""
import numpy as np
import torch

from oracle import head as oh


def make(T, D, V, dtype, seed=0, lean=4.0):
    """h and W (CPU tensors of dtype) with logits that spread by about 2, every token leaning towards one row by a
    random amount; y the rows leant to."""
    rng = np.random.Generator(np.random.PCG64(seed))
    W = torch.from_numpy((rng.normal(size=(V, D)) * 2.0 / np.sqrt(D)).astype(np.float32)).to(dtype)
    y = rng.integers(0, V, size=T)
    h = rng.normal(size=(T, D)) + rng.uniform(0, lean, size=(T, 1)) * W.double().numpy()[y]
    return rng, torch.from_numpy(h.astype(np.float32)).to(dtype), W, y.astype(np.int32)


class Bounds:
    def __init__(self, h, W):
        self.bf16 = h.dtype == torch.bfloat16
        self.h, self.W = h.double().numpy(), W.double().numpy()
        T, D = self.h.shape
        steps = D / 16 + 32 if self.bf16 else D / 2 + 32
        self.dl = steps * 2.0 ** -23 * (np.abs(self.h) @ np.abs(self.W).T).max(axis=1)

    def lse(self, lse):
        return self.dl + 2.0 ** -20 * (1 + np.abs(lse))

    def logp(self, lse):
        return 2 * self.dl + 2.0 ** -20 * (1 + np.abs(lse))

    def entropy(self, H):
        return 2 * (H + 1) * self.dl + 2.0 ** -18 * (1 + H)

    def _g(self, G, s):
        """Error of every entry of G; s: the row's largest coefficient."""
        logq, _ = oh.log_softmax(self.h @ self.W.T)
        q = np.exp(logq)
        dense = s[:, None] * (12 * q + q * np.abs(logq))
        e = (2 * self.dl + 2.0 ** -19)[:, None] * dense
        return e + (2.0 ** -11 * np.abs(G) + 2.0 ** -25 * s[:, None] if self.bf16 else 2.0 ** -22 * dense)

    def _sum(self, k):
        return (k / 16 + 32 if self.bf16 else k / 2 + 32) * 2.0 ** -23

    def dh(self, G, s, out):
        most = np.abs(self.W).max()
        copy = (2.0 ** -25 if 2.0 ** -6 <= most < 2.0 ** 15 else 2.0 ** -38 * most) * np.abs(G).sum(axis=1, keepdims=True)
        return (self._g(G, s) @ np.abs(self.W) + self._sum(G.shape[1]) * (np.abs(G) @ np.abs(self.W)) +
                (copy if self.bf16 else 0.0) + half_step(out) * np.abs(G @ self.W))

    def dW(self, G, s, out):
        rows = (np.abs(G) / np.maximum(s, 1e-300)[:, None]).sum(axis=0)[:, None]
        copy = 2 * 2.0 ** -39 * 2 * s.max() * np.abs(self.h).max() * rows
        return (self._g(G, s).T @ np.abs(self.h) + self._sum(G.shape[0]) * (np.abs(G).T @ np.abs(self.h)) +
                (copy if self.bf16 else 0.0) + half_step(out) * np.abs(G.T @ self.h))


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, exp, bound, name):
    got = got.detach().double().cpu().numpy()
    assert got.shape == exp.shape, (name, got.shape, exp.shape)
    bad = ~(np.abs(got - exp) <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} outside; worst "
                           f"{np.nanmax(np.abs(got - exp) / np.maximum(bound, 1e-300)):.3g} of the bound at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {exp[bad][0]}")


def check_grads(b, G, s, dh, dW):
    s = s.astype(np.float64)
    if dh is not None:
        within(dh, G @ b.W, b.dh(G, s, dh.dtype) + 1e-300, "dh")
    if dW is not None:
        within(dW, G.T @ b.h, b.dW(G, s, dW.dtype) + 1e-300, "dW")


def check_top(top_ids, top_logp, h, W, K, b):
    """Exact order by products in 64 bits, lower ids first among equal ones."""
    l = oh.head_logits(h, W)
    logq, lse = oh.log_softmax(l)
    order = np.argsort(-l, axis=1, kind="stable")[:, :K]
    np.testing.assert_array_equal(top_ids.cpu().numpy(), order)
    within(top_logp, np.take_along_axis(logq, order, axis=1), b.logp(lse)[:, None] * np.ones((1, K)), "top_logp")
