"""Single-exit LM-head operators on the GPU against the 64-bit oracle: types,
ragged sizes, absent and repeated tokens, workspaces from the smallest up,
streams, captured graphs, and a run of them together."""
import numpy as np
import pytest
import torch

from lm_head_loss_junction_b200 import (new_status, status_read, token_logprobs, token_logprobs_bwd,
                                        token_logprobs_bwd_workspace, token_logprobs_workspace, topk_distill_bwd,
                                        topk_distill_fwd, topk_distill_workspace)
from oracle import head as oh
from tests.head_helpers import Bounds, check_grads, check_top, make, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [  # T, D, V, dtype
    (1, 64, 1, BF), (1, 64, 300, BF), (2, 128, 127, BF), (3, 64, 128, BF), (5, 192, 129, BF), (33, 320, 1000, BF),
    (128, 64, 256, BF), (130, 512, 2049, BF), (256, 128, 5000, BF), (257, 256, 513, BF), (600, 64, 3333, BF),
    (1, 1024, 20011, BF), (24, 640, 9001, BF),
    (1, 1, 1, F32), (1, 7, 33, F32), (65, 64, 512, F32), (130, 33, 200, F32), (256, 192, 512, F32),
]


def gpu(*ts):
    return [t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in ts]


def some_ids(rng, T, V, N):
    """Given tokens: some absent, some repeated inside a row, the first and last of the vocabulary among them."""
    ids = rng.integers(0, V, size=(T, N)).astype(np.int32)
    ids[rng.random((T, N)) < 0.2] = -1
    ids[0, 0] = V - 1
    if N > 1:
        ids[:, 1] = np.where(rng.random(T) < 0.5, ids[:, 0], ids[:, 1])
    if T > 1:
        ids[1, :] = -1
        ids[-1, 0] = 0
    return ids


@pytest.mark.parametrize("T,D,V,dtype", SHAPES)
@pytest.mark.parametrize("N,K", [(1, 0), (3, 0), (64, 0), (1, 1), (2, 9), (0, 64)])
def test_scores(T, D, V, dtype, N, K):
    K = min(K, V)
    rng, h, W, _ = make(T, D, V, dtype, seed=T + V)
    ids = some_ids(rng, T, V, N) if N else None
    hg, Wg = gpu(h, W)
    st = new_status()
    logp, stats, top_ids, top_logp = token_logprobs(gpu(ids)[0] if N else None, hg, Wg, top_k=K, status=st)
    assert status_read(st)[0] == 0
    r = oh.token_logprobs(ids, h, W)
    b = Bounds(h, W)
    within(stats[0], r["lse"], b.lse(r["lse"]), "lse")
    within(stats[1], r["entropy"], b.entropy(r["entropy"]), "entropy")
    if N:
        within(logp, r["logp"], b.logp(r["lse"])[:, None] * (ids >= 0), "logp")
    if K:
        check_top(top_ids, top_logp, h, W, K, b)
    else:
        assert top_ids is None and top_logp is None


@pytest.mark.parametrize("T,D,V,dtype", SHAPES)
@pytest.mark.parametrize("N,entropy,dW_dtype", [(1, True, F32), (4, False, BF), (64, True, BF)])
def test_score_gradients(T, D, V, dtype, N, entropy, dW_dtype):
    rng, h, W, _ = make(T, D, V, dtype, seed=2 * T + V)
    ids = some_ids(rng, T, V, N)
    # rows of very different weight, and gradients of absent tokens that are not numbers
    g = (rng.normal(size=(T, N)) * 10.0 ** rng.uniform(-6, 0, size=(T, 1))).astype(np.float32)
    ge = (rng.normal(size=T) * 0.1).astype(np.float32) * (rng.random(T) < 0.7) if entropy else None
    G = oh.token_logprobs_grad(ids, h, W, g, ge)
    g[ids < 0] = np.nan
    ig, hg, Wg, gg = gpu(ids, h, W, g)
    geg = gpu(ge.astype(np.float32))[0] if entropy else None
    st = new_status()
    _, stats, _, _ = token_logprobs(ig, hg, Wg, status=st)
    dh, dW = token_logprobs_bwd(ig, hg, Wg, stats, gg, geg, dW_dtype=dW_dtype if dtype == BF else F32, status=st)
    assert status_read(st)[0] == 0
    gz = np.where(ids >= 0, np.nan_to_num(g), 0.0)
    s = np.maximum(np.abs(gz.sum(1)), np.abs(gz).max(1))
    if entropy:
        s = np.maximum(s, np.abs(ge))
    check_grads(Bounds(h, W), G, s, dh, dW)


def some_teacher(rng, T, V, K, y):
    """Teacher lists: absent tokens with logits that are not numbers, rows with none, rows of -infinity or of the
    lowest value, repeated ids, the target among them."""
    ids = rng.integers(0, V, size=(T, K)).astype(np.int32)
    z = (rng.normal(size=(T, K)) * 3 + 10).astype(np.float32)
    ids[:, 0] = np.where(rng.random(T) < 0.5, y, ids[:, 0])
    if K > 1:
        ids[:, 1] = np.where(rng.random(T) < 0.3, ids[:, 0], ids[:, 1])
    gone = rng.random((T, K)) < 0.2
    if T > 2:
        gone[2] = True
    ids[gone] = -1
    z[gone] = rng.choice([np.nan, np.inf, -np.inf], size=int(gone.sum()))
    if T > 5:
        z[3] = -np.inf
        z[4] = np.finfo(np.float32).min
        z[5, K // 2:] = np.finfo(np.float32).min
    return ids, z


def coefficients(r_G, y, tid, z, w, alpha, T, V):
    p, _, some = oh.teacher_probs(tid, z, V)
    wg = np.abs(np.ones(T) if w is None else w.astype(np.float64)) / T
    return wg * np.maximum((1 - alpha) + alpha * some, np.maximum(1 - alpha, alpha * p.max(1)))


@pytest.mark.parametrize("T,D,V,dtype", SHAPES)
@pytest.mark.parametrize("K,alpha,weighted,dW_dtype", [(1, 0.3, False, F32), (8, 0.3, True, BF), (64, 1.0, True, F32),
                                                       (5, 0.0, False, BF)])
def test_distillation(T, D, V, dtype, K, alpha, weighted, dW_dtype):
    rng, h, W, y = make(T, D, V, dtype, seed=3 * T + V)
    tid, z = some_teacher(rng, T, V, K, y)
    w = None
    if weighted:
        w = rng.uniform(0.1, 2.0, size=T).astype(np.float32)
        w[rng.random(T) < 0.3] = 0.0
        y = np.where((w == 0) & (rng.random(T) < 0.5), -7, y).astype(np.int32)     # padding: any target
    scale = 2.5
    r = oh.topk_distill(y, tid, z, h, W, alpha, w, grad_scale=scale)
    yg, tg, zg, hg, Wg = gpu(y, tid, z, h, W)
    wg = gpu(w)[0] if weighted else None
    st = new_status()
    losses, stats = topk_distill_fwd(yg, tg, zg, hg, Wg, alpha, token_weights=wg, status=st)
    dh, dW = topk_distill_bwd(yg, tg, zg, hg, Wg, stats, alpha, scale, token_weights=wg,
                              dW_dtype=dW_dtype if dtype == BF else F32, status=st)
    assert status_read(st)[0] == 0
    b = Bounds(h, W)
    lse = r["stats"][0]
    within(stats[0], lse, b.lse(lse), "lse")
    within(stats[1], r["stats"][1], b.logp(lse), "ce")
    within(stats[2], r["stats"][2], b.logp(lse) + 2.0 ** -20 * np.abs(r["stats"][2]), "kd")
    ww = np.ones(T) if w is None else w
    tol = np.mean(ww * (b.logp(lse) + 2.0 ** -19 * (1 + r["stats"][1:].max(0))))
    within(losses, r["losses"], np.full(3, tol), "losses")
    check_grads(b, r["G"], scale * coefficients(r["G"], y, tid, z, w, alpha, T, V), dh, dW)


def _distill_inputs(T, D, V, K, seed=0, dtype=BF):
    rng, h, W, y = make(T, D, V, dtype, seed=seed)
    tid, z = some_teacher(rng, T, V, K, y)
    return [y, tid, z, h, W], gpu(y, tid, z, h, W)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_workspaces_from_the_smallest_up(dtype):
    """Pieces of any size give the results of one piece: bitwise where only tokens are split, within rounding where
    dh is summed over chunks of the vocabulary."""
    T, D, V, K = 600, 64, 2500, 6
    _, (y, tid, z, h, W) = _distill_inputs(T, D, V, K, dtype=dtype)
    f_b, f_min, b_b, b_min = topk_distill_workspace(T, D, V, K, dtype)
    s_b, s_min = token_logprobs_workspace(T, D, V, 1, 7, dtype)
    ref = topk_distill_fwd(y, tid, z, h, W)
    ref_s = token_logprobs(y, h, W, top_k=7)
    for n in {f_min, (f_min + f_b) // 2, f_b, f_b + 4096}:
        got = topk_distill_fwd(y, tid, z, h, W, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for n in {s_min, (s_min + s_b) // 2, s_b + 64}:
        got = token_logprobs(y, h, W, top_k=7, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, ref_s))
    dh, dW = topk_distill_bwd(y, tid, z, h, W, ref[1])
    for n in {b_min, (3 * b_min + b_b) // 4, (b_min + b_b) // 2, b_b + 64}:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        dh2, dW2 = topk_distill_bwd(y, tid, z, h, W, ref[1], workspace=ws)
        scale = dh.float().abs().max()
        assert (dh2.float() - dh.float()).abs().max() <= 2.0 ** -7 * scale
        assert (dW2 - dW).abs().max() <= 2.0 ** -16 * dW.abs().max()
    with pytest.raises(RuntimeError):
        topk_distill_bwd(y, tid, z, h, W, ref[1], workspace=torch.empty(b_min - 1, dtype=torch.uint8, device="cuda"))


def test_chunked_backward_matches_the_oracle():
    T, D, V, K = 300, 128, 3000, 4
    (y, tid, z, h, W), g = _distill_inputs(T, D, V, K, seed=5)
    _, stats = topk_distill_fwd(*g)
    _, _, _, b_min = topk_distill_workspace(T, D, V, K, BF)
    for dW_dtype in (F32, BF):
        dh, dW = topk_distill_bwd(*g, stats, dW_dtype=dW_dtype,
                                  workspace=torch.empty(b_min, dtype=torch.uint8, device="cuda"))
        r = oh.topk_distill(y, tid, z, h, W, 0.3)
        check_grads(Bounds(h, W), r["G"], coefficients(r["G"], y, tid, z, None, 0.3, T, V), dh, dW)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_accumulated_and_single_gradients(dtype):
    T, D, V, K = 140, 64, 700, 3
    _, (y, tid, z, h, W) = _distill_inputs(T, D, V, K, dtype=dtype)
    _, stats = topk_distill_fwd(y, tid, z, h, W)
    dh, dW = topk_distill_bwd(y, tid, z, h, W, stats)
    base = torch.randn_like(dW)
    acc = base.clone()
    topk_distill_bwd(y, tid, z, h, W, stats, dW=acc, accumulate_dW=True)
    assert torch.allclose(acc, base + dW, rtol=0, atol=2.0 ** -23 * float((base.abs() + dW.abs()).max()))
    only_dh, none = topk_distill_bwd(y, tid, z, h, W, stats, want_dW=False)
    assert none is None and torch.equal(only_dh, dh)
    none, only_dW = topk_distill_bwd(y, tid, z, h, W, stats, want_dh=False)
    assert none is None and torch.equal(only_dW, dW)


@pytest.mark.parametrize("T", [140, 600])
def test_one_gradient_alone_equals_both(T):
    """With the fp16 copies in a kernel of their own (few tokens) and beside the gradient's."""
    _, x = _distill_inputs(T, 128, 1300, 5, seed=6)
    _, stats = topk_distill_fwd(*x)
    dh, dW = topk_distill_bwd(*x, stats, dW_dtype=BF)
    assert torch.equal(topk_distill_bwd(*x, stats, want_dW=False)[0], dh)
    assert torch.equal(topk_distill_bwd(*x, stats, want_dh=False, dW_dtype=BF)[1], dW)


@pytest.mark.parametrize("T", [20, 140, 600])
@pytest.mark.parametrize("shift", [-60, -18, 18, 60])
def test_magnitudes_outside_fp16(T, shift):
    """W times 2^shift and h times 2^-shift have the same logits; their fp16 copies need a scale of their own."""
    _, h, W, y = make(T, 128, 900, BF, seed=4)
    h, W = torch.ldexp(h.float(), torch.tensor(-shift)).to(BF), torch.ldexp(W.float(), torch.tensor(shift)).to(BF)
    yg, hg, Wg = gpu(y, h, W)
    tid = yg[:, None].repeat(1, 2)
    z = torch.zeros(T, 2, device="cuda")
    _, stats = topk_distill_fwd(yg, tid, z, hg, Wg, 0.5)
    dh, dW = topk_distill_bwd(yg, tid, z, hg, Wg, stats, 0.5, 3.0)
    r = oh.topk_distill(y, tid.cpu().numpy(), z.cpu().numpy(), h, W, 0.5, grad_scale=3.0)
    check_grads(Bounds(h, W), r["G"], np.full(T, 3.0 / T), dh, dW)


def test_views_of_fp32_rows():
    """fp32 rows of odd width start at any 4-byte boundary."""
    rng, h, W, y = make(40, 7, 90, F32, seed=8)
    hg, Wg, yg = gpu(h, W, y)
    whole = token_logprobs(yg, hg, Wg, top_k=3)
    part = token_logprobs(yg[3:], hg[3:], Wg, top_k=3)
    assert torch.equal(whole[0][3:], part[0]) and torch.equal(whole[2][3:], part[2])
    dh, dW = token_logprobs_bwd(yg[3:], hg[3:], Wg, part[1], torch.ones(37, device="cuda"))
    G = oh.token_logprobs_grad(y[3:, None], h[3:], W, np.ones((37, 1)))
    check_grads(Bounds(h[3:], W), G, np.ones(37), dh, dW)


def test_host_threads_at_once():
    """Calls of several host threads, on a stream each and with shapes of their own."""
    import threading
    shapes = [(200, 64, 700, 4), (30, 128, 40000, 9), (300, 64, 2000, 33), (140, 128, 300, 1)]
    data = [_distill_inputs(T, D, V, K, seed=20 + K)[1] for T, D, V, K in shapes]

    def work(i):
        x = data[i]
        K = shapes[i][3]
        losses, stats = topk_distill_fwd(*x)
        return [losses, stats, *topk_distill_bwd(*x, stats), *token_logprobs(x[0], x[3], x[4], top_k=K)]

    ref = [work(i) for i in range(len(shapes))]
    torch.cuda.synchronize()
    got, errors = [None] * len(shapes), []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = work(i)
            s.synchronize()
        except Exception as e:                                   # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for r, g in zip(ref, got):
        assert all(torch.equal(a, b) for a, b in zip(r, g))


def test_offsets_past_32_bits():
    """One piece of more than 2^32 bytes of logits and 2^31 gradient entries equals pieces of it."""
    T, D, V = 45056, 64, 50021
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn(V, D, generator=g, device="cuda").to(BF) * 0.25
    h = torch.randn(T, D, generator=g, device="cuda").to(BF)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ref = token_logprobs(ids, h, W, top_k=2)
    # [partial statistics, 16 bytes per token and split][fp32 logits of all tokens]
    big = torch.empty(T * (V // 128 + 1) * 16 + T * ((V + 63) // 64 * 64) * 4 + 4096, dtype=torch.uint8, device="cuda")
    got = token_logprobs(ids, h, W, top_k=2, workspace=big)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    grad = torch.ones(T, device="cuda") / T
    dh, dW = token_logprobs_bwd(ids, h, W, ref[1], grad, dW_dtype=BF, workspace=big)
    dh2, dW2 = token_logprobs_bwd(ids, h, W, ref[1], grad, dW_dtype=BF)
    assert torch.equal(dW, dW2)                       # a chunk of columns or all of them: the same sums over tokens
    assert (dh.float() - dh2.float()).abs().max() <= 2.0 ** -7 * dh.float().abs().max()
    # the last rows against the definition
    l = h[-4:].double() @ W.double().T
    q = torch.softmax(l, 1)
    q[torch.arange(4), ids[-4:].long()] -= 1
    exp = (-q @ W.double()) / T
    assert (dh[-4:].double() - exp).abs().max() <= 2.0 ** -7 * exp.abs().max()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_logits_rank_by_id(dtype):
    """Repeated rows of W tie exactly; so does a head of zeros."""
    rng, h, W, _ = make(70, 64, 900, dtype)
    W = W[torch.from_numpy(rng.integers(0, 40, size=900))]
    hg, Wg = gpu(h, W)
    for K in (1, 20, 64):
        _, _, top, logp = token_logprobs(None, hg, Wg, top_k=K)
        check_top(top, logp, h, W, K, Bounds(h, W))
    _, stats, top, _ = token_logprobs(None, hg, torch.zeros_like(Wg), top_k=64)
    assert torch.equal(top.cpu(), torch.arange(64, dtype=torch.int32).expand(70, 64))
    assert torch.allclose(stats.cpu(), torch.full((2, 70), float(np.log(900.0))), rtol=2e-6)


def test_order_does_not_depend_on_the_batch():
    """One token alone, in a batch, and at another place of it gets the same alternatives."""
    _, h, W, _ = make(300, 256, 7000, BF, seed=9)
    hg, Wg = gpu(h, W)
    _, _, top, _ = token_logprobs(None, hg, Wg, top_k=40)
    for t in (0, 131, 299):
        _, _, alone, _ = token_logprobs(None, hg[t:t + 1], Wg, top_k=40)
        assert torch.equal(alone[0], top[t])
    _, _, turned, _ = token_logprobs(None, hg.flip(0).contiguous(), Wg, top_k=40)
    assert torch.equal(turned.flip(0), top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ids_outside_the_vocabulary_are_reported(dtype):
    T, D, V, K = 20, 64, 150, 3
    (y, tid, z, h, W), (yg, tg, zg, hg, Wg) = _distill_inputs(T, D, V, K, dtype=dtype)
    bad = tg.clone()
    bad[7, 1] = V
    bad[8, 0] = -2
    st = new_status()
    logp, stats, _, _ = token_logprobs(bad, hg, Wg, status=st)
    assert status_read(st)[0] == 5
    assert logp[7, 1] == 0 and logp[8, 0] == 0
    dh, dW = token_logprobs_bwd(bad, hg, Wg, stats, torch.ones_like(logp), status=st)
    assert status_read(st)[0] == 5
    absent = torch.where((bad < 0) | (bad >= V), -1, bad)
    dh2, dW2 = token_logprobs_bwd(absent, hg, Wg, stats, torch.ones_like(logp), status=st)
    assert status_read(st)[0] == 0
    assert torch.equal(dh, dh2) and torch.equal(dW, dW2)
    # a target outside the vocabulary: the token counts nowhere, as if its weight were 0
    yb = yg.clone()
    yb[4] = V + 3
    w = torch.ones(T, device="cuda")
    losses, stats = topk_distill_fwd(yb, tg, zg, hg, Wg, status=st)
    assert status_read(st)[0] == 5
    dh, dW = topk_distill_bwd(yb, tg, zg, hg, Wg, stats, status=st)
    assert status_read(st)[0] == 5
    w[4] = 0
    losses2, stats2 = topk_distill_fwd(yb, tg, zg, hg, Wg, token_weights=w, status=st)
    dh2, dW2 = topk_distill_bwd(yb, tg, zg, hg, Wg, stats2, token_weights=w, status=st)
    assert status_read(st)[0] == 0
    assert torch.equal(losses, losses2)
    assert torch.equal(dh, dh2) and torch.equal(dW, dW2)
    assert not dh[4].any() and stats[1, 4] == 0 and stats[2, 4] == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_rows_of_any_content_change_nothing(dtype):
    """Tokens of weight 0 hold NaN; losses and gradients are those of the other tokens."""
    T, D, V, K = 150, 64, 333, 4
    _, (y, tid, z, h, W) = _distill_inputs(T, D, V, K, dtype=dtype)
    w = torch.ones(T, device="cuda")
    w[40:60] = 0
    l0, s0 = topk_distill_fwd(y, tid, z, h, W, token_weights=w)
    g0 = topk_distill_bwd(y, tid, z, h, W, s0, token_weights=w)
    dirty = h.clone()
    dirty[40:60] = float("nan")
    l1, s1 = topk_distill_fwd(y, tid, z, dirty, W, token_weights=w)
    g1 = topk_distill_bwd(y, tid, z, dirty, W, s1, token_weights=w)
    assert torch.equal(l0, l1) and torch.equal(g0[0], g1[0]) and torch.equal(g0[1], g1[1])
    assert not g1[0][40:60].any()


def test_rows_that_are_not_numbers_stay_their_own():
    _, h, W, _ = make(60, 64, 3000, BF)
    hg, Wg = gpu(h, W)
    ids = torch.zeros(60, dtype=torch.int32, device="cuda")
    logp, stats, top, tlp = token_logprobs(ids, hg, Wg, top_k=30)
    hg[17] = float("nan")
    hg[18, 3] = float("inf")
    got = token_logprobs(ids, hg, Wg, top_k=30)
    keep = torch.ones(60, dtype=torch.bool, device="cuda")
    keep[17:19] = False
    assert torch.equal(got[0][keep], logp[keep]) and torch.equal(got[1][:, keep], stats[:, keep])
    assert torch.equal(got[2][keep], top[keep]) and torch.equal(got[3][keep], tlp[keep])
    assert ((got[2] >= -1) & (got[2] < 3000)).all()


def test_gradient_scales_far_apart():
    """Rows weighted 2^-40 to 2^40 keep their own relative precision."""
    T, D, V = 64, 128, 500
    rng, h, W, y = make(T, D, V, BF)
    yg, hg, Wg = gpu(y, h, W)
    _, stats, _, _ = token_logprobs(yg, hg, Wg)
    g = torch.ones(T, device="cuda")
    ref, _ = token_logprobs_bwd(yg, hg, Wg, stats, g)
    k = torch.from_numpy(rng.integers(-40, 41, size=T)).cuda()
    far = torch.ldexp(g, k)
    k = k[:, None]
    dh, _ = token_logprobs_bwd(yg, hg, Wg, stats, far)
    assert torch.equal(torch.ldexp(ref.float(), k).to(BF), dh)


def test_other_stream_and_two_calls_at_once():
    _, a = _distill_inputs(260, 128, 3000, 8, seed=1)
    _, b = _distill_inputs(200, 64, 900, 3, seed=2)
    ref = []
    for x in (a, b):
        losses, stats = topk_distill_fwd(*x)
        ref.append((losses, stats, *topk_distill_bwd(*x, stats)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = [None, None]
    for _ in range(3):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                losses, stats = topk_distill_fwd(*x)
                out[i] = (losses, stats, *topk_distill_bwd(*x, stats))
    torch.cuda.synchronize()
    for r, o in zip(ref, out):
        assert all(torch.equal(p, q) for p, q in zip(r, o))


def test_stream_argument_owns_its_buffers():
    """On a stream given by argument, as an object or a handle: outputs and workspace come from its own pool, so work
    on the current stream that reuses freed memory meanwhile does not touch them."""
    _, x = _distill_inputs(600, 128, 5000, 9, seed=40)
    losses, stats = topk_distill_fwd(*x)
    ref = [losses, stats, *topk_distill_bwd(*x, stats), *token_logprobs(x[0], x[3], x[4], top_k=7)]
    grad = token_logprobs_bwd(x[0], x[3], x[4], ref[5], torch.ones(600, device="cuda"))
    one = torch.ones(600, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        got = []
        for _ in range(10):
            l, st = topk_distill_fwd(*x, stream=stream)
            got = [l, st, *topk_distill_bwd(*x, st, stream=stream), *token_logprobs(x[0], x[3], x[4], top_k=7, stream=stream)]
            g2 = token_logprobs_bwd(x[0], x[3], x[4], got[5], one, stream=stream)
            for n in (1 << 20, 1 << 24, 1 << 27):      # what the current stream is handed out next, it overwrites
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        assert all(torch.equal(a, b) for a, b in zip(grad, g2))


@pytest.mark.parametrize("dtype,T", [(BF, 20), (BF, 140), (BF, 600), (F32, 90)])
def test_inputs_written_just_before_the_call(dtype, T):
    """The kernels of a call are set up while the one before runs: nothing they read may be from before it."""
    sets = [_distill_inputs(T, 64, 700, 5, seed=30 + i, dtype=dtype)[1] for i in range(4)]
    x = [t.clone() for t in sets[0]]
    y, tid, z, h, W = x
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def work():
        losses, stats = topk_distill_fwd(y, tid, z, h, W, workspace=ws)
        dh, dW = topk_distill_bwd(y, tid, z, h, W, stats, workspace=ws)
        return [losses, stats, dh, dW, *token_logprobs(y, h, W, top_k=6, workspace=ws)]

    ref = []
    for s in sets:
        for d, v in zip(x, s):
            d.copy_(v)
        torch.cuda.synchronize()
        ref.append([t.clone() for t in work()])
        torch.cuda.synchronize()
    for turn in range(25):
        got = []
        for s in sets:
            for d, v in zip(x, s):
                d.copy_(v)
            got.append(work())
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert all(torch.equal(a, b) for a, b in zip(r, g)), turn


def test_captured_and_replayed_with_new_inputs():
    _, x = _distill_inputs(130, 64, 700, 5, seed=3)
    _, x2 = _distill_inputs(130, 64, 700, 5, seed=4)
    y, tid, z, h, W = [t.clone() for t in x]

    def step():
        losses, stats = topk_distill_fwd(y, tid, z, h, W)
        dh, dW = topk_distill_bwd(y, tid, z, h, W, stats)
        lp = token_logprobs(y, h, W, top_k=5)
        return [losses, stats, dh, dW, *lp]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for src in (x, x2, x):
        for dst, s in zip((y, tid, z, h, W), src):
            dst.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


FIRST_CAPTURED = """
import torch
from lm_head_loss_junction_b200 import token_logprobs, token_logprobs_bwd, topk_distill_bwd, topk_distill_fwd
g = torch.Generator(device="cuda").manual_seed(0)
def data(T, D, V, K, dt):
    h = torch.randn(T, D, generator=g, device="cuda").to(dt)
    W = torch.randn(V, D, generator=g, device="cuda").to(dt)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda", dtype=torch.int32)
    return h, W, ids, torch.randn(T, K, generator=g, device="cuda")
sets = [data(*x) for x in [(20, 64, 300, 3, torch.bfloat16), (600, 128, 700, 5, torch.bfloat16), (30, 9, 70, 2, torch.float32)]]
def work():
    out = []
    for h, W, ids, z in sets:
        y = ids[:, 0].contiguous()
        lp, st, a, b = token_logprobs(ids, h, W, top_k=4)
        l, s = topk_distill_fwd(y, ids, z, h, W)
        out += [lp, st, a, b, *token_logprobs_bwd(ids, h, W, st, z), l, s, *topk_distill_bwd(y, ids, z, h, W, s)]
    return out
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = work()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
assert all(torch.equal(p, q) for p, q in zip(got, work()))
print("captured first")
"""


def test_first_calls_of_a_process_may_be_captured():
    """No call needs a warm-up before it is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_outputs_stay_inside_their_buffers():
    from tests.test_guards import Guarded
    for dtype, T, D, V, K in ((BF, 131, 64, 333, 7), (F32, 31, 37, 201, 5)):
        _, (y, tid, z, h, W) = _distill_inputs(T, D, V, K, dtype=dtype)
        ins = [t.clone() for t in (y, tid, h, W)]
        bufs = {n: Guarded(s, t) for n, s, t in [
            ("logp", (T, K), F32), ("stats", (2, T), F32), ("top_ids", (T, K), torch.int32), ("top_logp", (T, K), F32),
            ("dh", (T, D), dtype), ("dW", (V, D), dtype), ("losses", (3,), F32), ("dstats", (3, T), F32)]}
        for n in (token_logprobs_workspace(T, D, V, K, K, dtype)):
            ws = Guarded((n,), torch.uint8)
            token_logprobs(tid, h, W, top_k=K, logp=bufs["logp"].t, stats=bufs["stats"].t, top_ids=bufs["top_ids"].t,
                           top_logp=bufs["top_logp"].t, workspace=ws.t)
            assert ws.intact()
        for n in (token_logprobs_bwd_workspace(T, D, V, K, dtype)):
            ws = Guarded((n,), torch.uint8)
            token_logprobs_bwd(tid, h, W, bufs["stats"].t, bufs["logp"].t, dh=bufs["dh"].t, dW=bufs["dW"].t,
                               workspace=ws.t)
            assert ws.intact()
        f_b, f_min, b_b, b_min = topk_distill_workspace(T, D, V, K, dtype)
        for n in (f_b, f_min):
            ws = Guarded((n,), torch.uint8)
            topk_distill_fwd(y, tid, z, h, W, losses=bufs["losses"].t, stats=bufs["dstats"].t, workspace=ws.t)
            assert ws.intact()
        for n in (b_b, b_min):
            ws = Guarded((n,), torch.uint8)
            topk_distill_bwd(y, tid, z, h, W, bufs["dstats"].t, dh=bufs["dh"].t, dW=bufs["dW"].t, workspace=ws.t)
            assert ws.intact()
        assert all(b.intact() for b in bufs.values())
        assert all(torch.equal(a, b) for a, b in zip(ins, (y, tid, h, W)))


def test_wrapper_refuses_wrong_tensors():
    _, (y, tid, z, h, W) = _distill_inputs(20, 64, 100, 3)
    with pytest.raises(ValueError):
        token_logprobs(y[:-1], h, W)
    with pytest.raises(ValueError):
        token_logprobs(y, h, W[:, :32].contiguous())
    with pytest.raises(ValueError):
        token_logprobs(y, h[:, ::1].t(), W)
    with pytest.raises(TypeError):
        token_logprobs(y.long(), h, W)
    with pytest.raises(TypeError):
        token_logprobs(y, h.half(), W.half())
    with pytest.raises(ValueError):
        topk_distill_fwd(y, tid, z[:, :2].contiguous(), h, W)
    with pytest.raises(ValueError):
        topk_distill_fwd(y.cpu(), tid, z, h, W)
    with pytest.raises(RuntimeError):
        token_logprobs(y, h, W, top_k=65)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_teacher_writes_its_top_tokens_and_a_student_learns_from_them(dtype):
    """The run a user makes: a wide teacher's top tokens with token_logprobs, a narrow student's distillation step
    on them, and the student's log probabilities afterwards.  A student equal to the teacher, distilled on all of
    its vocabulary, has no distillation gradient."""
    T, V, K = 150, 400, 16
    rng, ht, Wt, y = make(T, 256, V, dtype, seed=11)
    _, hs, Ws, _ = make(T, 128, V, dtype, seed=12)
    yg, htg, Wtg, hsg, Wsg = gpu(y, ht, Wt, hs, Ws)
    _, _, tid, tlp = token_logprobs(None, htg, Wtg, top_k=K)
    losses, stats = topk_distill_fwd(yg, tid, tlp, hsg, Wsg)
    dh, dW = topk_distill_bwd(yg, tid, tlp, hsg, Wsg, stats)
    t = oh.token_logprobs(None, ht, Wt, top_k=K)
    r = oh.topk_distill(y, t["top_ids"], t["top_logp"], hs, Ws, 0.3)
    b = Bounds(hs, Ws)
    # the teacher's log probabilities carry an error of their own: p_k is off by that, relatively
    extra = 2 * Bounds(ht, Wt).logp(t["lse"]).max()
    within(losses, r["losses"], np.full(3, b.logp(r["stats"][0]).max() + extra * 20), "losses")
    G = r["G"]
    s = coefficients(G, y, t["top_ids"], t["top_logp"], None, 0.3, T, V)
    within(dh, G @ b.W, b.dh(G, s, dh.dtype) + extra * (s[:, None] * np.abs(b.W).max(0)[None]), "dh")
    lp, _, _, _ = token_logprobs(tid, hsg, Wsg)
    kd = -(torch.softmax(tlp.double(), 1) * lp.double()).sum(1)
    within(stats[2], kd.cpu().numpy(), 3 * b.logp(r["stats"][0]), "kd from log probabilities")
    k64 = min(V, 64)
    h1, W1 = htg, Wtg[:k64].contiguous()
    y1 = torch.zeros(T, dtype=torch.int32, device="cuda")
    _, st1, ids, lps = token_logprobs(y1, h1, W1, top_k=k64)
    _, st2 = topk_distill_fwd(y1, ids, lps, h1, W1, 1.0)
    g, _ = topk_distill_bwd(y1, ids, lps, h1, W1, st2, 1.0)
    within(st2[2], oh.token_logprobs(None, ht, Wt[:k64])["entropy"], 4 * Bounds(ht, Wt[:k64]).dl + 1e-4, "own entropy")
    assert float(g.float().abs().max()) <= 2.0 ** -9 / T * float(W1.float().abs().sum(0).max())
