"""Post-training losses on the GPU: rows split over clusters, targets outside the
vocabulary, the ends of the logits' and temperatures' ranges.  Against the fp64
oracle; tolerances as derived in test_post_training_gpu."""
import math

import numpy as np
import pytest
import torch

from oracle import flce_oracle as O
from test_parity_gpu import assert_grad_close
from test_post_training import IGN, policy_case, teacher_case
from test_post_training_gpu import DT, EPS32, TINY, _check_distill, _check_policy, _close, _cuda, _delta, _head, _lib, _np

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- clusters --

# Few rows, each of them split over two, four or eight CTAs, most of whose warps
# have no tile: they exchange their records as soon as they start.
FEW = [(1, 4100), (4, 4097), (3, 8200), (2, 20001), (7, 33000), (18, 70001)]


@pytest.mark.parametrize("N,V", FEW)
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_few_rows_in_clusters(N, V, dtype):
    Z, y, old, adv, ref = policy_case(N, V, seed=N + V, dtype=dtype, ign=0.0)
    _check_policy(Z, y, old, adv, ref, ent=0.01)
    ids, u = teacher_case(N, V, 12, seed=V)
    _check_distill(Z, y, ids, u, ce=0.25)


@pytest.mark.parametrize("N,V", FEW)
def test_clusters_repeat_their_bits(N, V):
    F = _lib()
    Z, y, old, adv, ref = policy_case(N, V, seed=N, dtype=torch.float32, ign=0.0)
    ids, u = teacher_case(N, V, 12, seed=V)
    p, t = _cuda(Z, y, old, adv), _cuda(Z, y, ids, u)
    calls = (lambda: F.policy_loss(*p, entropy_coef=0.01), lambda: F.distill_topk(*t, row_loss=True))
    want = [call() for call in calls]
    for _ in range(100):
        for call, w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(call(), w))


# ------------------------------------- targets outside the vocabulary, through the head --


@pytest.mark.parametrize("reorder", [False, True])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_heads_with_targets_out_of_range(reduction, reorder):
    """Reported, and without a part in anything but the mean's count, whatever the
    row's vectors and the workspace hold: on a workspace of NaN, and on the same
    one again."""
    F = _lib()
    N, H, V, K = 700, 64, 3000, 20
    X, W, Z, y, old, adv, ref = _head(N, H, V, seed=6, ign=0.6 if reorder else 0.2)
    ids, u = teacher_case(N, V, K, seed=6)
    scale = torch.randn(N, generator=torch.Generator().manual_seed(1)) if reduction == "none" else None
    bad = torch.tensor([3, 257, N - 1])
    y[bad] = torch.tensor([V, -7, 2 ** 31 - 1], dtype=torch.int32)
    valid = y != IGN
    good = valid.clone()
    good[bad] = False
    yg = torch.where(good, y, IGN)
    share = int(good.sum()) / int(valid.sum()) if reduction == "mean" else 1.0
    nscale = None if scale is None else _np(scale)
    for t in (old, adv, ref, u) + (() if scale is None else (scale,)):
        t[bad] = math.nan
    d = _cuda(X, W, y)
    kw = dict(reduction=reduction, grad_row_scale=None if scale is None else scale.cuda())
    off = (~good).cuda()

    def check(f, args, size, reference, own):
        loss0, G, rows0 = reference
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        first = f(*d, *args, workspace=ws, **own, **kw)
        again = f(*d, *args, workspace=ws, **own, **kw)
        loss, status, rows, dX, dW = first
        assert status.item() == 4
        if reorder:
            assert F.row_order_info(ws)[0]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        _close(_np(rows), rows0, 1e-4 * (1 + np.abs(rows0)), "rows")
        assert not rows[off].any() and not dX[off].any()
        s = np.abs(O.row_scale(good.numpy(), reduction, nscale)) * share
        _close(loss.item(), loss0 * share, (s * (1 + np.abs(rows0)) * (1 + np.abs(np.nan_to_num(_np(adv))))).sum() * 2e-4, "loss")
        assert_grad_close(_np(dX), G @ _np(W) * share, "dX")
        assert_grad_close(_np(dW), G.T @ _np(X) * share, "dW")
        fl, _, frows, _, _ = f(*d, *args, workspace=ws, grads=False, **own, **kw)
        assert torch.equal(fl, loss) and torch.equal(frows, rows)

    p = O.policy_reference(Z, yg, old, adv, ref, 0.2, 0.28, 0.05, reduction=reduction, grad_row_scale=nscale)
    check(F.policy_forward_backward, _cuda(old, adv), F.policy_workspace_size(N, H, V, reorder), p[:3],
          dict(ref_logp=ref.cuda(), clip_high=0.28, kl_coef=0.05))
    t = O.distill_reference(Z, yg, ids, u, None, 1.0, 1.0, 0.5, reduction=reduction, grad_row_scale=nscale)
    check(F.distill_forward_backward, _cuda(ids, u), F.distill_workspace_size(N, H, V, K, reorder), t,
          dict(ce_weight=0.5, row_loss=True))


# ---------------------------------------------------------------- huge logits --


@pytest.mark.parametrize("ent", [0.0, 0.1])
@pytest.mark.parametrize("T", [1e-6, 0.01, 1.0, 1e3, 1e6])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_policy_logits_up_to_the_largest_value(dtype, T, ent, monkeypatch):
    """A token forced by the type's largest value, alone, at the end of a row, in
    several places, beside masked entries and against ordinary ones: the softmax
    is one token's (or an even one), its entropy 0 (or a logarithm)."""
    if dtype is torch.float16 and T < 1e-3:
        pytest.skip("gradients of |A| / (N T) are beyond fp16's 65504")
    N, V = 8, 3001
    Z, y, _, adv, _ = policy_case(N, V, seed=3, dtype=dtype, ign=0.0)
    big = torch.finfo(dtype).max
    Z[0, 7] = big
    Z[1, V - 1] = big
    Z[2, 40:44] = big
    Z[3] = Z[3].masked_fill(torch.rand(V, generator=torch.Generator().manual_seed(1)) < 0.5, -math.inf)
    Z[3, 1000] = big
    Z[4] = torch.finfo(dtype).min
    Z[4, 2000] = big
    Z[5] = big
    Z[6, 2999], Z[6, 5] = big, 0.75 * big
    top = Z.float().argmax(1).to(torch.int32)
    y = top if T < 1 else torch.where(torch.arange(N) % 2 == 0, top, y)  # a lower T takes -max / T out of fp32
    # exponentials below 2^-126 are 0; each has the factor (|A| + ent (H + 88)) / T <= 100 / T, with |A| < 5
    monkeypatch.setitem(TINY, dtype, max(TINY[dtype], 100 / T * 2.0 ** -126))
    _check_policy(Z, y, None, adv, None, kl=0.0, ent=ent, T=T)
    _check_policy(Z, y, None, adv, None, kl=0.0, ent=ent, T=T, grad="inplace", lead=1, pad=4)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_distill_logits_up_to_the_largest_value(dtype):
    N, V = 6, 3001
    Z, y, *_ = policy_case(N, V, seed=4, dtype=dtype, ign=0.0)
    ids, u = teacher_case(N, V, 3, seed=4, padded=False)
    Z[:3, 11] = torch.finfo(dtype).max
    Z[2, 2000] = torch.finfo(dtype).max
    ids[:3] = torch.tensor([11, -1, -1], dtype=torch.int32)
    y[:3] = 11
    _check_distill(Z, y, ids, u, T=2.0, ce=0.5)
    _check_distill(Z, y, ids, u, ce=0.5)


# --------------------------------------------- the distillation head's temperatures --


@pytest.mark.parametrize("T", [1e-6, 1e-4, 0.02, 1.0, 50.0, 1e3, 1e6])
def test_distill_head_temperature_range(T):
    """Logits that are exact sums in fp32, far from 0 and a few temperatures apart:
    32768 temperatures plus small multiples of one.  Probabilities hang on the
    differences alone, which the head has exactly."""
    F = _lib()
    N, H, V, K = 300, 16, 2100, 8
    g = torch.Generator().manual_seed(8)
    step = 2.0 ** round(math.log2(T))
    X = torch.zeros(N, H)
    X[:, 0] = 1
    X[:, 1:4] = torch.randint(-2, 3, (N, 3), generator=g).float()
    W = torch.zeros(V, H)
    W[:, 0] = 32768 * step
    W[:, 1:4] = torch.randint(-3, 4, (V, 3), generator=g).float() * step
    X, W = X.bfloat16(), W.bfloat16()
    Z = X.double() @ W.double().T
    assert torch.equal(Z.float().double(), Z)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int64).to(torch.int32)
    y[::7] = IGN
    ids, u = teacher_case(N, V, K, seed=8)
    ids[3] = -1
    u = u * step
    ce = 0.5 if T == 1.0 else 0.0
    loss, status, rows, dX, dW = F.distill_forward_backward(*_cuda(X, W, y, ids, u), temperature=T, ce_weight=ce, row_loss=True)
    assert status.item() == 0
    rloss, G, rrows = O.distill_reference(Z, y, ids, u, None, T, 1.0, ce)
    # one exponential per probability (argument below 40, 2^-24 of it, 2 steps more) and fp32 coefficients
    _close(_np(rows), rrows, 1e-5 * (1 + np.abs(rrows)), "row loss")
    _close(loss.item(), rloss, 1e-5 * (1 + np.abs(rrows)).mean(), "loss")
    # columns 1 to 3 of dW and dX; column 0 of dX is 32768 temperatures times a sum of 0
    assert_grad_close(_np(dW)[:, 1:4], (G.T @ _np(X))[:, 1:4], "dW")
    assert_grad_close(_np(dX)[:, 1:4], (G @ _np(W))[:, 1:4], "dX")
    fl, _, frows, _, _ = F.distill_forward_backward(*_cuda(X, W, y, ids, u), temperature=T, ce_weight=ce, row_loss=True,
                                                    grads=False)
    assert torch.equal(fl, loss) and torch.equal(frows, rows)


def test_distill_head_small_loss_at_a_low_temperature():
    """A teacher that agrees with the student: the loss is a small difference of
    terms of some 30 / T each."""
    F = _lib()
    N, H, V, K, T = 64, 8, 700, 700, 2.0 ** -12
    g = torch.Generator().manual_seed(9)
    X = torch.zeros(N, H)
    X[:, 0], X[:, 1] = 1, torch.randint(1, 3, (N,), generator=g).float()
    W = torch.zeros(V, H)
    W[:, 0], W[:, 1] = 32, torch.randint(-2, 3, (V,), generator=g).float() * T
    X, W = X.bfloat16(), W.bfloat16()
    Z = (X.double() @ W.double().T).float()
    y = torch.zeros(N, dtype=torch.int32)
    ids = torch.stack([torch.randperm(V, generator=g) for _ in range(N)]).to(torch.int32)
    u = Z.gather(1, ids.long()) - 31            # another constant: the same softmax
    loss, status, rows, dX, dW = F.distill_forward_backward(*_cuda(X, W, y, ids, u), temperature=T, row_loss=True)
    assert status.item() == 0
    _, G, rrows = O.distill_reference(Z, y, ids, u, None, T)
    assert np.abs(rrows).max() < 1e-10
    # 700 terms of q (a few 2^-24 of each) times logarithms below 12
    _close(_np(rows), rrows, 12 * 20 * EPS32, "row loss")


# ------------------------------------------------------------ infinite results --


def test_infinite_results_are_infinite():
    """A target (or a teacher's entry) of probability 0: lp is -infinity, the KL
    estimate and the row's loss +infinity, and the others stay as they are."""
    F = _lib()
    Z, y, old, adv, ref = policy_case(6, 100, seed=11, ign=0.0)
    ids, u = teacher_case(6, 100, 3, seed=11, padded=False)
    Z[1, y[1].long()] = -math.inf
    _, _, lp, H, kl, g = F.policy_loss(*_cuda(Z, y, old, adv), ref_logp=ref.cuda())
    assert lp[1].item() == -math.inf and kl[1].item() == math.inf and torch.isfinite(H).all() and torch.isfinite(g).all()
    _, _, rlp, rH, _ = O.policy_reference(Z, y, old, adv, None)
    _close(_np(H), rH, _delta(100) * (1 + rH), "entropy")
    keep = [0, 2, 3, 4, 5]
    _close(_np(lp)[keep], rlp[keep], _delta(100) + np.abs(rlp[keep]) * EPS32, "logp")
    Z[4, ids[4, 0].long()] = -math.inf
    _, _, rows, g = F.distill_topk(*_cuda(Z, y, ids, u), row_loss=True)
    want = [i for i in range(6) if Z[i, ids[i].long()].isneginf().any()]
    assert torch.isposinf(rows).nonzero().flatten().tolist() == want and torch.isfinite(g).all()


def test_policy_rows_of_probability_zero():
    F = _lib()
    l, y = torch.tensor([math.inf, 1.0, 2.0]), torch.tensor([1, 2, IGN], dtype=torch.int32)
    old, adv, ref = torch.tensor([-1.0, -1.0, 0.0]), torch.tensor([1.0, 1.0, 1.0]), torch.tensor([-2.0, -1.5, 0.0])
    loss, rows, kl, w, status = F.clipped_policy(*_cuda(l, y, old, adv), ref_logp=ref.cuda())
    assert kl.tolist()[0] == math.inf and kl.tolist()[2] == 0.0 and status.item() == 0
    assert abs(kl[1].item() - (math.exp(-0.5) - 0.5)) <= 2 * EPS32
    assert rows.tolist() == [0.0, -1.0, 0.0] and w.tolist() == [0.0, 0.5, 0.0] and loss.item() == -0.5


# --------------------------------------------------------- what other tests leave open --


def test_a_bad_row_leaves_the_others_alone():
    """NaN and infinity in a row make its own results NaN and no other row's."""
    F = _lib()
    Z, y, old, adv, ref = policy_case(12, 300, seed=10, ign=0.0)
    ids, u = teacher_case(12, 300, 5, seed=10)
    clean = F.policy_loss(*_cuda(Z, y, old, adv), entropy_coef=0.1), F.distill_topk(*_cuda(Z, y, ids, u), row_loss=True)
    Z[2, 5] = math.nan
    Z[3] = -math.inf
    Z[4, 7] = math.inf
    bad = torch.tensor([2, 3, 4])
    good = torch.tensor([i for i in range(12) if i not in (2, 3, 4)])
    got = F.policy_loss(*_cuda(Z, y, old, adv), entropy_coef=0.1), F.distill_topk(*_cuda(Z, y, ids, u), row_loss=True)
    for was, now in ((clean[0][2:4] + clean[0][5:], got[0][2:4] + got[0][5:]), (clean[1][2:], got[1][2:])):
        for a, b in zip(was, now):
            assert torch.equal(a.cpu()[good], b.cpu()[good])
    assert torch.isnan(got[0][5].cpu()[bad]).all() and torch.isnan(got[0][0]).all() and torch.isnan(got[1][0]).all()
    assert torch.isnan(got[1][3].cpu()[bad]).all()


@pytest.mark.parametrize("T", [1e-6, 1e-3, 1e3, 1e6])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_gradients_over_the_temperature_range(T, dtype):
    if dtype is torch.float16 and (T < 1e-3 or T > 1e3):
        pytest.skip("logits of this size are not fp16 numbers")
    g = torch.Generator().manual_seed(3)
    step = 2.0 ** round(math.log2(T))
    Z = (torch.randint(-6, 7, (9, 300), generator=g).double() * step).to(dtype)
    mask = torch.rand(9, 300, generator=g) < 0.3
    mask[:, 0] = False
    Z = Z.masked_fill(mask, -math.inf)
    y = torch.zeros(9, dtype=torch.int32)
    adv = torch.randn(9, generator=g)
    _check_policy(Z, y, None, adv, None, kl=0.0, ent=0.1, T=T)
    ids, u = teacher_case(9, 300, 5)
    ids = torch.where(mask.gather(1, ids.long().clamp(min=0)), -1, ids).to(torch.int32)
    _check_distill(Z, y, ids, (u * step).float(), T=T)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_loss_of_heads_with_reordered_rows(reduction):
    F = _lib()
    N, H, V, K = 1300, 64, 3000, 20
    X, W, Z, y, old, adv, ref = _head(N, H, V, seed=4, ign=0.6)
    ids, u = teacher_case(N, V, K, seed=4)
    scale = torch.randn(N, generator=torch.Generator().manual_seed(1)) if reduction == "none" else None
    nscale = None if scale is None else _np(scale)
    s = np.abs(O.row_scale((y != IGN).numpy(), reduction, nscale))
    kw = dict(reduction=reduction, grad_row_scale=None if scale is None else scale.cuda())
    d = _cuda(X, W, y)
    ws = torch.empty(F.policy_workspace_size(N, H, V, True), dtype=torch.uint8, device="cuda")
    loss, *_ = F.policy_forward_backward(*d, *_cuda(old, adv), ref_logp=ref.cuda(), clip_high=0.28, kl_coef=0.05,
                                         workspace=ws, **kw)
    assert F.row_order_info(ws)[0]
    want = O.policy_reference(Z, y, old, adv, ref, 0.2, 0.28, 0.05, reduction=reduction, grad_row_scale=nscale)[0]
    # 1e-5 a row: the log-probabilities' error, times |dL/dlp| <= 1.28 |A| + kl |e^d - 1|
    _close(loss.item(), want, (s * (1.3 * np.abs(_np(adv)) + 0.2)).sum() * 1e-5 + abs(want) * EPS32, "policy loss")
    ws = torch.empty(F.distill_workspace_size(N, H, V, K, True), dtype=torch.uint8, device="cuda")
    loss, *_ = F.distill_forward_backward(*d, *_cuda(ids, u), ce_weight=0.5, workspace=ws, **kw)
    assert F.row_order_info(ws)[0]
    want, _, rows = O.distill_reference(Z, y, ids, u, None, 1.0, 1.0, 0.5, reduction=reduction, grad_row_scale=nscale)
    _close(loss.item(), want, (s * (1 + np.abs(rows))).sum() * 1e-5 + abs(want) * EPS32, "distillation loss")


@pytest.mark.parametrize("N,H,V", [(700, 64, 60000), (3, 1024, 30000), (260, 520, 20011), (513, 136, 70001)])
def test_distill_head_on_every_workspace(N, H, V):
    """Wide chunks with and without the reordering area, and the least that a call
    takes: the oracle's results, and the same bits again."""
    F = _lib()
    K = 12
    X, W, Z, y, *_ = _head(N, H, V, seed=N, ign=0.0 if N < 5 else 0.55)
    ids, u = teacher_case(N, V, K, seed=N)
    d = _cuda(X, W, y, ids, u)
    rloss, G, rrows = O.distill_reference(Z, y, ids, u, None, 1.0, 1.0, 0.5)
    rX, rW = G @ _np(W), G.T @ _np(X)
    for nbytes in (F.distill_workspace_size(N, H, V, K), F.distill_workspace_size(N, H, V, K, True),
                   F.distill_workspace_size(N, H, 1, K)):
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        loss, status, rows, dX, dW = F.distill_forward_backward(*d, ce_weight=0.5, row_loss=True, workspace=ws)
        assert status.item() == 0
        _close(_np(rows), rrows, 1e-4 * (1 + np.abs(rrows)), "row loss")
        _close(loss.item(), rloss, 1e-5 * (1 + np.abs(rrows)).mean(), "loss")
        assert_grad_close(_np(dX), rX, "dX")
        assert_grad_close(_np(dW), rW, "dW")
        again = F.distill_forward_backward(*d, ce_weight=0.5, row_loss=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, status, rows, dX, dW)))


def test_another_stream_with_inputs_made_before_it():
    """The side stream waits for the inputs once; every operator there has the bits
    of the current stream's call."""
    F = _lib()
    Z, y, old, adv, ref = policy_case(64, 3001, seed=31, dtype=torch.bfloat16)
    ids, u = teacher_case(64, 3001, 24, seed=31)
    X, W, _, hy, hold, hadv, _ = _head(64, 64, 3001, seed=32)
    Zd, yd, ld, od, ad, rd, idd, ud, Xd, Wd, hyd, hod, had = _cuda(Z, y, -old, old, adv, ref, ids, u, X, W, hy, hold, hadv)
    calls = [lambda s=None: F.clipped_policy(ld, yd, rd, ad, stream=s),
             lambda s=None: F.policy_loss(Zd, yd, od, ad, ref_logp=rd, kl_coef=0.1, entropy_coef=0.01, stream=s),
             lambda s=None: F.distill_topk(Zd, yd, idd, ud, ce_weight=0.5, temperature=2.0, row_loss=True, stream=s),
             lambda s=None: F.policy_forward_backward(Xd, Wd, hyd, hod, had, stream=s),
             lambda s=None: F.distill_forward_backward(Xd, Wd, hyd, idd, ud, row_loss=True, stream=s)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [[call(side) for call in calls] for _ in range(5)]
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(want, outs):
            assert all(torch.equal(x, z) for x, z in zip(a, b))
