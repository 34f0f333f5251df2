"""Post-training losses on the GPU against the fp64 oracle.

Tolerances for the losses on logits count the kernels' roundings.  With
eps = 2^-24 (half a step of fp32): an exponential e = 2^((z - m) zs) has a
relative error of at most |arg| ln2 2 eps (zs and the product) + 4 eps (the
hardware's 2^x, 2 steps); a sum of n terms held in T-wide partial sums adds at
most (n / T + 40) eps; the per-row factors add a few eps.  DELTA bounds their
sum for the sizes below; a value that depends on the row's log-probability
inherits it as an absolute error of lp.  Outputs add half a step of their type.
"""
import math

import numpy as np
import pytest
import torch

from oracle import flce_oracle as O
from test_parity_gpu import assert_grad_close
from test_post_training import IGN, policy_case, teacher_case

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}  # half the smallest step


def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import lm_head_linear_03_b200 as F
    F.load_library()
    return F


def _np(t):
    return t.detach().double().cpu().numpy()


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _delta(V):
    return (V / 256 + 120) * EPS32  # arguments down to -50 count; smaller exponentials are below eps


def _close(got, ref, tol, what):
    got, ref = np.asarray(got), np.asarray(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    bad = ~(np.abs(got - ref) <= tol) & np.isfinite(ref)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, e.g. {got[bad][0]} against {ref[bad][0]}"


def _padded(Z, pad, lead=0):
    """Z on the GPU as columns of a buffer with `lead` columns of NaN in front and `pad` behind."""
    if not pad and not lead:
        return Z.cuda(), None
    buf = torch.full((Z.shape[0], lead + Z.shape[1] + pad), math.nan, dtype=Z.dtype).cuda()
    view = buf[:, lead:lead + Z.shape[1]]
    view.copy_(Z)
    return view, buf


def _check_policy(Z, y, old, adv, ref, *, pad=0, lead=0, kl=0.1, ent=0.0, T=1.0, reduction="mean", scale=None, grad="new"):
    F = _lib()
    Zd, buf = _padded(Z, pad, lead)
    yd, od, ad, rd, sd = _cuda(y, old, adv, ref, scale)
    before = Zd.clone()
    loss, status, lp, H, klo, g = F.policy_loss(Zd, yd, od, ad, ref_logp=rd, clip_low=0.2, clip_high=0.28, kl_coef=kl,
                                                entropy_coef=ent, temperature=T, reduction=reduction, grad_row_scale=sd,
                                                grad=grad)
    torch.cuda.synchronize()
    assert status.item() == 0
    rloss, rG, rlp, rH, rkl = O.policy_reference(Z, y, old, adv, ref, 0.2, 0.28, kl, ent, T, reduction=reduction,
                                                 grad_row_scale=None if scale is None else _np(scale))
    N, V = Z.shape
    d = _delta(V)
    valid = _np(y) != IGN
    A = np.where(valid, np.abs(_np(adv)), 0)
    r = np.ones(N) if old is None else np.where(valid, np.exp(rlp - np.where(valid, _np(old), 0)), 1)
    ed = np.zeros(N) if ref is None else np.where(valid, np.exp(np.where(valid, _np(ref), 0) - rlp), 0)
    _close(_np(lp), rlp, d + np.abs(rlp) * EPS32, "logp")
    _close(_np(H), rH, d * (1 + np.abs(rH)), "entropy")
    _close(_np(klo), rkl, d * np.abs(ed - 1) + d * d * (ed + 1) + rkl * EPS32, "kl")
    s = O.row_scale(valid, reduction, None if scale is None else _np(scale))
    slack = A * r + kl * np.abs(ed - 1) + kl * (ed + 1) * d + ent * (1 + rH)  # |dL/dlp| and its change over d
    rows_tol = np.abs(s) * (slack * d * 2)
    _close(loss.item(), rloss, rows_tol.sum() + abs(rloss) * EPS32 * 2, "loss")
    if grad == "none":
        assert g is None and torch.equal(torch.nan_to_num(Zd), torch.nan_to_num(before))
        return None
    with np.errstate(divide="ignore", invalid="ignore"):
        logp_all, P = O._softmax_rows(np.where(valid[:, None], _np(Z), 0.0) / T)
        plog = np.where(P > 0, P * np.abs(np.where(P > 0, logp_all, 0)), 0)
    gmag = np.abs(s) / T * (A * np.maximum(r, 1) + kl * (1 + ed))
    onehot = np.zeros_like(P)
    onehot[np.arange(N), np.where(valid, _np(y), 0).astype(int)] = 1
    tol = gmag[:, None] * (P + onehot) * 4 * d + (np.abs(s) / T * ent)[:, None] * (plog + P * (1 + rH)[:, None]) * 4 * d
    tol = tol + np.abs(rG) * (torch.finfo(Z.dtype).eps / 2) + TINY[Z.dtype]
    _close(_np(g), rG, tol, "dlogits")
    if buf is not None:
        assert torch.isnan(buf[:, :lead]).all() and torch.isnan(buf[:, lead + V:]).all(), "columns outside were written"
        if grad == "new":
            assert torch.equal(torch.nan_to_num(Zd), torch.nan_to_num(before))
    return g


DT = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V,pad", [(1, 1, 0), (1, 2, 0), (3, 7, 0), (2, 8, 3), (5, 100, 0), (17, 1001, 0), (40, 4096, 0),
                                     (12, 4093, 19), (9, 32064, 0), (3, 50021, 43), (2, 131071, 0)])
def test_policy_sizes(N, V, pad, dtype):
    Z, y, old, adv, ref = policy_case(N, V, seed=N + V, dtype=dtype, ign=0.0 if N < 5 else 0.2)
    _check_policy(Z, y, old, adv, ref, pad=pad)


@pytest.mark.parametrize("N,V", [(1, 262151), (2, 600001)])
def test_policy_long_rows(N, V):
    Z, y, old, adv, ref = policy_case(N, V, seed=3, dtype=torch.bfloat16, ign=0.0)
    _check_policy(Z, y, old, adv, ref, ent=0.01)


@pytest.mark.parametrize("kl,ent,T,reduction", [(0.0, 0.0, 1.0, "mean"), (0.0, 0.05, 1.0, "sum"), (0.2, 0.0, 0.6, "mean"),
                                                (0.1, 0.02, 1.7, "none"), (0.1, 0.02, 3.0, "mean")])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_policy_options(kl, ent, T, reduction, dtype):
    Z, y, old, adv, ref = policy_case(50, 2051, seed=5, dtype=dtype, temperature=T)
    scale = torch.randn(50, generator=torch.Generator().manual_seed(1)) if reduction == "none" else None
    _check_policy(Z, y, old, adv, ref if kl else None, kl=kl, ent=ent, T=T, reduction=reduction, scale=scale)


# More rows than run at the same time, in each shape of CTA (one warp, four,
# eight, clusters), with rows of every alignment, long and scattered gaps.
MANY = [(2600, 1001), (700, 20003), (330, 60001), (160, 140001)]


def _gaps(y):
    y = y.clone()
    n = len(y)
    y[n // 8: n // 3] = IGN
    y[-3:] = IGN
    return y


@pytest.mark.parametrize("N,V", MANY)
@pytest.mark.parametrize("grad", ["new", "inplace"])
def test_policy_many_rows(N, V, grad):
    Z, y, old, adv, ref = policy_case(N, V, seed=N, dtype=torch.bfloat16, ign=0.25)
    _check_policy(Z, _gaps(y), old, adv, ref, ent=0.01 if grad == "new" else 0.0, grad=grad)


@pytest.mark.parametrize("N,V", MANY)
def test_distill_many_rows(N, V):
    Z, y, *_ = policy_case(N, V, seed=N, dtype=torch.float16, ign=0.25)
    g = torch.Generator().manual_seed(N)
    ids = torch.randint(0, V, (N, 40), generator=g, dtype=torch.int64).to(torch.int32)
    ids[:, 30:] = ids[:, :10] // 2                 # clustered, some of them twice
    u = torch.randn(N, 40, generator=g) * 2
    _check_distill(Z, _gaps(y), ids, u, ce=0.25)


@pytest.mark.parametrize("which", ["every_third", "last", "first_half", "none"])
def test_policy_rows_that_do_not_count(which):
    """Long rows, more of them than run at the same time: wherever those lie that
    count, they have their results and the others zeros; targets outside [0, V)
    are reported and counted, and nothing behind a row's V entries is written."""
    F = _lib()
    N, V, pad = 900, 52001, 3
    g = torch.Generator().manual_seed(9)
    Z = torch.randn(N, V, generator=g).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int64).to(torch.int32)
    adv = torch.randn(N, generator=g)
    i = torch.arange(N)
    keep = {"every_third": i % 3 == 1, "last": i == N - 1, "first_half": i < N // 2, "none": i < 0}[which]
    y[~keep] = IGN
    y[N - 2], y[5] = V, -7
    pick = torch.nonzero(keep & (y >= 0) & (y < V)).flatten().tolist()
    Zd, buf = _padded(Z, pad)
    loss, status, lp, H, kl, dz = F.policy_loss(Zd, y.cuda(), None, adv.cuda(), entropy_coef=0.01, grad="inplace")
    assert status.item() == 4
    assert dz.data_ptr() == Zd.data_ptr() and torch.isnan(buf[:, V:]).all()
    off = torch.ones(N, dtype=torch.bool)
    off[pick] = False
    for t in (lp, H, kl, dz):
        assert torch.count_nonzero(t[off.cuda()]).item() == 0
    if len(pick):
        want = O.policy_reference(Z[pick], y[pick], None, adv[pick], entropy_coef=0.01)
        _close(_np(lp)[pick], want[2], _delta(V) + np.abs(want[2]) * EPS32, "logp")
        count = int((y != IGN).sum())  # the mean is over all rows that are not ignored
        assert_grad_close(_np(dz)[pick], want[1] * (len(pick) / count), "dlogits")


def test_rows_behind_two_to_the_31_elements():
    """17000 x 128256 logits: the last rows lie beyond 2^31 elements."""
    F = _lib()
    N, V = 17000, 128256
    g = torch.Generator(device="cuda").manual_seed(5)
    Z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, 1000):
        Z[i:i + 1000] = torch.randn(1000, V, generator=g, device="cuda")
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    adv = torch.randn(N, generator=g, device="cuda")
    y[: N - 40] = IGN
    pick = torch.arange(N - 40, N, device="cuda")
    want = O.policy_reference(Z[pick].cpu(), y[pick].cpu(), None, adv[pick].cpu())
    loss, status, lp, H, kl, dz = F.policy_loss(Z, y, None, adv)
    assert status.item() == 0
    _close(_np(lp[pick]), want[2], _delta(V) + np.abs(want[2]) * EPS32, "logp")
    assert_grad_close(_np(dz[pick]), want[1], "dlogits")
    assert not any(torch.count_nonzero(dz[i:i + 1000]).item() for i in range(0, N - 1000, 1000))
    ids = torch.randint(0, V, (N, 20), generator=g, device="cuda", dtype=torch.int32)
    u = torch.randn(N, 20, generator=g, device="cuda")
    want = O.distill_reference(Z[pick].cpu(), y[pick].cpu(), ids[pick].cpu(), u[pick].cpu())
    loss, status, rows, _ = F.distill_topk(Z, y, ids, u, row_loss=True, grad="inplace")
    _close(_np(rows[pick]), want[2], 1e-5 * (1 + np.abs(want[2])), "row loss")
    assert_grad_close(_np(Z[pick]), want[1], "dlogits in place")


def test_policy_on_policy_and_metrics_only():
    Z, y, old, adv, ref = policy_case(33, 515, seed=6)
    _check_policy(Z, y, None, adv, ref, kl=0.1)       # ratio 1
    _check_policy(Z, y, old, adv, ref, kl=0.0)        # KL reported, not in the loss
    _check_policy(Z, y, old, adv, ref, grad="none")


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad", [0, 5])
def test_policy_in_place(dtype, pad):
    Z, y, old, adv, ref = policy_case(21, 3001, seed=7, dtype=dtype)
    new = _check_policy(Z, y, old, adv, ref, pad=pad, ent=0.01)
    same = _check_policy(Z, y, old, adv, ref, pad=pad, ent=0.01, grad="inplace")
    assert torch.equal(new, same)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_policy_unaligned_views(dtype):
    """Rows that start anywhere: a slice of columns of a wider buffer, with a
    gradient whose rows are aligned otherwise, and in place.  Where a row starts
    decides which elements share a partial sum, so the views agree with the
    oracle, not bit by bit with one another."""
    Z, y, old, adv, ref = policy_case(6, 1234, seed=8, dtype=dtype)
    for lead in range(1, 9):
        new = _check_policy(Z, y, old, adv, ref, lead=lead, pad=66)
        same = _check_policy(Z, y, old, adv, ref, lead=lead, pad=66, grad="inplace")
        assert torch.equal(new, same)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_policy_masked_vocabulary(dtype, low):
    """Entries masked with -infinity or the type's lowest value, a row that is
    the lowest value everywhere, and ignored rows that hold NaN."""
    Z, y, old, adv, ref = policy_case(24, 777, seed=9, dtype=dtype, ign=0.3)
    v = -math.inf if low == "inf" else torch.finfo(dtype).min
    mask = torch.rand(24, 777, generator=torch.Generator().manual_seed(2)) < 0.4
    mask[torch.arange(24), y.clamp(min=0).long()] = False
    Z = Z.masked_fill(mask, v)
    if low == "lowest":
        i = int((y != IGN).nonzero()[0])
        Z[i] = v
        old[i], ref[i] = -math.log(777), -math.log(777) + 0.1
    gone = y == IGN
    for t in (old, adv, ref):
        t[gone] = math.nan
    Z[gone] = math.nan
    _check_policy(Z, y, old, adv, ref, kl=0.05, ent=0.03)


@pytest.mark.parametrize("T", [1e-6, 1e-3, 1e3, 1e6])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_temperature_range(T, dtype):
    """The ends of the range, with masked entries, beside the same softmax of
    pre-scaled logits at temperature 1 (logits of T's magnitude, powers of two
    apart, so that both are the same numbers)."""
    F = _lib()
    g = torch.Generator().manual_seed(3)
    step = 2.0 ** round(math.log2(T))
    Z = torch.randint(-6, 7, (9, 300), generator=g).double() * step
    Z = Z.clamp(-60000, 60000) if dtype is torch.float16 else Z
    if dtype is torch.float16 and T < 1e-3:
        pytest.skip("logits of this size are not fp16 numbers")
    Z = Z.to(dtype)
    mask = torch.rand(9, 300, generator=g) < 0.3
    mask[:, 0] = False
    Z = Z.masked_fill(mask, -math.inf)
    y = torch.zeros(9, dtype=torch.int32)
    adv = torch.randn(9, generator=g)
    out = F.policy_loss(*_cuda(Z, y), None, adv.cuda(), temperature=T, entropy_coef=0.1)
    ref = O.policy_reference(Z, y, None, adv, None, entropy_coef=0.1, temperature=T)
    assert torch.isfinite(out[5]).all()
    _close(_np(out[2]), ref[2], 1e-5 * (1 + np.abs(ref[2])), "logp")
    _close(_np(out[3]), ref[3], 1e-5 * (1 + np.abs(ref[3])), "entropy")
    ids, u = teacher_case(9, 300, 5)
    ids = torch.where(mask.gather(1, ids.long().clamp(min=0)), -1, ids).to(torch.int32)
    _, _, rows, gd = F.distill_topk(*_cuda(Z, y, ids, u * step), temperature=T, row_loss=True)
    want = O.distill_reference(Z, y, ids, u * step, temperature=T)
    _close(_np(rows), want[2], 1e-5 * (1 + np.abs(want[2])), "row loss")


def test_policy_bad_values_stay_in_their_rows():
    F = _lib()
    Z, y, old, adv, ref = policy_case(8, 300, seed=10, ign=0.0)
    Z[2, 5] = math.nan
    Z[3] = -math.inf
    Z[4, 7] = math.inf
    args = _cuda(Z, y, old, adv)
    g = F.policy_loss(*args)[-1]
    for i in range(8):
        assert torch.isnan(g[i]).all() == (i in (2, 3, 4))


def test_policy_clip_borders_and_extreme_ratios():
    """Exactly representable borders: a ratio on the border passes its gradient,
    one beyond it does not; infinite ratios are clipped."""
    F = _lib()
    N, V = 6, 4
    Z = torch.zeros(N, V)
    lp = -math.log(4.0)
    y = torch.zeros(N, dtype=torch.int32)
    old = torch.full((N,), lp)
    old[4], old[5] = -1000.0, -1000.0            # ratio overflows
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0, 2.0, 0.0])
    args = _cuda(Z, y, old, adv)
    loss, status, _, _, _, g = F.policy_loss(*args, clip_low=0.0, clip_high=0.0, reduction="sum")
    rloss, rG, *_ = O.policy_reference(Z, y, None, adv, None, 0.0, 0.0, reduction="sum")
    # old is lp rounded to fp32, so rows 0..3 sit within a rounding of the border: either side is right
    assert abs(loss.item() - (-2.0)) <= 1e-5
    assert torch.count_nonzero(g[4]).item() == 0 and torch.count_nonzero(g[5]).item() == 0
    _, _, _, _, _, g = F.policy_loss(args[0], args[1], None, args[3], clip_low=0.0, clip_high=0.0, reduction="sum")
    _close(_np(g), rG, np.abs(rG) * 1e-5, "ratio 1 on both borders")


def test_policy_target_out_of_range():
    F = _lib()
    Z, y, old, adv, ref = policy_case(16, 100, ign=0.0)
    y[3], y[7] = 100, -1
    loss, status, lp, H, kl, g = F.policy_loss(*_cuda(Z, y, old, adv))
    assert status.item() == 4
    assert torch.count_nonzero(g[3]).item() == 0 and torch.count_nonzero(g[7]).item() == 0
    loss, status, rows, g = F.distill_topk(*_cuda(Z, y, *teacher_case(16, 100, 3)))
    assert status.item() == 4


def test_all_rows_ignored():
    F = _lib()
    Z, y, old, adv, ref = policy_case(16, 100)
    y[:] = IGN
    ids, u = teacher_case(16, 100, 3)
    loss, status, lp, H, kl, g = F.policy_loss(*_cuda(Z, y, old, adv), ref_logp=ref.cuda(), kl_coef=0.1)
    assert loss.item() == 0 and status.item() == 0 and torch.count_nonzero(g).item() == 0
    loss, status, rows, g = F.distill_topk(*_cuda(Z, y, ids, u), row_loss=True)
    assert loss.item() == 0 and torch.count_nonzero(g).item() == 0 and torch.count_nonzero(rows).item() == 0
    loss, rows, kl, w, status = F.clipped_policy(*_cuda(-old, y, old, adv))
    assert loss.item() == 0 and torch.count_nonzero(w).item() == 0
    X, W = torch.randn(16, 64).bfloat16().cuda(), torch.randn(100, 64).bfloat16().cuda()
    loss, status, lp, dX, dW = F.policy_forward_backward(X, W, y.cuda(), *_cuda(old, adv))
    assert loss.item() == 0 and torch.count_nonzero(dX).item() == 0 and torch.count_nonzero(dW).item() == 0
    loss, status, rows, dX, dW = F.distill_forward_backward(X, W, y.cuda(), *_cuda(ids, u))
    assert loss.item() == 0 and torch.count_nonzero(dX).item() == 0 and torch.count_nonzero(dW).item() == 0


# --------------------------------------------------------------- distillation --


def _check_distill(Z, y, ids, u, *, lse=None, pad=0, T=1.0, kd=1.0, ce=0.0, reduction="mean", scale=None, grad="new"):
    F = _lib()
    Zd, buf = _padded(Z, pad)
    yd, idd, ud, ld, sd = _cuda(y, ids, u, lse, scale)
    loss, status, rows, g = F.distill_topk(Zd, yd, idd, ud, teacher_lse=ld, temperature=T, kd_weight=kd, ce_weight=ce,
                                           reduction=reduction, grad_row_scale=sd, row_loss=True, grad=grad)
    torch.cuda.synchronize()
    assert status.item() == 0
    rloss, rG, rrows = O.distill_reference(Z, y, ids, u, lse, T, kd, ce, reduction=reduction,
                                           grad_row_scale=None if scale is None else _np(scale))
    N, V = Z.shape
    # q: fp32 exponential (2 steps) and a K-term sum on top of the softmax's errors
    d = _delta(V) + ids.shape[1] / 32 * EPS32
    valid = _np(y) != IGN
    with np.errstate(divide="ignore", invalid="ignore"):
        logp, P = O._softmax_rows(np.where(valid[:, None], _np(Z), 0.0) / T)
        logp1, P1 = O._softmax_rows(np.where(valid[:, None], _np(Z), 0.0))
    sparse, rowmag = np.zeros_like(P), np.zeros(N)
    Q = np.zeros(N)
    uu = np.where((_np(ids) >= 0) & valid[:, None], _np(u) / T, -np.inf)
    for i in np.nonzero(valid)[0]:
        k = np.nonzero(uu[i] > -np.inf)[0]
        if len(k):
            m = uu[i, k].max()
            lq = uu[i, k] - (m + np.log(np.exp(uu[i, k] - m).sum()) if lse is None else float(_np(lse)[i]))
            q = np.exp(lq)
            Q[i] = q.sum()
            np.add.at(sparse[i], _np(ids)[i, k].astype(int), abs(kd) / T * q)
            rowmag[i] += abs(kd) * (q * (1 + np.abs(lq - logp[i, _np(ids)[i, k].astype(int)]))).sum()
        if ce:
            sparse[i, int(y[i])] += abs(ce)
            rowmag[i] += abs(ce) * (1 + abs(logp1[i, int(y[i])]))
    s = np.abs(O.row_scale(valid, reduction, None if scale is None else _np(scale)))
    _close(_np(rows), rrows, 4 * d * rowmag + np.abs(rrows) * EPS32, "row loss")
    _close(loss.item(), rloss, (s * 4 * d * rowmag).sum() + abs(rloss) * 2 * EPS32, "loss")
    if g is None:
        return None
    tol = 4 * d * s[:, None] * ((abs(kd) / T * Q)[:, None] * P + abs(ce) * P1 + sparse)
    tol = tol + np.abs(rG) * (torch.finfo(Z.dtype).eps / 2) + TINY[Z.dtype]
    _close(_np(g), rG, tol, "dlogits")
    if buf is not None:
        assert torch.isnan(buf[:, V:]).all()
    return g


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,V,K,pad", [(1, 1, 1, 0), (1, 5, 5, 0), (3, 7, 2, 1), (17, 1001, 16, 0), (20, 4096, 64, 0),
                                       (7, 4093, 33, 19), (5, 32064, 50, 0), (2, 131071, 256, 0), (3, 2000, 1024, 8)])
def test_distill_sizes(N, V, K, pad, dtype):
    Z, y, *_ = policy_case(N, V, seed=N + V, dtype=dtype, ign=0.0 if N < 5 else 0.2)
    ids, u = teacher_case(N, V, K, seed=V, dtype=dtype)
    _check_distill(Z, y, ids, u, pad=pad)


@pytest.mark.parametrize("T,kd,ce,reduction", [(1.0, 1.0, 0.5, "mean"), (2.0, 4.0, 0.0, "sum"), (3.0, 1.0, 0.5, "none"),
                                               (1.0, 0.0, 1.0, "mean"), (0.5, 1.0, 2.0, "mean")])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("given", [False, True])
def test_distill_options(T, kd, ce, reduction, dtype, given):
    Z, y, *_ = policy_case(40, 2051, seed=11, dtype=dtype)
    ids, u = teacher_case(40, 2051, 20, seed=12)
    ids[4] = -1                                    # no entry at all
    u[5, :10] = -math.inf                          # entries of probability 0
    lse = torch.logsumexp(u / T, 1) + 0.3 if given else None
    scale = torch.randn(40, generator=torch.Generator().manual_seed(1)) if reduction == "none" else None
    _check_distill(Z, y, ids, u, lse=lse, T=T, kd=kd, ce=ce, reduction=reduction, scale=scale)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,gap", [(3.0, 110.0), (50.0, 1000.0), (1000.0, 20000.0)])
def test_distill_peak_behind_the_first_tiles(T, gap, dtype):
    """A logit `gap` above the others, behind a warp's first tile: near them at
    temperature T, beyond fp32's exponents (88) at that of the hard labels."""
    N, V, K = 6, 200001, 9
    g = torch.Generator().manual_seed(12)
    Z = torch.randn(N, V, generator=g)
    at = torch.tensor([17000, 43000, 69500, 95001, 120002, V - 1])
    Z[torch.arange(N), at] += gap
    ids, u = teacher_case(N, V, K, seed=3)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int64).to(torch.int32)
    y[::2] = at[::2].to(torch.int32)
    _check_distill(Z.to(dtype), y, ids, u, T=T, ce=0.5)


def test_distill_same_id_twice_and_target_in_the_list():
    Z, y, *_ = policy_case(30, 60, seed=13)
    ids, u = teacher_case(30, 60, 48, seed=14, duplicates=True)
    ids[:, 7] = y.clamp(min=0)
    _check_distill(Z, y, ids, u, ce=0.5)
    _check_distill(Z, y, torch.zeros_like(ids), u)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "fp16", "fp32"])
def test_distill_in_place_and_forward_only(dtype):
    Z, y, *_ = policy_case(21, 3001, seed=15, dtype=dtype)
    ids, u = teacher_case(21, 3001, 40, seed=15, dtype=torch.bfloat16)
    new = _check_distill(Z, y, ids, u, ce=0.2, T=2.0)
    same = _check_distill(Z, y, ids, u, ce=0.2, T=2.0, grad="inplace")
    assert torch.equal(new, same)
    _check_distill(Z, y, ids, u, ce=0.2, T=2.0, grad="none")


def test_distill_masked_vocabulary_and_ignored_rows():
    Z, y, *_ = policy_case(24, 777, seed=16, ign=0.3)
    ids, u = teacher_case(24, 777, 12, seed=16)
    mask = torch.rand(24, 777, generator=torch.Generator().manual_seed(2)) < 0.4
    mask.scatter_(1, ids.long().clamp(min=0), False)
    mask[torch.arange(24), y.clamp(min=0).long()] = False
    Z = Z.masked_fill(mask, -math.inf)
    gone = y == IGN
    Z[gone], u[gone] = math.nan, math.nan
    ids[gone] = 1 << 30                            # never looked at
    _check_distill(Z, y, ids, u, ce=0.5)


def test_distill_id_out_of_range():
    F = _lib()
    Z, y, *_ = policy_case(8, 100, ign=0.0)
    ids, u = teacher_case(8, 100, 4, padded=False)
    bad = ids.clone()
    bad[2, 1] = 100
    loss, status, rows, g = F.distill_topk(*_cuda(Z, y, bad, u), row_loss=True)
    assert status.item() == 4
    ids[2, 1] = -1                                 # counts as an empty slot
    _, _, rows2, g2 = F.distill_topk(*_cuda(Z, y, ids, u), row_loss=True)
    assert torch.equal(g, g2) and torch.equal(rows, rows2)


# ----------------------------------------------------------------- policy rows --


@pytest.mark.parametrize("N", [1, 2, 31, 256, 257, 2048, 2049, 5000, 40000])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_clipped_policy_rows(N, reduction):
    F = _lib()
    _, y, old, adv, ref = policy_case(N, 5, seed=N, ign=0.3)
    g = torch.Generator().manual_seed(N)
    lp = (old + 0.3 * torch.randn(N, generator=g)).float()
    for b in (0.8, 1.28):                          # fp64 on both sides; only keep off exact borders
        near = ((lp.double() - old.double()).exp() - b).abs() < 1e-9
        lp[near] += 1e-3
    scale = torch.randn(N, generator=g) if reduction == "none" else None
    for t in (old, adv, ref):
        t[y == IGN] = math.nan
    loss, rows, kl, w, status = F.clipped_policy(*_cuda(-lp, y, old, adv), ref_logp=ref.cuda(), clip_high=0.28, kl_coef=0.1,
                                                 reduction=reduction, row_scale=None if scale is None else scale.cuda())
    valid = (y != IGN).numpy()
    L, dL, rkl = O.clipped_policy(lp, valid, old, adv, ref, 0.2, 0.28, 0.1)
    s = O.row_scale(valid, reduction, None if scale is None else _np(scale))
    assert status.item() == 0
    # fp64 arithmetic (a few 2^-53, sums of N terms), fp32 outputs
    _close(loss.item(), (s * L).sum(), (np.abs(s * L).sum() + 1e-300) * (N + 50) * 2.0 ** -53, "loss")
    _close(_np(rows), L, np.abs(L) * EPS32 * 1.001 + 1e-13, "rows")
    _close(_np(kl), rkl, np.abs(rkl) * EPS32 * 1.001 + 1e-14, "kl")
    _close(_np(w), -dL * s, np.abs(dL * s) * EPS32 * 1.001 + np.abs(s) * 1e-13, "weight")


# ------------------------------------------------------------ through the head --


def _head(N, H, V, seed=0, ign=0.2):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(N, H, generator=g).bfloat16()
    W = (torch.randn(V, H, generator=g) * 1.5 / math.sqrt(H)).bfloat16()
    Z = X.double() @ W.double().T
    _, y, _, adv, _ = policy_case(N, V, seed=seed, ign=ign)
    lp = torch.log_softmax(Z, 1)[torch.arange(N), y.long().clamp(min=0)]
    delta = 0.3 * torch.randn(N, generator=g, dtype=torch.float64)
    for b in (math.log(0.8), math.log(1.28)):
        delta = torch.where((delta - b).abs() < 1e-3, b + 2e-3, delta)
    return X, W, Z, y, (lp - delta).float(), adv, (lp - 0.3 * torch.randn(N, generator=g, dtype=torch.float64)).float()


# A head's logits are fp32 sums of H bf16 products: |error| <= H 2^-24 sum |x w|
# bounds them, a few 1e-6 of the logits' scale in practice.  The losses are held
# to the library's 1e-4 and the gradients to its bounds, log-probabilities to
# 1e-4 absolute.
HEAD_SIZES = [(1, 8, 1), (1, 64, 300), (5, 16, 33), (256, 256, 4096), (300, 264, 5003), (515, 136, 2049), (700, 64, 9000)]


@pytest.mark.parametrize("N,H,V", HEAD_SIZES)
@pytest.mark.parametrize("kl,reduction", [(0.0, "mean"), (0.1, "mean"), (0.05, "none"), (0.05, "sum")])
def test_policy_head(N, H, V, kl, reduction):
    F = _lib()
    X, W, Z, y, old, adv, ref = _head(N, H, V, seed=N, ign=0.0 if N < 5 else 0.2)
    scale = torch.randn(N, generator=torch.Generator().manual_seed(1)) if reduction == "none" else None
    d = _cuda(X, W, y, old, adv)
    loss, status, lp, dX, dW = F.policy_forward_backward(*d, ref_logp=ref.cuda() if kl else None, clip_high=0.28,
                                                         kl_coef=kl, reduction=reduction,
                                                         grad_row_scale=None if scale is None else scale.cuda())
    assert status.item() == 0
    rloss, G, rlp, _, _ = O.policy_reference(Z, y, old, adv, ref if kl else None, 0.2, 0.28, kl, reduction=reduction,
                                             grad_row_scale=None if scale is None else _np(scale))
    _close(_np(lp), rlp, 1e-4, "logp")
    s = np.abs(O.row_scale(_np(y) != IGN, reduction, None if scale is None else _np(scale)))
    _close(loss.item(), rloss, (s * (np.abs(_np(adv)) * 2 + kl)).sum() * 1e-4 + 1e-12, "loss")
    if V > 1:
        assert_grad_close(_np(dX), G @ _np(W), "dX")
        assert_grad_close(_np(dW), G.T @ _np(X), "dW")
    fl, fs, flp, nX, nW = F.policy_forward_backward(*d, ref_logp=ref.cuda() if kl else None, clip_high=0.28, kl_coef=kl,
                                                    reduction=reduction, grads=False,
                                                    grad_row_scale=None if scale is None else scale.cuda())
    assert nX is None and nW is None and torch.equal(fl, loss) and torch.equal(flp, lp)


@pytest.mark.parametrize("N,H,V", HEAD_SIZES)
@pytest.mark.parametrize("K,T,ce", [(1, 1.0, 0.0), (16, 2.0, 0.0), (64, 1.0, 0.5), (300, 1.0, 0.25)])
def test_distill_head(N, H, V, K, T, ce):
    F = _lib()
    X, W, Z, y, *_ = _head(N, H, V, seed=N + K, ign=0.0 if N < 5 else 0.2)
    ids, u = teacher_case(N, V, K, seed=V, dtype=torch.bfloat16)
    if N > 4:
        ids[3] = -1
        ids[4] = torch.arange(K, dtype=torch.int32).clamp(max=V - 1)  # clustered at the start of the vocabulary
    d = _cuda(X, W, y, ids, u)
    loss, status, rows, dX, dW = F.distill_forward_backward(*d, temperature=T, ce_weight=ce, row_loss=True)
    assert status.item() == 0
    rloss, G, rrows = O.distill_reference(Z, y, ids, u, None, T, 1.0, ce)
    _close(_np(rows), rrows, 1e-4 * (1 + np.abs(rrows)), "row loss")
    _close(loss.item(), rloss, 1e-4 * (1 + abs(rloss)), "loss")
    if V > 1:
        assert_grad_close(_np(dX), G @ _np(W), "dX")
        assert_grad_close(_np(dW), G.T @ _np(X), "dW")
    fl, _, frows, nX, nW = F.distill_forward_backward(*d, temperature=T, ce_weight=ce, row_loss=True, grads=False)
    assert nX is None and nW is None and torch.equal(fl, loss) and torch.equal(frows, rows)


@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_heads_with_reordered_rows(reduction):
    """Scattered ignored rows and a workspace that lets the call reorder: the
    same results, in the caller's order."""
    F = _lib()
    N, H, V, K = 1300, 64, 3000, 20
    X, W, Z, y, old, adv, ref = _head(N, H, V, seed=4, ign=0.6)
    ids, u = teacher_case(N, V, K, seed=4)
    scale = torch.randn(N, generator=torch.Generator().manual_seed(1)).cuda() if reduction == "none" else None
    nscale = None if scale is None else _np(scale)
    d = _cuda(X, W, y)
    ws = F.alloc_workspace(N, H, V, reorder=True)
    loss, status, lp, dX, dW = F.policy_forward_backward(*d, *_cuda(old, adv), ref_logp=ref.cuda(), clip_high=0.28,
                                                         kl_coef=0.05, workspace=ws, reduction=reduction,
                                                         grad_row_scale=scale)
    assert F.row_order_info(ws)[0] and status.item() == 0
    rloss, G, rlp, _, _ = O.policy_reference(Z, y, old, adv, ref, 0.2, 0.28, 0.05, reduction=reduction, grad_row_scale=nscale)
    _close(_np(lp), rlp, 1e-4, "logp")
    assert_grad_close(_np(dX), G @ _np(W), "dX")
    assert_grad_close(_np(dW), G.T @ _np(X), "dW")
    ws = torch.empty(F.distill_workspace_size(N, H, V, K, True), dtype=torch.uint8, device="cuda")
    loss, status, rows, dX, dW = F.distill_forward_backward(*d, *_cuda(ids, u), ce_weight=0.5, workspace=ws, row_loss=True,
                                                            reduction=reduction, grad_row_scale=scale)
    assert F.row_order_info(ws)[0] and status.item() == 0
    rloss, G, rrows = O.distill_reference(Z, y, ids, u, None, 1.0, 1.0, 0.5, reduction=reduction, grad_row_scale=nscale)
    _close(_np(rows), rrows, 1e-4 * (1 + np.abs(rrows)), "row loss")
    assert_grad_close(_np(dX), G @ _np(W), "dX")
    assert_grad_close(_np(dW), G.T @ _np(X), "dW")


@pytest.mark.parametrize("N,H,V", [(700, 64, 60000), (3, 1024, 30000), (260, 520, 20011), (513, 136, 70001)])
def test_heads_on_both_workspaces(N, H, V):
    """The heads' own workspace (wide chunks, dX in several vocabulary ranges,
    one or more chunks) and the cross-entropy head's: both agree with the
    oracle, in the caller's row order where rows are reordered too."""
    F = _lib()
    X, W, Z, y, old, adv, ref = _head(N, H, V, seed=N, ign=0.0 if N < 5 else 0.55)
    d = _cuda(X, W, y, old, adv)
    rloss, G, rlp, _, _ = O.policy_reference(Z, y, old, adv, None, 0.2, 0.28)
    rX, rW = G @ _np(W), G.T @ _np(X)
    sizes = (F.policy_workspace_size(N, H, V), F.policy_workspace_size(N, H, V, True), F.workspace_size(N, H))
    for nbytes in sizes:
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        loss, status, lp, dX, dW = F.policy_forward_backward(*d, clip_high=0.28, workspace=ws)
        assert status.item() == 0
        _close(_np(lp), rlp, 1e-4, "logp")
        assert_grad_close(_np(dX), rX, "dX")
        assert_grad_close(_np(dW), rW, "dW")
        again = F.policy_forward_backward(*d, clip_high=0.28, workspace=ws)
        assert torch.equal(again[3], dX) and torch.equal(again[4], dW)


def test_policy_step_as_separate_calls():
    """Row losses, clipped_policy, weighted gradients: the same step as
    policy_forward_backward, and as policy_loss on the logits."""
    F = _lib()
    X, W, Z, y, old, adv, ref = _head(400, 128, 3000, seed=21)
    Xd, Wd, yd, od, ad, rd = _cuda(X, W, y, old, adv, ref)
    _, st1, row_loss, _, _ = F.forward_backward_ex(Xd, Wd, yd, reduction="none", row_loss=True, grads=False)
    loss, rows, kl, weight, st2 = F.clipped_policy(row_loss, yd, od, ad, ref_logp=rd, kl_coef=0.05)
    _, st3, _, dX, dW = F.forward_backward_ex(Xd, Wd, yd, reduction="none", grad_row_scale=weight)
    floss, st4, lp, fX, fW = F.policy_forward_backward(Xd, Wd, yd, od, ad, ref_logp=rd, kl_coef=0.05)
    assert not any(int(s.item()) for s in (st1, st2, st3, st4))
    assert abs(loss.item() - floss.item()) <= 1e-6 * (1 + abs(loss.item()))
    assert torch.equal(lp, -row_loss)
    assert_grad_close(_np(fX), _np(dX), "dX")
    assert_grad_close(_np(fW), _np(dW), "dW")
    logits = (Xd.float() @ Wd.float().T)
    zloss, _, zlp, _, _, _ = F.policy_loss(logits, yd, od, ad, ref_logp=rd, kl_coef=0.05)
    assert abs(zloss.item() - floss.item()) <= 1e-4


def test_distill_head_is_cross_entropy_without_a_teacher():
    F = _lib()
    X, W, Z, y, *_ = _head(300, 64, 1000, seed=22)
    ids = torch.full((300, 4), -1, dtype=torch.int32)
    d = _cuda(X, W, y)
    loss, _, rows, dX, dW = F.distill_forward_backward(*d, *_cuda(ids, torch.zeros(300, 4)), ce_weight=1.0, row_loss=True)
    closs, _, crows, cX, cW = F.forward_backward_ex(*d, row_loss=True)
    assert abs(loss.item() - closs.item()) <= 1e-6 * closs.item()
    assert_grad_close(_np(dX), _np(cX), "dX")
    assert_grad_close(_np(dW), _np(cW), "dW")


def test_head_mean_count():
    F = _lib()
    X, W, Z, y, old, adv, ref = _head(300, 64, 1000, seed=23)
    ids, u = teacher_case(300, 1000, 8)
    n = int((y != IGN).sum())
    cnt = torch.tensor([2 * n], dtype=torch.int32).cuda()
    d = _cuda(X, W, y)
    for f, a in ((F.policy_forward_backward, _cuda(old, adv)), (F.distill_forward_backward, _cuda(ids, u))):
        whole, half = f(*d, *a), f(*d, *a, mean_count=cnt)
        assert abs(half[0].item() - whole[0].item() / 2) <= 1e-6 * abs(whole[0].item())
        assert_grad_close(_np(half[3]) * 2, _np(whole[3]), "dX")


# ------------------------------------------------- streams, graphs, repetition --


def _calls(F):
    """Every operator on one set of inputs: [(name, call(stream, scratch) -> outputs)]."""
    Z, y, old, adv, ref = policy_case(64, 3001, seed=31, dtype=torch.bfloat16)
    ids, u = teacher_case(64, 3001, 24, seed=31)
    X, W, _, hy, hold, hadv, href = _head(64, 64, 3001, seed=32)
    Zd, yd, od, ad, rd, idd, ud = _cuda(Z, y, old, adv, ref, ids, u)
    Xd, Wd, hyd, hod, had = _cuda(X, W, hy, hold, hadv)
    kw = dict(ref_logp=rd, kl_coef=0.1)
    return [("clipped_policy", lambda s=None: F.clipped_policy(-od, yd, rd, ad, stream=s)),
            ("policy_loss", lambda s=None: F.policy_loss(Zd, yd, od, ad, entropy_coef=0.01, stream=s, **kw)),
            ("distill_topk", lambda s=None: F.distill_topk(Zd, yd, idd, ud, ce_weight=0.5, temperature=2.0, row_loss=True,
                                                           stream=s)),
            ("policy_forward_backward", lambda s=None: F.policy_forward_backward(Xd, Wd, hyd, hod, had, stream=s)),
            ("distill_forward_backward", lambda s=None: F.distill_forward_backward(Xd, Wd, hyd, idd, ud, row_loss=True,
                                                                                   stream=s))]


def test_same_bits_every_time_and_on_another_stream():
    F = _lib()
    side = torch.cuda.Stream()
    for name, call in _calls(F):
        first = call()
        torch.cuda.synchronize()
        again = call()
        side.wait_stream(torch.cuda.current_stream())
        other = call(side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(first, again, other):
            if a is not None:
                assert torch.equal(a, b) and torch.equal(a, c), name


def test_two_streams_at_once():
    F = _lib()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for name, call in _calls(F)[:3]:
        want = call()
        torch.cuda.synchronize()
        got = [[call(s) for s in streams] for _ in range(10)]
        torch.cuda.synchronize()
        for pair in got:
            for out in pair:
                for a, b in zip(want, out):
                    if a is not None:
                        assert torch.equal(a, b), name


def test_graph_replays_on_new_inputs():
    """Captured once, replayed on other values in the same buffers: the result
    of an eager call on those values."""
    F = _lib()
    cases = [policy_case(48, 2000, seed=s, dtype=torch.bfloat16) for s in (41, 42)]
    teachers = [teacher_case(48, 2000, 10, seed=s) for s in (41, 42)]
    Zd, yd, od, ad, rd = _cuda(*cases[0])
    idd, ud = _cuda(*teachers[0])
    X, W = torch.randn(48, 64).bfloat16().cuda(), (torch.randn(2000, 64) * 0.2).bfloat16().cuda()

    def step():
        return (F.clipped_policy(-od, yd, rd, ad), F.policy_loss(Zd, yd, od, ad, ref_logp=rd, kl_coef=0.1),
                F.distill_topk(Zd, yd, idd, ud, row_loss=True), F.policy_forward_backward(X, W, yd, od, ad),
                F.distill_forward_backward(X, W, yd, idd, ud, row_loss=True))

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, each with scratch of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for t, src in zip((Zd, yd, od, ad, rd), cases[1]):
        t.copy_(src)
    idd.copy_(teachers[1][0])
    ud.copy_(teachers[1][1])
    graphs[0][0].replay()
    graphs[1][0].replay()
    graphs[0][0].replay()
    want = step()
    torch.cuda.synchronize()
    for _, out in graphs:
        for a, b in zip(want, out):
            for x, z in zip(a, b):
                if x is not None:
                    assert torch.equal(x, z)


def test_workspace_refusals_on_device():
    F = _lib()
    Z, y, old, adv, ref = policy_case(64, 100)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        F.policy_loss(*_cuda(Z, y, old, adv), workspace=small)
    with pytest.raises(ValueError, match="advantages"):
        F.policy_loss(*_cuda(Z, y, old, adv[:63]))
    with pytest.raises(ValueError, match="old_logp"):
        F.policy_loss(*_cuda(Z, y, old.double(), adv))
    with pytest.raises(ValueError, match="reduction"):
        F.policy_loss(*_cuda(Z, y, old, adv), grad_row_scale=adv.cuda())
    with pytest.raises(ValueError, match="columns"):
        F.distill_topk(*_cuda(Z, y, torch.zeros(64, 1025, dtype=torch.int32), torch.zeros(64, 1025)))
    with pytest.raises(F.FlceError, match="INVALID_ARGUMENT"):
        F.policy_loss(*_cuda(Z, y, old, adv), kl_coef=0.1)
    with pytest.raises(F.FlceError, match="INVALID_ARGUMENT"):
        F.policy_loss(*_cuda(Z, y, old, adv), temperature=0.0)
    X = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    ids, u = teacher_case(64, 64, 3)
    with pytest.raises(F.FlceError, match="UNSUPPORTED"):
        F.distill_forward_backward(X, X, *_cuda(y, ids, u), temperature=2.0, ce_weight=0.5)
    with pytest.raises(F.FlceError, match="WORKSPACE"):
        F.distill_forward_backward(X, X, *_cuda(y, ids, u), workspace=F.alloc_workspace(64, 64))
