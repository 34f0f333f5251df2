"""Post-training losses without a GPU: the fp64 oracle's clipped policy loss and
top-logit distillation against torch fp64 autograd, finite differences and
closed forms, and the library's and the binding's refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import flce_oracle as O

IGN = -100


def policy_case(N, V, seed=0, dtype=torch.float32, std=2.0, ign=0.2, temperature=1.0):
    """Logits, targets and per-row vectors; log-ratios spread over both clip
    borders (0.8 and 1.28) and kept 1e-3 away from them."""
    g = torch.Generator().manual_seed(seed)
    Z = (torch.randn(N, V, generator=g) * std).to(dtype)
    y = torch.randint(0, V, (N,), generator=g, dtype=torch.int64).to(torch.int32)
    lp = torch.log_softmax(Z.double() / temperature, 1)[torch.arange(N), y.long()]
    delta = 0.3 * torch.randn(N, generator=g, dtype=torch.float64)
    for b in (math.log(0.8), math.log(1.28)):
        delta = torch.where((delta - b).abs() < 1e-3, b + 2e-3, delta)
    old = (lp - delta).float()
    ref = (lp - 0.3 * torch.randn(N, generator=g, dtype=torch.float64)).float()
    adv = torch.randn(N, generator=g)
    k = int(ign * N)
    if k:
        y[torch.randperm(N, generator=g)[:k]] = IGN
    return Z, y, old, adv, ref


def teacher_case(N, V, K, seed=0, dtype=torch.float32, padded=True, duplicates=False):
    g = torch.Generator().manual_seed(seed + 1000)
    if duplicates or K > V:
        ids = torch.randint(0, V, (N, K), generator=g)
    else:
        ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)])
    if padded and K > 1:
        ids[torch.rand(N, K, generator=g) < 0.15] = -1
    u = (torch.randn(N, K, generator=g) * 2 + 3).to(dtype)
    return ids.to(torch.int32), u


def _torch_policy(Z, y, old, adv, ref, kl_coef, ent_coef, T):
    z = Z.double().clone().requires_grad_(True)
    valid = y != IGN
    lp_all = torch.log_softmax(z / T, 1)
    lp = lp_all.gather(1, torch.where(valid, y, 0).long()[:, None])[:, 0]
    r = (lp - old.double()).exp()
    A = adv.double()
    L = -torch.min(r * A, r.clamp(0.8, 1.28) * A)
    d = ref.double() - lp
    kl = d.exp() - d - 1
    H = -(lp_all.exp() * lp_all).sum(1)
    L = L + kl_coef * kl - ent_coef * H
    loss = L[valid].mean() if valid.any() else (L * 0).sum()
    loss.backward()
    return loss.item(), z.grad.numpy(), (lp * valid).detach().numpy(), (H * valid).detach().numpy(), (kl * valid).detach().numpy()


@pytest.mark.parametrize("kl,ent,T", [(0.0, 0.0, 1.0), (0.1, 0.0, 1.0), (0.05, 0.02, 0.7), (0.0, 0.1, 2.0)])
def test_oracle_policy_against_autograd(kl, ent, T):
    Z, y, old, adv, ref = policy_case(40, 60, temperature=T)
    want = _torch_policy(Z, y, old, adv, ref, kl, ent, T)
    got = O.policy_reference(Z, y, old, adv, ref, 0.2, 0.28, kl, ent, T)
    assert abs(got[0] - want[0]) <= 1e-12
    for a, b in zip(got[1:], want[1:]):
        np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-13)


def _torch_distill(Z, y, ids, u, T, kd, ce):
    z = Z.double().clone().requires_grad_(True)
    valid = y != IGN
    uu = (u.double() / T).masked_fill(ids < 0, -math.inf)
    some = (ids >= 0).any(1)
    q = torch.softmax(torch.where(some[:, None], uu, 0.0), 1) * some[:, None]
    logq = torch.log_softmax(torch.where(some[:, None], uu, 0.0), 1)
    logp = torch.log_softmax(z / T, 1).gather(1, ids.long().clamp(min=0))
    L = kd * torch.where(ids >= 0, q * (torch.where(ids >= 0, logq, 0.0) - logp), 0.0).sum(1)
    lp1 = torch.log_softmax(z, 1).gather(1, torch.where(valid, y, 0).long()[:, None])[:, 0]
    L = (L - ce * lp1) * valid
    loss = L.sum() / max(1, int(valid.sum()))
    loss.backward()
    return loss.item(), z.grad.numpy(), L.detach().numpy()


@pytest.mark.parametrize("T,kd,ce,dup", [(1.0, 1.0, 0.0, False), (2.5, 0.8, 0.0, True), (1.0, 0.5, 0.5, False),
                                         (2.0, 4.0, 0.3, True)])
def test_oracle_distill_against_autograd(T, kd, ce, dup):
    Z, y, *_ = policy_case(30, 50)
    ids, u = teacher_case(30, 50, 7, duplicates=dup)
    ids[3] = -1
    loss, dZ, rows = O.distill_reference(Z, y, ids, u, None, T, kd, ce)
    want = _torch_distill(Z, y, ids, u, T, kd, ce)
    assert abs(loss - want[0]) <= 1e-12
    np.testing.assert_allclose(dZ, want[1], rtol=1e-9, atol=1e-13)
    np.testing.assert_allclose(rows, want[2], rtol=1e-9, atol=1e-13)


def test_oracle_gradients_against_differences():
    Z, y, old, adv, ref = policy_case(4, 9, ign=0.0)
    ids, u = teacher_case(4, 9, 3, padded=False)
    lse = torch.logsumexp(u.double(), 1).float() + 0.4
    z0 = Z.double().numpy()
    fs = [lambda z: O.policy_reference(z, y, old, adv, ref, 0.2, 0.28, 0.1, 0.05, 1.3),
          lambda z: O.distill_reference(z, y, ids, u, lse, 1.0, 1.0, 0.25)]
    for f in fs:
        G = f(z0)[1]
        h = 1e-5
        for i in range(4):
            for j in range(9):
                zp, zm = z0.copy(), z0.copy()
                zp[i, j] += h
                zm[i, j] -= h
                d = (f(zp)[0] - f(zm)[0]) / (2 * h)
                # central differences: h^2/6 of a third derivative of order 10
                assert abs(d - G[i, j]) <= 1e-9 + 1e-7 * abs(G[i, j])


def test_oracle_closed_forms():
    # ratio 1, no KL: the policy loss is -mean advantage and its gradient the
    # advantage-weighted cross-entropy's
    Z, y, old, adv, ref = policy_case(12, 20, ign=0.0)
    loss, dZ, *_ = O.policy_reference(Z, y, None, adv, None)
    assert abs(loss + adv.double().mean().item()) <= 1e-12
    _, dce, *_ = O.ce_reference(Z, y, reduction="none", grad_row_scale=adv.double().numpy() / 12)
    np.testing.assert_allclose(dZ, dce, rtol=1e-12, atol=1e-15)
    # a teacher with one entry at the target is cross-entropy
    loss, dZ, _ = O.distill_reference(Z, y, y[:, None], torch.zeros(12, 1))
    ref_loss, ref_dZ, *_ = O.ce_reference(Z, y)
    assert abs(loss - ref_loss) <= 1e-12
    np.testing.assert_allclose(dZ, ref_dZ, rtol=1e-12, atol=1e-15)
    # a teacher equal to the student over the whole vocabulary costs nothing
    ids = torch.arange(20, dtype=torch.int32).repeat(12, 1)
    loss, dZ, _ = O.distill_reference(Z, y, ids, Z, temperature=3.0)
    assert abs(loss) <= 1e-14 and np.abs(dZ).max() <= 1e-15


# ------------------------------------------------------------------ refusals --


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_03_b200 import flce
    return flce.load_library()


FAKE = 1 << 20
INF, NAN = math.inf, math.nan


def _clipped(lib, **kw):
    a = dict(row_loss=FAKE, y=FAKE, N=8, ign=-100, old=FAKE, adv=FAKE, ref=FAKE, lo=0.2, hi=0.2, kl=0.1, red=0, scale=None,
             loss=FAKE, rows=FAKE, out_kl=FAKE, w=FAKE, status=FAKE, ws=FAKE, nbytes=1 << 20)
    a.update(kw)
    return lib.flce_clipped_policy(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(row_loss=None), 1), (dict(adv=None), 1), (dict(w=None), 1), (dict(ws=None, N=5000), 1), (dict(N=0), 1),
    (dict(N=(1 << 30) + 1), 1), (dict(lo=-0.1), 1), (dict(lo=1.1), 1), (dict(hi=NAN), 1), (dict(kl=INF), 1),
    (dict(ref=None), 1), (dict(red=3), 1), (dict(loss=FAKE + 4), 2), (dict(adv=FAKE + 2), 2), (dict(ws=FAKE + 128), 2),
    (dict(nbytes=64, N=5000), 3)])
def test_clipped_policy_refusals(lib, kw, status):
    assert _clipped(lib, **kw) == status


def _policy(lib, **kw):
    a = dict(z=FAKE, dt=0, ld=64, y=FAKE, N=8, V=60, ign=-100, T=1.0, old=FAKE, adv=FAKE, ref=FAKE, lo=0.2, hi=0.2, kl=0.1,
             ent=0.0, red=0, scale=None, loss=FAKE, logp=FAKE, H=FAKE, out_kl=FAKE, status=FAKE, dz=FAKE, ldg=64, ws=FAKE,
             nbytes=1 << 20)
    a.update(kw)
    return lib.flce_policy_loss(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None, dz=None), 1), (dict(dt=3), 1), (dict(ld=59, ldg=59), 1), (dict(ldg=59), 1), (dict(ldg=65), 1),
    (dict(dz=FAKE + 2), 1), (dict(dz=FAKE + (7 * 64 + 60) * 2 - 2), 1), (dict(V=0), 1), (dict(T=0.0), 1), (dict(T=-1.0), 1),
    (dict(T=NAN), 1), (dict(T=INF), 1), (dict(T=1e-7), 1), (dict(T=2e6), 1), (dict(ent=NAN), 1), (dict(logp=None), 1), (dict(H=None), 1),
    (dict(z=FAKE + 1, dz=FAKE + 1), 2), (dict(status=FAKE + 2), 2), (dict(nbytes=100), 3)])
def test_policy_loss_refusals(lib, kw, status):
    assert _policy(lib, **kw) == status


def _distill(lib, **kw):
    a = dict(z=FAKE, dt=0, ld=64, y=FAKE, N=8, V=60, ign=-100, ids=FAKE, u=FAKE, ut=0, K=4, lse=None, T=1.0, kd=1.0, ce=0.0,
             red=0, scale=None, loss=FAKE, rows=FAKE, status=FAKE, dz=FAKE, ldg=64, ws=FAKE, nbytes=1 << 20)
    a.update(kw)
    return lib.flce_distill_topk(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), 1), (dict(u=None), 1), (dict(ut=7), 1), (dict(K=0), 1), (dict(K=1025), 1), (dict(T=0.0), 1),
    (dict(kd=NAN), 1), (dict(ce=INF), 1), (dict(ids=FAKE + 2), 2), (dict(u=FAKE + 1), 2), (dict(loss=FAKE + 1), 2),
    (dict(nbytes=0), 3)])
def test_distill_topk_refusals(lib, kw, status):
    assert _distill(lib, **kw) == status


def _head_distill(lib, **kw):
    a = dict(X=FAKE, W=FAKE, y=FAKE, N=8, H=64, V=60, ign=-100, ids=FAKE, u=FAKE, ut=0, K=4, lse=None, T=1.0, kd=1.0, ce=0.5,
             red=0, scale=None, cnt=None, loss=FAKE, rows=None, status=FAKE, dX=FAKE, dW=FAKE, ws=FAKE, nbytes=1 << 30)
    a.update(kw)
    return lib.flce_distill_forward_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), 1), (dict(dX=None), 1), (dict(loss=None), 1), (dict(K=2000), 1), (dict(H=60), 2), (dict(T=2.0), 2),
    (dict(X=FAKE + 8), 2), (dict(nbytes=1 << 10), 3)])
def test_distill_head_refusals(lib, kw, status):
    assert _head_distill(lib, **kw) == status


def _head_policy(lib, **kw):
    a = dict(X=FAKE, W=FAKE, y=FAKE, N=8, H=64, V=60, ign=-100, old=FAKE, adv=FAKE, ref=None, lo=0.2, hi=0.2, kl=0.0, red=0,
             scale=None, cnt=None, loss=FAKE, logp=FAKE, status=FAKE, dX=FAKE, dW=FAKE, ws=FAKE, nbytes=1 << 30)
    a.update(kw)
    return lib.flce_policy_forward_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(adv=None), 1), (dict(logp=None), 1), (dict(dW=None), 1), (dict(kl=0.1), 1), (dict(hi=-0.5), 1), (dict(H=4), 2),
    (dict(old=FAKE + 1), 2), (dict(nbytes=1 << 10), 3)])
def test_policy_head_refusals(lib, kw, status):
    assert _head_policy(lib, **kw) == status


def test_workspace_sizes(lib):
    from lm_head_linear_03_b200 import flce
    import lm_head_linear_03_b200 as F
    area = flce.packed_x_bytes(300, 264)
    for V in (1, 2048, 5003, 128256):
        assert F.policy_workspace_size(300, 264, V) >= flce.workspace_size(300, 264)
        assert F.distill_workspace_size(300, 264, V, 16) > F.policy_workspace_size(300, 264, V)
        assert F.policy_workspace_size(300, 264, V, True) - F.policy_workspace_size(300, 264, V) == area
        assert F.distill_workspace_size(300, 264, V, 16, True) - F.distill_workspace_size(300, 264, V, 16) == area
    # a wider chunk buffer stays within 64 MB; dX's shares exist for fewer than 74
    # tiles of 256 x 256, at most 148 + 73 tiles of fp32 in all
    for N in (1, 300, 2048, 8192, 32768):
        for H in (8, 256, 4096):
            extra = F.policy_workspace_size(N, H, 256000) - flce.workspace_size(N, H)
            assert 0 <= extra <= (64 << 20) + 221 * 256 * 256 * 4 + 4096
    for bad in ((0, 264, 10), (300, 260, 10), (300, 264, 0)):
        assert F.policy_workspace_size(*bad) == 0 and F.distill_workspace_size(*bad, 4) == 0
    for K in (0, 1025):
        assert F.distill_workspace_size(300, 264, 10, K) == 0


def test_binding_refuses_before_any_call(lib):
    import lm_head_linear_03_b200 as F
    Z, y, old, adv, ref = policy_case(8, 16)
    ids, u = teacher_case(8, 16, 3)
    with pytest.raises(ValueError, match="CUDA"):
        F.policy_loss(Z, y, old, adv)
    with pytest.raises(ValueError, match="CUDA"):
        F.distill_topk(Z, y, ids, u)
    with pytest.raises(ValueError, match="CUDA"):
        F.clipped_policy(old, y, old, adv)
    with pytest.raises(ValueError, match="adjacent"):
        F.policy_loss(Z.t(), y, old, adv)
    with pytest.raises(ValueError, match="adjacent"):
        F.policy_loss(Z[:1].expand(8, 16), y, old, adv)
    with pytest.raises(ValueError, match="expected"):
        F.policy_loss(Z.double(), y, old, adv)
    X = torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.distill_forward_backward(X, X, y, ids, u)
    with pytest.raises(ValueError, match="CUDA"):
        F.policy_forward_backward(X, X, y, old, adv)
