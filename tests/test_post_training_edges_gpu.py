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
from test_post_training_gpu import DT, EPS32, _check_distill, _check_policy, _close, _cuda, _delta, _head, _lib, _np

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
