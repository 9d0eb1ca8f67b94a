"""Experts that a bias keeps out are not chosen; their scores count in the softmax's sum all the same."""
import math

import pytest
import torch

import gemm_any4_amd as any4
from tests import gpu_util as gu
from tests.test_gpu_route import logits_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    gu.require_gpu()
    any4.lib()


@pytest.mark.parametrize("out", [-math.inf, math.nan])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_beside_experts_that_a_bias_keeps_out(out, score):
    l, k = logits_of(20, 30), 4
    b = torch.zeros(30, device=gu.DEV)
    b[3], b[17] = out, out
    w, ids = any4.route(l, k, bias=b, score=score, renorm=False)
    s = torch.softmax(l.double(), 1) if score == "softmax" else torch.special.expit(l.double())
    left = s.clone()
    left[:, [3, 17]] = -1
    want, order = left.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order[:, :k])
    assert ((w.double() - want[:, :k]).abs() <= 2.0 ** -22 * want[:, :k]).all()
