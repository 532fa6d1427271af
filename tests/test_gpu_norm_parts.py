"""Gradients of the norms that are left out: the others are what they are with all of them."""

import itertools

import pytest
import torch

from differential_attention_03_gb300 import binding as da
from .test_gpu_block import TYPES, _norm_inputs

pytestmark = pytest.mark.gpu

PARTS = {"dx": ("dx",), "dresidual": ("dresidual",), "dgate": ("dgate",), "dgammas": ("dgamma", "dgamma_post")}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("rows,D,G", [(12, 72, 3), (700, 128, 700), (30, 250, 1), (60, 1001, 4), (600, 1000, 600), (300, 2048, 1), (40, 4104, 40),
                                      (350, 5002, 2)])
@pytest.mark.parametrize("types", list(TYPES))
@pytest.mark.parametrize("post", [False, True])
def test_each_set_of_gradients(rows, D, G, types, post):
    x, res, gate, gp, ga, dy, ds = _norm_inputs(rows, D, types, post, G, rows + D)
    s = da.residual_norm(x, res, gate=gate, scale=0.7, gamma_post=gp, gamma=ga)[1]
    a = dict(gate=gate, scale=0.7, gamma_post=gp, gamma=ga)
    whole = da.residual_norm_backward(x, s, dy, ds, **a)
    assert set(whole) == {"dx", "dresidual", "dgate", "dgamma"} | ({"dgamma_post"} if post else set())
    for n in (1, 2, 3, 4):
        for left in itertools.combinations(PARTS, n):
            got = da.residual_norm_backward(x, s, dy, ds, **a, **{k: False for k in left})
            assert set(got) == set(whole) - {name for k in left for name in PARTS[k]}, left
            for k, t in got.items():
                assert torch.equal(t, whole[k]), (left, k)
    with pytest.raises(ValueError):
        da.residual_norm_backward(x, s, dy, ds, **a, dx=False, out={"dx": torch.empty_like(x)})
    da.device_status()
