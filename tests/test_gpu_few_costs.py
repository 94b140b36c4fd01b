"""few_token_moe with as many costs beyond one as there can be, in neighbouring experts and spread over all groups of 32."""

import pytest

from tests.few_costs import most_costs
from tests.gpu_util import require_gpu
from tests.test_gpu_few_tokens import Layer, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("E,start,step,S", [(41, 0, 1, 0), (64, 23, 1, 128), (1024, 5, 25, 0)])
def test_most_costs(fmt, E, start, step, S):
    dev = require_gpu()
    layer = Layer(dev, E, 128, 128, S, fmt=fmt, seed=E)
    x, _, p = inputs(dev, 32, 128, E, 32, E)
    ids = most_costs(E, start, step).to(dev)
    layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_32_experts_of_all_tokens(fmt):
    dev = require_gpu()
    layer = Layer(dev, 70, 256, 128, fmt=fmt, seed=2)
    x, ids, p = inputs(dev, 32, 256, 70, 32, 2)
    ids[:] = ids[0]
    layer.check(layer.call(x, ids, p), x, ids, p)
