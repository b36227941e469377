"""Calls of the serving operators that a program may make and the other files do not."""
import pytest
import torch

import sparse_compressed_attention_gb300 as V
from tests.tree_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["whole", "few_parts", "many_parts", "nothing_to_see", "f32", "bf16_cuda_cores"])
def test_sinks_that_are_no_numbers(kind):
    """A NaN sink makes its head NaN, one of +inf takes all of it (o = 0, lse = +inf), one of -inf is none; the other heads
    and rows are as without."""
    kw = {"whole": dict(lens=[20] * 100, nodes=[1] * 100),
          "few_parts": dict(lens=[700, 30], nodes=[1, 1], window=-1),
          "many_parts": dict(lens=[20000], nodes=[1], window=-1),
          "nothing_to_see": dict(lens=[0, 9], nodes=[1, 1], window=0, ratio=128),
          "f32": dict(lens=[300, 40], nodes=[2, 1], H=9, D=64, R=16, dt=torch.float32),
          "bf16_cuda_cores": dict(lens=[300, 40], nodes=[2, 1], H=9)}[kind]
    c = Case(sink=True, seed=31, **kw)
    x = c.device_inputs()
    o0, l0 = c.run(x)
    x["sink"] = x["sink"].clone()
    x["sink"][1], x["sink"][4], x["sink"][6] = float("nan"), float("inf"), float("-inf")
    o, lse = c.run(x)
    assert torch.isnan(o[:, 1].float()).all() and torch.isnan(lse[:, 1]).all()
    assert (o[:, 4] == 0).all() and (lse[:, 4] == float("inf")).all()
    rest = [h for h in range(c.H) if h not in (1, 4, 6)]
    assert torch.equal(o[:, rest], o0[:, rest]) and torch.equal(lse[:, rest], l0[:, rest])
    none = c.run({k: v for k, v in x.items() if k != "sink"})
    assert torch.equal(o[:, 6], none[0][:, 6]) and torch.equal(lse[:, 6], none[1][:, 6])
    assert V.v4_get_device_status() == 0
