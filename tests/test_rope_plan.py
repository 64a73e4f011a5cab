"""A rotation kept by a model is copied and pickled with it: the copy stands alone and turns by the same angles."""
import copy
import ctypes
import gc
import pickle

import pytest

import activation_sparse_gemm_b200 as rl

PLANS = [dict(axes=(44, 42, 42)), dict(axes=(128,), theta=1e6, pairing=rl.ROPE_HALF),
         dict(axes=(8, 4), inv_freq=[0.5, 0.25, 0.1, 0.0, 2.0, 1e-3])]


def fields(plan):
    """What the library reads at the address that the calls pass."""
    specs = (rl.RopeSpec * 3).from_address(plan._at)
    return [(s.n_axes, list(s.axis_dim), s.pairing, s.pos_type, s.theta, s.inv_freq[:sum(plan.axes) // 2]) for s in specs]


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))],
                         ids=["copy", "deepcopy", "pickle"])
@pytest.mark.parametrize("kwargs", PLANS, ids=str)
def test_copies(kwargs, how):
    plan = rl.Rope(**kwargs)
    plan.note = "kept"
    want = fields(plan)
    other = how(plan)
    assert other.axes == plan.axes and other.note == "kept"
    assert other._at != plan._at
    assert ctypes.addressof(other.specs[0].inv_freq.contents) != ctypes.addressof(plan.specs[0].inv_freq.contents)
    assert [type(s) for s in other.specs] == [rl.RopeSpec] * 3 and want[0][2] == kwargs.get("pairing", 0)
    del plan
    gc.collect()
    assert fields(other) == want
    assert fields(how(other)) == want


def test_copy_of_a_model_that_holds_one():
    import torch

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.weight = torch.nn.Parameter(torch.ones(4))
            self.plan = rl.Rope((16, 16))

    block = Block()
    twin = copy.deepcopy(block)
    assert fields(twin.plan) == fields(block.plan) and twin.plan is not block.plan
