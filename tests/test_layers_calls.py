"""CPU checks of the sequence-layer wrappers: copies of plans and handles, and calls that are refused before any device is
asked."""
import copy
import pickle

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_b200 as pn


@pytest.mark.parametrize("make", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_copies_are_handles_of_their_own(make):
    """A copy holds a handle of its own, made from the same arguments, and outlives its original (as in the copy of a model
    that holds one)."""
    r = pn.Rotary(64, 5e5, "interleaved", "yarn", 8.0, 2048, 16.0, 2.0, 1.25)
    s = make(r)
    assert s.h and s.h != r.h and s.rot_dim == 64 and s._args == r._args
    a = pn.LinearAttention(4, 2, 64, 96, torch.tensor([0.0, -0.1, -1.0, -9.0]), scale=0.25, dtype=torch.bfloat16)
    b = make(a)
    assert b.h and b.h != a.h
    assert (b.heads, b.kv_heads, b.dk, b.dv, b.scale, b.dtype) == (4, 2, 64, 96, 0.25, torch.bfloat16)
    assert np.array_equal(a._args[4], b._args[4])
    del r, a
    assert pn.lib.pn_linattn_workspace(b.h, 1, 2, 4096, 0, 0) > 0
    both = make([b, s, b])
    del both, s, b
