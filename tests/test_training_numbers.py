"""Numbers of the calls may be anything that Python takes for a float: an int, numpy's, a tensor of one element."""
import numpy as np
import pytest
import torch

import shampoo_roots_gb300 as sr
from test_training_refusals import h  # noqa: F401  (a host-only handle)

f = lambda *s: torch.zeros(*s)  # noqa: E731


@pytest.mark.parametrize("one", [1, 1.0, np.float32(1), np.float64(1), np.float16(1), np.int64(1), torch.tensor(1.0)], ids=lambda v: type(v).__name__)
def test_numbers(h, one):  # noqa: F811
    assert sr.precond_rms_norm(h, f(6, 64), f(64), one, y=f(6, 64), stream=0, raw=True) == sr.ENODEV
    assert sr.precond_layer_norm(h, f(6, 64), f(64), one, bias=f(64), y=f(6, 64), stream=0, raw=True) == sr.ENODEV
    assert sr.precond_policy(h, f(6, 50), torch.zeros(6, dtype=torch.int64), advantage=f(6), ref_logp=f(6), temperature=one, clip_low=one,
                             clip_high=one, kl=one, loss=f(6), stream=0, raw=True) == sr.ENODEV
    assert sr.precond_clip_grads(h, [f(64)], one, f(1), stream=0, raw=True) == sr.ENODEV
