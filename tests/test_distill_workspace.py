"""precond_distill_workspace of a type that the call does not take raises, as the call does."""
import pytest
import torch

import shampoo_roots_gb300 as sr


def test_types():
    assert sr.precond_distill_workspace(2000, 1000, 5, torch.float32) == 16000
    assert sr.precond_distill_workspace(2000, 1000, 5, torch.bfloat16) == 16000
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError):
            sr.precond_distill_workspace(2000, 1000, 5, dtype)
