"""All tensors of a call are on one device: an argument on another one, or several, are refused before anything is
enqueued (stand-ins for tensors that say where they are; a host-only handle, so that a call which
passes returns ENODEV)."""
import pytest
import torch

import shampoo_roots_gb300 as sr
from test_training_refusals import h  # noqa: F401  (a host-only handle)


class On:
    """A tensor's attributes, on device `where`."""

    def __init__(self, t, where):
        self.t, self.where, self.shape, self.dtype = t, where, t.shape, t.dtype

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()

    def data_ptr(self):
        return self.t.data_ptr()

    def get_device(self):
        return self.where


f = lambda *s: torch.zeros(*s)  # noqa: E731
CALLS = {
    "policy": (sr.precond_policy, dict(logits=f(6, 50), ids=torch.zeros(6, dtype=torch.int64), advantage=f(6), old_logp=f(6), ref_logp=f(6),
                                       weight=f(6), loss=f(6), logp=f(6), dlogits=f(6, 50)), dict(kl=0.1)),
    "score": (sr.precond_policy, dict(logits=f(6, 50), ids=torch.zeros(6, dtype=torch.int32), logp=f(6)), {}),
    "norm": (lambda h, grads, **kw: sr.precond_grad_norm(h, [grads], **kw), dict(grads=f(1 << 20), norm=f(1), workspace=f(100000)), {}),
    "clip": (lambda h, grads, **kw: sr.precond_clip_grads(h, [grads], 1.0, **kw), dict(grads=f(1 << 20), norm=f(1), workspace=f(100000)), {}),
    "given": (lambda h, grads, **kw: sr.precond_clip_grads(h, [grads], 1.0, given=True, **kw), dict(grads=f(64), norm=f(1)), {}),
    "layer_norm": (sr.precond_layer_norm, dict(x=f(6, 64), weight=f(64), bias=f(64), residual=f(6, 64), total=f(6, 64), y=f(6, 64), mean=f(6),
                                               rstd=f(6)), dict(eps=1e-5)),
    "layer_norm_grad": (sr.precond_layer_norm_grad, dict(dy=f(6, 64), x=f(6, 64), weight=f(64), mean=f(6), rstd=f(6), dx=f(6, 64), dw=f(64),
                                                         db=f(64), dresidual=f(6, 64), workspace=f(100000)), {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_one_device(h, name):  # noqa: F811
    call, tensors, rest = CALLS[name]
    for here, there in ((0, -1), (0, 1), (1, 0), (-1, 0)):
        on = {k: On(t, here) for k, t in tensors.items()}
        assert call(h, **on, **rest, stream=0, raw=True) == sr.ENODEV
        for k, t in tensors.items():
            with pytest.raises(ValueError, match="one device"):
                call(h, **{**on, k: On(t, there)}, **rest, stream=0, raw=True)
        for n in range(1, len(tensors)):                                   # the first n here, the others there
            with pytest.raises(ValueError, match="one device"):
                call(h, **{k: On(t, here if i < n else there) for i, (k, t) in enumerate(tensors.items())}, **rest, stream=0, raw=True)
