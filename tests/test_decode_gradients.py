"""The decode operators give no gradients: tensors that ask for one are refused, as torch refuses them
for outputs that are given. No GPU is needed."""

import pytest
import torch

from tests.test_decode_binding import handle, lc  # noqa: F401  (fixtures)

X = torch.zeros(3, 2, 128)
I = torch.zeros(4, dtype=torch.int32)


def test_tensors_that_require_gradients_are_refused(lc, handle):
    y = X.clone().requires_grad_()
    calls = {
        "q": (lambda t: lc.ar_qk_norm_rope(t, X, X, X)),
        "k": (lambda t: lc.ar_kv4_append(handle, t, X, I, X, X)),
    }
    for name, call in calls.items():
        for t in (y, y * 2):
            with pytest.raises(ValueError, match=f"{name}: requires a gradient"):
                call(t)
        # nothing is recorded here, so nothing is lost: the next check is reached
        for t in (X, y.detach()):
            with pytest.raises(ValueError, match="not on the GPU"):
                call(t)
        with torch.no_grad(), pytest.raises(ValueError, match="not on the GPU"):
            call(y)
        with torch.inference_mode(), pytest.raises(ValueError, match="not on the GPU"):
            call(y)
