"""Training on drafted blocks at the ends of its range, on the GPU, through the
C ABI: non-finite logits and gradients, masks of large finite values, very
large and very small temperatures, large soft caps."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import train_oracle as O  # noqa: E402
from test_gpu_train import backward, dev, near, score, to  # noqa: E402,F401


def test_a_masked_token_beside_a_nan_logit(dev):
    """The row-step is NaN, and not that of an ordinary masked token."""
    for V, softcap in ((520, 0.0), (1288, 0.0), (520, 20.0)):
        d = O.inputs(4, 2, V, 64, seed=50)
        d["base"][1, 1, d["tokens"][1, 1]] = -math.inf
        d["base"][1, 1, (d["tokens"][1, 1] + 300) % V] = math.nan
        d["base"][2, 0, d["tokens"][2, 0]] = -math.inf
        lp, lse = (x.cpu() for x in score(to(d, dev), None, dev, softcap=softcap))
        assert lp[1, 1].isnan() and lse[1, 1].isnan()
        rest = torch.ones(4, 2, dtype=torch.bool)
        rest[1, 1] = False
        assert not lp[rest].isnan().any()
        if not softcap:
            assert float(lp[2, 0]) == -math.inf
