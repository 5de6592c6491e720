"""The binary64 formulas that the training kernels are held to: their
gradients against central differences, on the CPU."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import train_oracle as O  # noqa: E402


def _block(d, base=None, w1=None, w2=None, **kw):
    return O.Block(d["base"] if base is None else base, d["w1"] if w1 is None else w1,
                   d["w2"] if w2 is None else w2, d["prev"], d["tokens"], **kw)


@pytest.mark.parametrize("mult,softcap,masked", [(1.0, 0.0, 0.0), (0.7, 5.0, 0.0), (1.0, 0.0, 0.5)])
def test_gradients_against_differences(mult, softcap, masked):
    d = O.inputs(3, 4, 40, 16, seed=1, masked=masked)
    d["tokens"][1, 2] = -1                      # not scored, and clamped where it feeds
    lengths = torch.tensor([4, 4, 2], dtype=torch.int32)
    kw = dict(lengths=lengths, temperature=d["temperature"], mult=mult, softcap=softcap)
    f = {n: d[n].double() for n in ("base", "w1", "w2")}
    old = _block(d, **kw).logprobs.view(3, 4) + d["old_gap"]
    ref = _block(d, **kw).logprobs.view(3, 4) + d["ref_gap"]

    def loss(base=f["base"], w1=f["w1"], w2=f["w2"]):
        b = _block(d, base, w1, w2, **kw)
        return b, b.loss(b.logprobs, old, ref, d["advantages"], 0.2, 0.2, 0.1)

    b, (stats, grad) = loss()
    assert not b.scored.view(3, 4)[1, 2] and not b.scored.view(3, 4)[2, 2:].any()
    gradients = dict(zip(("base", "w1", "w2"), (x for x, _ in b.backward(grad))))
    g = torch.Generator().manual_seed(2)
    for name, want in gradients.items():
        way = torch.randn(f[name].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = (loss(**{name: f[name] + s * h * way})[1][0][0] for s in (1, -1))
        by_difference = float((up - down) / (2 * h))
        by_formula = float((want * way).sum())
        # the difference's own error: h^2 and the rounding of the losses / h
        assert abs(by_difference - by_formula) < 1e-7 * max(1.0, abs(by_formula)), name


def test_nearest_e4m3_is_the_format():
    """Every E4M3 value maps to itself, and each midpoint to the even code."""
    values = sorted({(-1) ** s * (2.0 ** (e - 7) * (1 + f / 8) if e else 2.0 ** -6 * f / 8)
                     for s in (0, 1) for e in range(16) for f in range(8) if (e, f) != (15, 7)})
    v = np.array(values)
    assert np.array_equal(O.e4m3_nearest(v), v)
    mid = (v[1:] + v[:-1]) / 2
    got = O.e4m3_nearest(mid)
    of = torch.tensor(mid).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, of)
