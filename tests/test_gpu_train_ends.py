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


@pytest.mark.parametrize("R,V,softcap", [(64, 1160, 0.0), (256, 520, 0.0), (512, 520, 0.0), (32, 520, 15.0)])
@pytest.mark.parametrize("bad", [-math.inf, math.inf])
def test_infinite_gradients(dev, R, V, softcap, bad):
    """What the loss gives for a token that is masked under the policy alone:
    masked entries and those without mass have gradient 0, the others an
    infinite one, and other row-steps their own."""
    d = O.inputs(6, 3, V, R, seed=51, masked=0.5)
    own, masked = (1, 1), (2, 0)                       # a token with mass, and one without
    d["base"][(*masked, d["tokens"][masked])] = -math.inf
    d["base"][1, 1, 5:9] = -300.0                      # a probability that counts as 0
    d["tokens"][1, 1] = 11
    d["base"][1, 1, 11] = 2.0
    # row-steps of their own: nothing else is fed by their tokens or hits them
    g = to(d, dev)
    lp, lse = score(g, None, dev, softcap=softcap)
    clean = backward(g, None, lse, g["grad"], dev, softcap=softcap)
    grad = g["grad"].clone()
    grad[own], grad[masked] = bad, bad
    gb, g1, g2 = (x.cpu() for x in backward(g, None, lse, grad, dev, softcap=softcap))
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], softcap=softcap)
    p = torch.exp(b.u - b.lse[:, None]).view(6, 3, V)
    for r, s in (own, masked):
        none = (p[r, s] * b.slope.view(6, 3, V)[r, s]).abs() < 2.0 ** -140
        some = (p[r, s] * b.slope.view(6, 3, V)[r, s]).abs() > 2.0 ** -110
        want = torch.full((V,), -bad)
        if (r, s) == own:
            want[11] = bad
        assert (gb[r, s][none] == 0).all() and none.any()
        assert (gb[r, s][some] == want[some]).all() and some.any()
        assert not gb[r, s].isnan().any()
    keep = torch.ones(6, 3, dtype=torch.bool)
    keep[own] = keep[masked] = False
    assert torch.equal(gb[keep], clean[0].cpu()[keep])
    # w2's rows that both leave at 0 have the gradient that they have without them
    zero = (gb[own] == 0) & (gb[masked] == 0)
    without = torch.where(keep.to(dev), g["grad"], 0.0)
    alone = backward(g, None, lse, without, dev, softcap=softcap)
    assert zero.any() and torch.equal(g2[zero], alone[2].cpu()[zero])
    # the token's own: an infinite share of its feeding token's row, with its signs
    if not softcap:
        emb = d["w1"][d["tokens"][1, 0]].float()
        only = torch.zeros(6, 3, device=dev)
        only[own] = bad
        w2 = backward(g, None, lse, only, dev, softcap=softcap)[2].cpu()
        assert torch.equal(w2[11].float()[emb != 0], (bad * emb)[emb != 0])
    fed = set(b.fed.view(6, 3)[own].reshape(-1).tolist() + b.fed.view(6, 3)[masked].reshape(-1).tolist())
    rows = torch.ones(V, dtype=torch.bool)
    rows[list(fed)] = False
    assert torch.equal(g1[rows], clean[1].cpu()[rows])


def test_a_gradient_past_bf16(dev):
    """A token's own gradient that rounds to a bf16 infinity is one, not NaN, in w2's."""
    d = O.inputs(2, 1, 520, 64, seed=52)
    d["temperature"][:] = 1.0
    d["base"][0, 0, :] = -math.inf
    t, other = 77, 78
    d["tokens"][0, 0] = t
    d["base"][0, 0, t], d["base"][0, 0, other] = -120.0, 0.0      # p of the token is 0
    d["w2"][t] = d["w2"][other] = 0
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    grad = torch.tensor([[3.4e38], [0.0]], device=dev)            # past bf16's largest, 3.39e38
    gb, g1, g2 = (x.cpu() for x in backward(g, None, lse, grad, dev))
    emb = d["w1"][d["prev"][0]].float()
    assert float(gb[0, 0, t]) == math.inf and float(gb[0, 0, other]) == -math.inf
    assert torch.equal(g2[t].float()[emb != 0], (math.inf * emb)[emb != 0])


def flat(d):
    """Row-steps whose corrections are 0: their logits are the base logits."""
    d["w1"][:] = 0
    return d


@pytest.mark.parametrize("V", [512, 520, 1288])
@pytest.mark.parametrize("R,softcap", [(32, 0.0), (512, 0.0), (64, 10.0)])
def test_infinite_temperatures_are_flat(dev, V, R, softcap):
    """Every entry that is not masked counts the same, the type's lowest and
    largest values too."""
    d = flat(O.inputs(5, 2, V, R, seed=53))
    d["temperature"][:] = math.inf
    low = torch.finfo(torch.bfloat16).min
    d["base"][1, 0, ::3], d["base"][2, 1] = low, low
    if not softcap:
        d["base"][3, 0, 1::2] = -math.inf
        d["tokens"][3, 0] = 4
    g = to(d, dev)
    lp, lse = (x.cpu().double() for x in score(g, None, dev, softcap=softcap))
    n = torch.full((5, 2), float(V), dtype=torch.float64)
    if not softcap:
        n[3, 0] = V - V // 2
    # the sum's steps, and a factor that is not quite 0: 2^-149 of 3.4e38 is 2^-21
    off = (V / 64 + 40) * O.ADD + 2.0 ** -20
    near(lse, n.log(), off, "lse")
    near(lp, -n.log(), 2 * off, "logprobs")
    out = backward(g, None, lse.float().to(dev), g["grad"], dev, softcap=softcap)
    assert not any(x.any() for x in out)


@pytest.mark.parametrize("V", [512, 520])
@pytest.mark.parametrize("mult", [0.0, 1e-30])
def test_a_multiplier_that_flattens(dev, V, mult):
    """z = mult x with a factor of 0, or one that the temperature takes past the
    smallest number: flat, but for masks."""
    d = O.inputs(4, 2, V, 32, seed=54)
    d["temperature"][1:] = 1e25
    d["base"][1, 1, ::2] = -math.inf
    d["tokens"][1, 1] = 3
    g = to(d, dev)
    lp, lse = (x.cpu().double() for x in score(g, None, dev, mult=mult))
    n = torch.full((4, 2), float(V), dtype=torch.float64)
    n[1, 1] = V // 2
    off = (V / 64 + 40) * O.ADD + 2.0 ** -20
    near(lse, n.log(), off, "lse")
    near(lp, -n.log(), 2 * off, "logprobs")
    gb, g1, g2 = backward(g, None, lse.float().to(dev), g["grad"], dev, mult=mult)
    # the slope is the multiplier: below 1e-29 in every gradient
    assert all(x.isfinite().all() and x.float().abs().max() < 1e-28 for x in (gb, g1, g2))


LOW = torch.finfo(torch.bfloat16).min


@pytest.mark.parametrize("V,R", [(520, 64), (1288, 256), (392, 512)])
@pytest.mark.parametrize("value", [-1e4, -1e9, -1e10, -1e30, LOW])
def test_rows_of_nothing_but_finite_masks(dev, V, R, value):
    """Every entry the same large negative value, over a whole row-step or beside
    -inf: the entries are equally likely, and where binary32 cannot hold the
    logarithm of their number beside the value they have no gradient."""
    d = flat(O.inputs(6, 2, V, R, seed=55))
    d["temperature"] = torch.tensor([1.0, 0.5, 3.0, 0.0, 1.5, 1.0])
    n = torch.full((6, 2), float(V), dtype=torch.float64)
    for r in range(5):
        d["base"][r, 1] = value
    d["base"][4, 1, 1::2], n[4, 1], d["tokens"][4, 1] = -math.inf, V - V // 2, 6
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    c = float(torch.tensor(value).bfloat16())
    heat = torch.where(d["temperature"] == 0, 1.0, d["temperature"]).double()
    want = (c / heat[:5] + n[:5, 1].log()).float().double()
    near(lse[:5, 1], want, 2.0 ** -22 * want.abs().clamp(max=3e38), "lse")
    # exact differences of equal logits: the sum's own steps remain
    near(lp[:5, 1], -n[:5, 1].log(), 2 * (V / 64 + 40) * O.ADD, "logprobs")
    out = backward(g, None, lse, g["grad"], dev)
    assert all(x.isfinite().all() for x in out)
    gb = out[0].cpu().double()
    if value < -2.0 ** 24 * 3:
        assert not gb[:5, 1].any()
    else:
        p = torch.where(d["base"][:5, 1] == -math.inf, 0.0, 1.0).double() / n[:5, 1, None]
        hit = torch.zeros(5, V, dtype=torch.float64).scatter_(1, d["tokens"][:5, 1:], 1.0)
        scale = (d["grad"][:5, 1].double() / heat[:5])[:, None]
        # lse to half a step of its size, z / T likewise, and the steps of exp
        off = scale.abs() * p * 1.1 * (want.abs()[:, None] * 3 * 2.0 ** -24 + 16 * O.ADD) + 16 * O.ADD * scale.abs() * hit
        near(gb[:5, 1], scale * (hit - p), off + O.BF16 * (scale * (hit - p)).abs(), "grad_base")
    # the ordinary row-steps are what they are without these
    keep = torch.zeros(6, 2)
    keep[:, 0] = keep[5] = 1
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"])
    want, off = b.backward(d["grad"] * keep)[0]
    near(gb[keep.bool()], want[keep.bool()], off[keep.bool()], "grad_base of the others")


@pytest.mark.parametrize("V,R,softcap", [(520, 64, 0.0), (1288, 256, 0.0), (392, 512, 0.0), (520, 16, 0.0),
                                         (520, 64, 30.0), (1288, 256, 5.0), (264, 128, 500.0)])
@pytest.mark.parametrize("T", [1e-3, 1e-5, 1e-8, 1e-20, 1e-36])
def test_small_temperatures(dev, V, R, softcap, T):
    """Temperatures that leave one token: it has log-probability 0 and no
    gradient, another one the distance to it and its own gradient alone."""
    d = O.inputs(40, 2, V, R, seed=56, spread=0.5, weights=0.1)
    d["temperature"] = torch.where(torch.arange(40) % 4 == 3, 1.0, T)
    cold = torch.arange(40) % 4 != 3
    # the largest by 2 or more: of the token itself at step 0, of another at step 1
    top = d["tokens"].clone()
    top[:, 1] = (top[:, 1] + 100) % V
    d["base"].clamp_(max=1.0)
    d["base"].scatter_(2, top[:, :, None], 5.0)
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], softcap=softcap)
    z = b.z.view(40, 2, V)
    assert ((z.topk(2, 2)[0] @ torch.tensor([1.0, -1.0]).double())[cold] > 0.1).all()
    g = to(d, dev)
    lp, lse = score(g, None, dev, softcap=softcap)
    first = z.amax(2)
    # z in binary32 (as the oracle counts it), relative
    z_off = (b.x_off.amax(1).view(40, 2) + 8 * O.ADD * (first.abs() + softcap)) + 4 * O.ADD * first.abs()
    heat = d["temperature"].double()[:, None]
    near(lse[cold], (first / heat)[cold].float().double(), (z_off / heat)[cold], "lse")
    own = z.gather(2, d["tokens"][:, :, None])[:, :, 0]
    assert not lp[cold][:, 0].any()
    want = ((own - first) / heat)[cold][:, 1]
    near(lp[cold][:, 1], want.float().double(), (2 * z_off / heat)[cold][:, 1], "logprobs")
    grad = g["grad"] * T                                # (gradients of g / T, so that they fit bf16)
    gb, g1, g2 = backward(g, None, lse, grad, dev, softcap=softcap)
    assert all(x.isfinite().all() for x in (gb, g1, g2))
    gb = gb.cpu().double()
    assert not gb[cold][:, 0].any()
    want = torch.zeros(40, V, dtype=torch.float64)
    slope = b.slope.view(40, 2, V)[:, 1]
    s = ((d["grad"].float() * T).double()[:, 1] / heat[:, 0])[:, None]
    want.scatter_(1, d["tokens"][:, 1:], s * slope.gather(1, d["tokens"][:, 1:]))
    want.scatter_(1, top[:, 1:], -s * slope.gather(1, top[:, 1:]))
    # the slope to its steps and x's, as the oracle counts them
    off = 16 * O.ADD * want.abs() + O.BF16 * want.abs()
    if softcap:
        off = off + s.abs() * (want != 0) * 2 / softcap * b.x_off.view(40, 2, V)[:, 1]
    near(gb[:, 1][cold], want[cold], 1.01 * off[cold], "grad_base")


@pytest.mark.parametrize("V,R", [(520, 64), (1288, 256)])
def test_negative_factors(dev, V, R):
    """Negated logits at a negative temperature, or under a negative multiplier,
    are the same distribution."""
    d = O.inputs(12, 2, V, R, seed=58)
    d["temperature"][::3] = 1e-5
    d["base"][4, 1] = -1e9
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    gb = backward(g, None, lse, g["grad"] * 1e-5, dev)[0]
    for n in ("base", "w1"):
        d[n] = -d[n]
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], mult=-1.0)
    _, off = b.backward(d["grad"] * 1e-5)[0]
    for mult, turn in ((-1.0, 1.0), (1.0, -1.0)):
        o = to(d, dev)
        o["temperature"] *= turn
        lp2, lse2 = score(o, None, dev, mult=mult)
        near(lp2, lp.cpu().double(), 4 * b.off.view(12, 2), "logprobs")
        near(lse2, lse.cpu().double(), 2 * b.off.view(12, 2), "lse")
        assert torch.equal(lp2[::3], lp[::3]) and torch.equal(lse2[::3], lse[::3]) and torch.equal(lp2[4, 1], lp[4, 1])
        gb2 = backward(o, None, lse2, g["grad"] * 1e-5, dev, mult=mult)[0]
        keep = torch.ones(12, 2, dtype=torch.bool)
        keep[::3] = keep[4, 1] = False
        near(-gb2[keep], gb.cpu().double()[keep], 2 * off[keep], "grad_base")
        assert torch.equal(-gb2[::3], gb[::3]) and not gb2[4, 1].any()


@pytest.mark.parametrize("mult,softcap", [(1.0, 100.0), (1.0, 1e3), (0.5, 1e5), (1.0, 1e7), (20.0, 80.0)])
def test_large_soft_caps(dev, mult, softcap):
    """A cap far above the logits leaves them as they are, not to a few steps of
    the cap but to a few of their own."""
    d = O.inputs(6, 3, 1096, 64, seed=57)
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], mult=mult, softcap=softcap)
    b.off = b.off - 8 * O.ADD * softcap / b.heat.abs()[:, 0]
    g = to(d, dev)
    lp, lse = score(g, None, dev, mult=mult, softcap=softcap)
    near(lse, b.lse, b.off, "lse")
    near(lp, b.logprobs, 2 * b.off, "logprobs")
    (want, off), (w1, w1_off), (w2, w2_off) = b.backward(d["grad"])
    out = backward(g, None, lse, g["grad"], dev, mult=mult, softcap=softcap)
    near(out[0], want, off, "grad_base")
    near(out[2], w2, w2_off, "grad_w2")
    near(out[1], w1, w1_off, "grad_w1")


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("T", [1e-5, 1e-8, 1e-12])
def test_small_temperatures_of_negative_logits(dev, T, softcap):
    """Logits that are all negative (log-probabilities, say) have the gradients that
    positive ones have."""
    d = flat(O.inputs(8, 2, 520, 64, seed=59, spread=0.5))
    d["temperature"][:] = T
    d["base"] = d["base"].clamp(max=1.0) - 16.0
    other = (d["tokens"] + 100) % 520
    d["base"].scatter_(2, d["tokens"][:, :, None], -13.0)
    d["base"].scatter_(2, other[:, :, None], -12.0)
    g = to(d, dev)
    lp, lse = score(g, None, dev, softcap=softcap)
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], softcap=softcap)
    z, slope = b.z.view(8, 2, 520), b.slope.view(8, 2, 520)
    heat = d["temperature"].double()[:, None]
    top, own = z.amax(2), z.gather(2, d["tokens"][:, :, None])[:, :, 0]
    z_off = 12 * O.ADD * (top.abs() + softcap)
    near(lse, (top / heat).float().double(), z_off / heat, "lse")
    near(lp, ((own - top) / heat).float().double(), 2 * z_off / heat, "logprobs")
    gb = backward(g, None, lse, g["grad"] * T, dev, softcap=softcap)[0]
    s = ((d["grad"] * T).double() / heat)[:, :, None]
    want = torch.zeros(8, 2, 520, dtype=torch.float64)
    want.scatter_(2, d["tokens"][:, :, None], s * slope.gather(2, d["tokens"][:, :, None]))
    want.scatter_(2, other[:, :, None], -s * slope.gather(2, other[:, :, None]))
    near(gb, want, 1.01 * (16 * O.ADD + O.BF16) * want.abs(), "grad_base")


@pytest.mark.parametrize("rows,R", [(1, 16), (1, 256), (33, 64), (40, 512), (95, 128)])
def test_an_infinite_gradient_of_the_last_row_step(dev, rows, R):
    """What pads the row-steps adds nothing to it."""
    d = O.inputs(rows, 1, 520, R, seed=60)
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    grad = torch.zeros(rows, 1, device=dev)
    grad[-1] = math.inf
    gb, g1, g2 = (x.cpu().float() for x in backward(g, None, lse, grad, dev))
    emb = d["w1"][d["prev"][-1]].float()
    want = gb[-1, 0][:, None] * torch.where(emb == 0, 1.0, emb)
    mass = gb[-1, 0].isinf()
    assert mass.all() and torch.equal(g2[:, emb != 0], want[:, emb != 0])


@pytest.mark.parametrize("T,mult,softcap", [(1e-40, 1.0, 0.0), (1e-45, 1.0, 0.0), (1e-40, 1.0, 30.0), (-1e-40, -1.0, 0.0),
                                            (1e-20, 1e30, 0.0), (1e-38, -1e10, 0.0)])
def test_factors_past_binary32(dev, T, mult, softcap):
    """Temperatures whose inverse, or its product with the multiplier, is past
    binary32: the largest logit's token is certain, and nothing is NaN."""
    d = O.inputs(6, 2, 520, 64, seed=61, spread=0.5, weights=0.1)
    d["temperature"][::2] = T
    d["base"].clamp_(max=1.0)
    up = 1.0 if T * mult > 0 else -1.0                    # (a negative factor turns the order)
    d["base"].scatter_(2, d["tokens"][:, :, None], 5.0)
    d["base"] *= up
    d["w1"] *= up
    g = to(d, dev)
    lp, lse = score(g, None, dev, mult=mult, softcap=softcap)
    assert not lp[::2].any() and not lp.isnan().any() and not lse.isnan().any()
    gb, g1, g2 = backward(g, None, lse, g["grad"], dev, mult=mult, softcap=softcap)
    assert not gb[::2].any() and not any(x.isnan().any() for x in (gb, g1, g2))
    # and another token has none of it
    g["tokens"] = (g["tokens"] + 1) % 520
    lp, lse = score(g, None, dev, mult=mult, softcap=softcap)
    assert (lp[::2, 0] < -1e36).all() and not lp.isnan().any() and not lse.isnan().any()


@pytest.mark.parametrize("R", [32, 128, 256, 512])
def test_large_logits_are_rounded_once(dev, R):
    """Logits near 100 and corrections far below: base and product meet in one
    rounding, and 1 / T scales distances alone."""
    rows, k, V = 60, 4, 264
    d = O.inputs(rows, k, V, R, seed=62, weights=0.005)
    d["base"][:] = -math.inf
    t = d["tokens"]
    for i, value in enumerate((100.0, 100.5, 101.0)):
        d["base"].scatter_(2, ((t + 50 * i) % V)[:, :, None], value)
    d["temperature"][:20] = 1.0
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"])
    lp, lse = score(to(d, dev), None, dev)
    # half a step of a logit in [64, 128), the product's own sums, and of the softmax
    # (distances of at most 1.1, in powers of 2 and over T) three half steps of a
    # distance, two steps of an exponential and eight of sums and joins
    mass = (b.emb.abs() @ b.w2.abs().T).amax(1)
    heat = b.heat[:, 0]
    off = (2.0 ** -18 + (R + 2) * O.ADD * mass) / heat + 3 * 2.0 ** -24 * 1.6 / heat + 10 * O.ADD
    near(lp, b.logprobs, off + 2.0 ** -23 * b.logprobs.abs(), "logprobs")
    near(lse, b.lse, off + 2.0 ** -23 * b.lse.abs(), "lse")
