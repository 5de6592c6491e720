"""Training on drafted blocks on the GPU, through the C ABI: scoring, the
policy loss and the gradients against the binary64 formulas, and the whole
chain with the drafting loop and the verifier."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import markov_draft_sampling_step_amd as m  # noqa: E402
import train_oracle as O  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m.lib()
    return torch.device("cuda:0")


def to(d, dev):
    return {n: x.to(dev) for n, x in d.items()}


def score(d, lengths, dev, heat=True, space=None, stream=None, **kw):
    rows, k, V = d["base"].shape
    lp, lse = (torch.full((rows, k), 5.0, device=dev) for _ in range(2))
    space = m.new_score_workspace(rows, V, d["w1"].shape[1], k) if space is None else space
    m.score_sequential(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], lengths,
                       d["temperature"] if heat else None, lp, lse, space, stream=stream, **kw)
    return lp, lse


def backward(d, lengths, lse, grad, dev, heat=True, in_place=False, space=None, stream=None, **kw):
    rows, k, V = d["base"].shape
    R = d["w1"].shape[1]
    gb = d["base"].clone() if in_place else torch.full_like(d["base"], 5.0)
    g1, g2 = torch.full_like(d["w1"], 5.0), torch.full_like(d["w2"], 5.0)
    space = m.new_score_workspace(rows, V, R, k) if space is None else space
    m.score_backward(gb if in_place else d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], lengths,
                     d["temperature"] if heat else None, lse, grad, gb, g1, g2, space, stream=stream, **kw)
    return gb, g1, g2


def near(got, want, off, what):
    got = got.cpu().double().reshape(want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= off))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4], got[bad][:4], want[bad][:4])


def check(d, dev, lengths=None, heat=True, grad=None, **kw):
    """Scoring and its gradients against the formulas."""
    rows, k, V = d["base"].shape
    b = O.Block(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], lengths,
                d["temperature"] if heat else None, **kw)
    g = to(d, dev)
    ln = None if lengths is None else lengths.to(dev)
    lp, lse = score(g, ln, dev, heat, **kw)
    near(lse, b.lse, b.off, "lse")
    near(lp, b.logprobs, 2 * b.off, "logprobs")
    grad = g["grad"] if grad is None else grad.to(dev)
    (want, off), (w1, w1_off), (w2, w2_off) = b.backward(grad)
    out = backward(g, ln, lse, grad, dev, heat, **kw)
    near(out[0], want, off, "grad_base")
    near(out[2], w2, w2_off, "grad_w2")
    near(out[1], w1, w1_off, "grad_w1")
    again = backward(g, ln, lse, grad, dev, heat, in_place=True, **kw)
    assert all(torch.equal(x, y) or x.isnan().any() for x, y in zip(out, again))
    return b, (lp, lse), out


@pytest.mark.parametrize("rows,k,V,R", [
    (1, 1, 8, 16), (1, 1, 8, 512), (2, 3, 4096, 32), (1, 5, 1000, 256), (3, 1, 520, 64), (16, 5, 1288, 256),
    (5, 4, 72, 128), (17, 1, 1032, 16), (13, 5, 2056, 512), (9, 8, 264, 256), (33, 4, 776, 32), (64, 5, 640, 256),
    (43, 3, 4104, 128), (150, 2, 264, 64)])
def test_shapes(dev, rows, k, V, R):
    check(O.inputs(rows, k, V, R, seed=rows + V), dev)


@pytest.mark.parametrize("rows,k,V,R,softcap", [
    (128, 4, 12808, 256, 0.0), (103, 5, 18504, 256, 0.0), (130, 4, 20008, 64, 20.0), (103, 5, 9000, 16, 0.0),
    (64, 8, 8200, 512, 9.0), (131, 4, 9992, 128, 0.0), (171, 3, 9992, 32, 5.0), (4, 2, 60008, 128, 0.0)])
def test_many_tiles_and_tokens(dev, rows, k, V, R, softcap):
    """Several tiles and units for each workgroup, and more than 512 row-steps."""
    check(O.inputs(rows, k, V, R, seed=rows + R), dev, softcap=softcap)


def test_offsets_past_32_bits(dev):
    """The largest vocabulary, base logits and gradients of 17 GB: the block of
    128 row-steps whose last begins 4.26e9 bytes after its first, and the last."""
    rows, k, V, R = 513, 1, 1 << 24, 16
    free = torch.cuda.mem_get_info()[0]
    if free < 60 << 30:
        pytest.skip("not enough memory")
    torch.manual_seed(21)
    base = torch.empty(rows, k, V, dtype=torch.bfloat16, device=dev).normal_()
    w1, w2 = (torch.empty(V, R, device=dev).normal_().mul_(0.3).bfloat16() for _ in range(2))
    prev = torch.randint(0, V, (rows,), device=dev)
    tokens = torch.randint(0, V, (rows, k), device=dev)
    at = [0, 127, 128, 512]
    tokens[at[1]], tokens[at[3]], prev[at[3]] = V - 1, V - 2, V - 1
    base.scatter_(2, tokens[:, :, None], 5.0)
    lp, lse = (torch.empty(rows, k, device=dev) for _ in range(2))
    space = m.new_score_workspace(rows, V, R, k)
    m.score_sequential(base, w1, w2, prev, tokens, None, None, lp, lse, space)
    # the probabilities of 2^24 entries are near 2^-24: gradients that show
    grad = torch.empty(rows, k, device=dev).normal_() * 2.0 ** 20
    gb, g1, g2 = torch.full_like(base, 5.0), torch.full_like(w1, 5.0), torch.full_like(w2, 5.0)
    m.score_backward(base, w1, w2, prev, tokens, None, None, lse, grad, gb, g1, g2, space)
    for i in at:
        # (the formulas in binary64, with the tolerances of the oracle's Block)
        terms = w2.double() * w1[prev[i]].double()
        x = base[i, 0].double() + terms.sum(1)
        x_off = (R + 2) * O.ADD * (terms.abs().sum(1) + x.abs())
        want = torch.logsumexp(x, 0)
        off = float(x_off.max() + 8 * O.ADD * x.abs().max()) + (V / 64 + 40) * O.ADD
        assert abs(float(lse[i]) - float(want)) <= off, i
        assert abs(float(lp[i]) - float(x[tokens[i, 0]] - want)) <= 2 * off, i
        # (dL/dx = g (hit - p), with the kernel's own lse for p)
        p = torch.exp(x - lse[i, 0].double())
        d = -grad[i, 0].double() * p
        d[tokens[i, 0]] += grad[i, 0].double()
        scale = float(grad[i].abs())
        d_off = 1.01 * scale * (p * 2.2 * (x_off + 8 * O.ADD * x.abs().max()) + 16 * O.ADD * p + 2.0 ** -126)
        d_off[tokens[i, 0]] += 16 * O.ADD * scale * 1.01
        bad = (gb[i, 0].double() - d).abs() > d_off + O.BF16 * d.abs()
        assert not bad.any(), (i, bad.nonzero()[:4])
    # gradients of w2 at both ends and around, from the stored d (whose
    # rounding the kernel's sums share but for a row-step's own entry)
    emb = w1[prev].double()
    for v0 in (0, 12345678 // 128 * 128, V - 128):
        d = gb[:, 0, v0:v0 + 128].double()
        own = ((tokens >= v0) & (tokens < v0 + 128)).any(1)
        off = O.BF16 * (d[own].abs().T @ emb[own].abs())
        want = d.T @ emb
        off = off + O.BF16 * want.abs() + 515 * O.ADD * (d.abs().T @ emb.abs()) + 2.0 ** -133
        assert ((g2[v0:v0 + 128].double() - want).abs() <= 1.01 * off).all(), v0
    # and of w1: rows that fed a row-step, and none other
    fed = torch.zeros(V, dtype=torch.bool, device=dev)
    fed[prev] = True
    assert torch.equal(g1.any(1), fed)
    i = at[3]
    alone = (prev == prev[i]).sum() == 1
    d, own = gb[i, 0].double(), float(gb[i, 0, tokens[i, 0]].double().abs())
    terms = d[:, None] * w2.double()
    want = terms.sum(0)
    off = O.BF16 * own * w2[tokens[i, 0]].double().abs() + (V + 2) * O.ADD * terms.abs().sum(0) + O.BF16 * want.abs()
    assert alone and ((g1[prev[i]].double() - want).abs() <= 1.01 * off).all()


@pytest.mark.parametrize("mult,softcap", [(1.0, 30.0), (0.5, 4.0), (-1.5, 0.0), (2.0, 0.5)])
def test_transforms(dev, mult, softcap):
    check(O.inputs(6, 3, 1096, 64, seed=5), dev, mult=mult, softcap=softcap)


def test_lengths_tokens_and_feeds_out_of_range(dev):
    """Row-steps past the length or with no token in range give zeros, their
    logits (NaN here) are never read, and feeding tokens are clamped."""
    d = O.inputs(9, 4, 1048, 64, seed=6)
    lengths = torch.tensor([4, 0, 2, 9, -3, 4, 1, 4, 3], dtype=torch.int32)
    d["tokens"][5] = torch.tensor([3, -1, 1048, 2 ** 40])
    d["tokens"][7, 1] = -2 ** 63
    d["prev"][:3] = torch.tensor([-1, 1048, 2 ** 62])
    for r in range(9):
        d["base"][r, max(0, int(lengths[r])):] = float("nan")
    d["base"][5, 1:] = float("nan")
    d["base"][7, 1] = float("nan")
    b, (lp, lse), out = check(d, dev, lengths)
    off = ~b.scored.view(9, 4)
    assert off.sum() >= 18 and not lp.cpu()[off].any() and not lse.cpu()[off].any()
    assert not out[0].cpu()[off].any()
    _, (lp, lse), out = check(d, dev, torch.zeros(9, dtype=torch.int32))
    assert not lp.any() and not out[0].any() and not out[1].any() and not out[2].any()


def test_temperatures(dev):
    d = O.inputs(6, 2, 520, 32, seed=7)
    d["temperature"][:4] = torch.tensor([0.0, -0.0, 0.05, 50.0])
    check(d, dev)
    check(d, dev, heat=False)
    # an infinite temperature, where a slab ends past the vocabulary
    d["temperature"][2] = math.inf
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    assert (lse[2].cpu() - math.log(520)).abs().max() < 1e-5 and torch.equal(lp[2], -lse[2])
    out = backward(g, None, lse, g["grad"], dev)
    assert not out[0][2].any() and all(x.isfinite().all() for x in out)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_masked_logits(dev, softcap):
    """-inf over most of a row, over all of it, and on the token itself; the
    type's lowest value as a mask."""
    d = O.inputs(8, 3, 1160, 64, seed=8, masked=0.9)
    d["base"][1, 1] = -math.inf
    d["base"][2, 0, d["tokens"][2, 0]] = -math.inf
    d["base"][3, 2] = torch.finfo(torch.bfloat16).min
    d["base"][3, 2, d["tokens"][3, 2]] = 1.0
    d["base"][4, 1, :] = -math.inf
    d["base"][4, 1, d["tokens"][4, 1]] = -2.0
    _, (lp, lse), out = check(d, dev, softcap=softcap)
    if not softcap:
        assert float(lp[1, 1]) == float(lse[1, 1]) == -math.inf and not out[0][1, 1].any()
        assert float(lp[2, 0]) == -math.inf and math.isfinite(float(lse[2, 0]))
        assert abs(float(lp[4, 1])) < 1e-5


def test_nan_and_inf_logits(dev):
    """A NaN or +inf logit makes its row-step NaN, and others not."""
    d = O.inputs(5, 3, 520, 32, seed=9)
    clean = to(d, dev)
    lp0, lse0 = score(clean, None, dev)
    d["base"][1, 1, 77], d["base"][3, 0, 500] = float("nan"), math.inf
    g = to(d, dev)
    lp, lse = score(g, None, dev)
    hit = torch.zeros(5, 3, dtype=torch.bool)
    hit[1, 1] = hit[3, 0] = True
    assert lp.cpu()[hit].isnan().all() and lse.cpu()[1, 1].isnan()
    assert torch.equal(lp.cpu()[~hit], lp0.cpu()[~hit])
    # a gradient of 0 for those row-steps keeps them out of every gradient
    grad = torch.where(hit.to(dev), 0.0, g["grad"])
    out = backward(g, None, lse, grad, dev)
    assert not any(x.isnan().any() for x in out) and not out[0].cpu()[hit].any()
    # and one that is not makes its own logits' gradient NaN
    out = backward(g, None, lse, g["grad"], dev)
    assert out[0].cpu()[hit].isnan().all() and not out[0].cpu()[~hit].isnan().any()


def test_zero_gradients_are_zero(dev):
    d = O.inputs(4, 3, 520, 256, seed=10)
    _, _, out = check(d, dev, grad=torch.zeros(4, 3))
    assert not any(x.any() for x in out)


def test_shared_feeds(dev):
    """Row-steps fed by one token: a few, and all of them."""
    d = O.inputs(40, 5, 1032, 128, seed=11)
    d["prev"][:] = 7
    d["tokens"][::2] = 7
    check(d, dev)
    d["tokens"][:] = 7
    _, _, out = check(d, dev)
    rows = out[1].any(1).nonzero().reshape(-1).tolist()
    assert rows == [7]


def test_confident_and_flat_rows(dev):
    """One token with nearly all of the mass, and a flat row."""
    d = O.inputs(4, 2, 4104, 64, seed=12, weights=0.01)
    d["base"][0] = 0.0
    d["base"][1, 0, d["tokens"][1, 0]] = 90.0
    d["base"][2, 0, d["tokens"][2, 0]] = -90.0
    check(d, dev)


def test_rows_do_not_depend_on_the_batch(dev):
    d = to(O.inputs(70, 3, 1288, 256, seed=13), dev)
    lp, lse = score(d, None, dev)
    gb = backward(d, None, lse, d["grad"], dev)[0]
    for n in (1, 5, 22, 43):
        part = {i: (x if i in ("w1", "w2") else x[:n].contiguous()) for i, x in d.items()}
        a, b = score(part, None, dev)
        assert torch.equal(a, lp[:n]) and torch.equal(b, lse[:n]), n
        assert torch.equal(backward(part, None, b, part["grad"], dev)[0], gb[:n]), n


def test_gradient_against_differences(dev):
    """The kernel's gradients against central differences of the loss in
    binary64, along random directions."""
    d = O.inputs(6, 4, 520, 64, seed=14)
    lengths = torch.tensor([4, 4, 3, 0, 2, 4], dtype=torch.int32)
    kw = dict(mult=0.9, softcap=12.0)
    b, (lp, lse), _ = check(d, dev, lengths, **kw)
    g = to(d, dev)
    old, ref = lp + g["old_gap"], lp + g["ref_gap"]
    stats, grad = torch.zeros(4, device=dev), torch.zeros(6, 4, device=dev)
    ln = lengths.to(dev)
    m.policy_loss(lp, old, ref, g["advantages"], g["tokens"], ln, 520, stats, grad, beta=0.1)
    out = dict(zip(("base", "w1", "w2"), backward(g, ln, lse, grad, dev, **kw)))
    offs = dict(zip(("base", "w1", "w2"), (x[1] for x in b.backward(grad))))
    gen = torch.Generator().manual_seed(15)
    for name in out:
        way = torch.randn(out[name].shape, generator=gen, dtype=torch.float64)

        def loss(step):
            f = {n: d[n].double() + (step * way if n == name else 0) for n in ("base", "w1", "w2")}
            bb = O.Block(f["base"], f["w1"], f["w2"], d["prev"], d["tokens"], lengths, d["temperature"], **kw)
            return float(bb.loss(bb.logprobs, old, ref, d["advantages"], 0.2, 0.2, 0.1)[0][0])

        h = 1e-5
        by_difference = (loss(h) - loss(-h)) / (2 * h)
        by_kernel = float((out[name].cpu().double() * way).sum())
        # the kernel's own tolerance along the direction, that of the loss's
        # gradient (binary32 of the log-probabilities), and the difference's
        off = float((offs[name] * way.abs()).sum()) + 1e-5 * float((out[name].cpu().double() * way).abs().sum()) + 1e-7
        assert abs(by_difference - by_kernel) <= off, (name, by_difference, by_kernel, off)


# -- the loss -----------------------------------------------------------------------

def loss_inputs(rows, k, V, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda: torch.randn(rows, k, generator=g)  # noqa: E731
    lp = -n().abs() * 4
    return dict(lp=lp, old=lp + 0.3 * n(), ref=lp + 0.3 * n(), adv=n(),
                tokens=torch.randint(0, V, (rows, k), generator=g))


def check_loss(d, V, dev, lengths=None, low=0.2, high=0.28, beta=0.05, ref=True):
    rows, k = d["lp"].shape
    b = O.Block.__new__(O.Block)
    ln = torch.full((rows,), k) if lengths is None else lengths.long()
    b.rows, b.k = rows, k
    b.scored = ((torch.arange(k)[None] < ln[:, None]) & (d["tokens"] >= 0) & (d["tokens"] < V)).reshape(-1)
    # the bounds and beta are binary32 arguments: at 0.05 the nearest is 2^-25
    # off, which a gradient whose two terms cancel shows
    low, high, beta = (float(torch.tensor(x, dtype=torch.float32)) for x in (low, high, beta))
    want, grad = b.loss(d["lp"], d["old"], d["ref"] if ref else None, d["adv"], low, high, beta)
    g = to(d, dev)
    stats, out = torch.full((4,), 9.0, device=dev), torch.full((rows, k), 9.0, device=dev)
    m.policy_loss(g["lp"], g["old"], g["ref"] if ref else None, g["adv"], g["tokens"],
                  None if lengths is None else lengths.to(dev), V, stats, out, clip_low=low, clip_high=high,
                  beta=beta)
    # binary64 inside, one rounding to binary32 of each result
    near(stats, want, 2.0 ** -22 * (want.abs() + (1 if len(d["lp"]) else 0) * float(d["adv"].abs().max())), "stats")
    near(out, grad, 2.0 ** -23 * grad.abs() + 2.0 ** -149, "grad_logprobs")
    return stats, out


@pytest.mark.parametrize("rows,k", [(1, 1), (2, 3), (64, 5), (256, 8), (341, 3), (65536, 1)])
def test_policy_loss(dev, rows, k):
    d = loss_inputs(rows, k, 1000, rows)
    for kw in (dict(), dict(beta=0.0, ref=False), dict(beta=0.0), dict(low=0.0, high=0.0), dict(low=1.0, high=1e9)):
        check_loss(d, 1000, dev, **kw)


def test_policy_loss_masks(dev):
    d = loss_inputs(6, 4, 1000, 3)
    d["tokens"][2] = torch.tensor([-1, 1000, 2 ** 40, 5])
    lengths = torch.tensor([4, 0, 4, -1, 2, 7], dtype=torch.int32)
    for name in ("lp", "old", "ref", "adv"):
        d[name][1], d[name][2, :3], d[name][3], d[name][4, 2:] = (float("nan"),) * 4
    check = {n: torch.where(d[n].isnan(), 0.0, d[n]) for n in ("lp", "old", "ref", "adv")}
    stats, out = check_loss({**d, **check}, 1000, dev, lengths)
    g = to(d, dev)
    s2, o2 = torch.zeros(4, device=dev), torch.zeros(6, 4, device=dev)
    m.policy_loss(g["lp"], g["old"], g["ref"], g["adv"], g["tokens"], lengths.to(dev), 1000, s2, o2,
                  clip_low=0.2, clip_high=0.28, beta=0.05)
    assert torch.equal(s2, stats) and torch.equal(o2, out)
    stats, out = check_loss({**d, **check}, 1000, dev, torch.zeros(6, dtype=torch.int32))
    assert not stats.any() and not out.any()


def test_policy_loss_extremes(dev):
    """A token of probability 0 under the policy, a ratio past every bound, an
    advantage of 0, an unchanged policy."""
    d = loss_inputs(1, 5, 1000, 4)
    d["lp"][0] = torch.tensor([-math.inf, -1.0, -200.0, -1.0, -2.0])
    d["old"][0] = torch.tensor([-1.0, -200.0, -1.0, -2000.0, -2.0])
    d["adv"][0] = torch.tensor([1.0, 2.0, -3.0, 0.0, 1.5])
    g = to(d, dev)
    stats, out = torch.zeros(4, device=dev), torch.zeros(1, 5, device=dev)
    m.policy_loss(g["lp"], g["old"], None, g["adv"], g["tokens"], None, 1000, stats, out)
    # ratios 0, e^199 (held at 1.2), e^-199 (A < 0: held at 0.8), past
    # binary64 with A = 0, and 1
    want = torch.tensor([0.0, 0.0, 0.0, 0.0, -1.5 / 5])
    near(out, want.double()[None], 2.0 ** -23 * want.abs()[None], "grad")
    surrogate = (0.0 + 1.2 * 2.0 - 0.8 * 3.0 + 0.0 + 1.5) / 5
    near(stats, torch.tensor([-surrogate, surrogate, 0.0, 0.4]).double(), 1e-6, "stats")


def test_policy_loss_of_masked_tokens(dev):
    """Log-probabilities of -inf: under the policy alone, under the reference
    alone, and under all three."""
    inf = math.inf
    one = lambda *x: torch.tensor([x], device=dev)  # noqa: E731
    tokens = torch.zeros(1, 3, dtype=torch.int64, device=dev)
    stats, out = torch.zeros(4, device=dev), torch.zeros(1, 3, device=dev)

    def loss(lp, old, ref):
        m.policy_loss(one(*lp), one(*old), one(*ref), one(1.0, -1.0, 2.0), tokens, None, 16, stats, out, beta=0.5)
        return stats.tolist(), out.reshape(-1).tolist()

    s, g = loss((-inf, -1.0, -1.0), (-inf, -1.0, -1.0), (-inf, -1.0, -1.0))
    assert s[1:] == [torch.tensor(2 / 3).item(), 0.0, 0.0] and s[0] == -s[1]
    assert g == torch.tensor([-1 / 3, 1 / 3, -2 / 3]).tolist()
    # e^gap - gap - 1 goes to infinity on both sides, its slope on one
    s, g = loss((-inf, -1.0, -1.0), (-1.0, -1.0, -1.0), (-1.0, -1.0, -1.0))
    assert s[0] == s[2] == inf and g[0] == -inf and g[1:] == torch.tensor([1 / 3, -2 / 3]).tolist()
    s, g = loss((-1.0, -1.0, -1.0), (-1.0, -1.0, -1.0), (-inf, -1.0, -1.0))
    assert s[0] == s[2] == inf and g == torch.tensor([-0.5 / 3, 1 / 3, -2 / 3]).tolist()


# -- used together ------------------------------------------------------------------

def test_streams_and_shared_workspace(dev):
    """A side stream, and a workspace used by one call after another."""
    big = to(O.inputs(60, 5, 1288, 128, seed=16), dev)
    space = m.new_score_workspace(60, 1288, 128, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = score(big, None, dev, space=space, stream=side)
    side.synchronize()
    b = score(big, None, dev)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    small = {i: (x if i in ("w1", "w2") else x[:3].contiguous()) for i, x in big.items()}
    lp, lse = score(small, None, dev, space=space)
    out = backward(small, None, lse, small["grad"], dev, space=space)
    ref = backward(small, None, lse, small["grad"], dev)
    assert torch.equal(lp, b[0][:3]) and all(torch.equal(x, y) for x, y in zip(out, ref))


def test_two_steps_at_once(dev):
    """Two streams, each with its own workspace, and nothing between them."""
    sets = [to(O.inputs(30 + 41 * i, 4, 4104, 64, seed=40 + i), dev) for i in range(2)]
    spaces = [m.new_score_workspace(len(d["prev"]), 4104, 64, 4) for d in sets]
    outs = [[torch.zeros_like(d["grad"]), torch.zeros_like(d["grad"]), torch.zeros_like(d["base"]),
             torch.zeros_like(d["w1"]), torch.zeros_like(d["w2"])] for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, o, ws, st in zip(sets, outs, spaces, streams):
            m.score_sequential(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], o[0], o[1],
                               ws, stream=st)
            m.score_backward(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], o[1],
                             d["grad"], o[2], o[3], o[4], ws, stream=st)
    torch.cuda.synchronize()
    for d, o in zip(sets, outs):
        lp, lse = score(d, None, dev)
        want = (lp, lse, *backward(d, None, lse, d["grad"], dev))
        assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_training_step_in_a_graph(dev):
    """Scoring, loss, gradients and the clip captured once, replayed on new
    inputs, each replay against the eager calls; two graphs share a workspace."""
    rows, k, V, R = 12, 4, 1544, 64
    d = to(O.inputs(rows, k, V, R, seed=17), dev)
    space = m.new_score_workspace(rows, V, R, k)
    f = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731

    def outputs():
        return dict(lp=f(rows, k), lse=f(rows, k), stats=f(4), grad=f(rows, k), gb=torch.zeros_like(d["base"]),
                    g1=torch.zeros_like(d["w1"]), g2=torch.zeros_like(d["w2"]), c1=torch.zeros_like(d["w1"]),
                    c2=torch.zeros_like(d["w2"]), norm=f(1))

    old, clip_space = f(rows, k) - 4.0, m.new_clip_workspace(2)

    def step(o, ws, cs):
        m.score_sequential(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], o["lp"],
                           o["lse"], ws, softcap=20.0)
        m.policy_loss(o["lp"], old, old, d["advantages"], d["tokens"], None, V, o["stats"], o["grad"], beta=0.1)
        m.score_backward(d["base"], d["w1"], d["w2"], d["prev"], d["tokens"], None, d["temperature"], o["lse"],
                         o["grad"], o["gb"], o["g1"], o["g2"], ws, softcap=20.0)
        m.clip_gradients([o["g1"], o["g2"]], [o["c1"], o["c2"]], 0.1, o["norm"], cs)

    step(outputs(), space, clip_space)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        o, graph = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(o, space, clip_space)
        graphs.append((graph, o))
    for i in range(4):
        new = to(O.inputs(rows, k, V, R, seed=30 + i), dev)
        for n in d:
            d[n].copy_(new[n])
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        eager = outputs()
        step(eager, m.new_score_workspace(rows, V, R, k), m.new_clip_workspace(2))
        torch.cuda.synchronize()
        for n, x in graphs[i % 2][1].items():
            assert torch.equal(x, eager[n]), (i, n)


def test_the_whole_chain(dev):
    """Head product -> drafting loop -> verifier -> scoring of the accepted
    tokens -> policy loss -> gradients -> clip."""
    rows, k, V, R, H = 6, 4, 1032, 64, 272
    g = torch.Generator().manual_seed(18)
    w = (torch.randn(V, H, generator=g) * 3 * H ** -0.5).bfloat16().to(dev)
    x = torch.randn(rows, k + 1, H, generator=g).bfloat16().to(dev)
    q = torch.empty(V, H, dtype=torch.uint8, device=dev)
    s = torch.empty(-(-V // 128), -(-H // 128), device=dev)
    m.quantize_head_fp8(w, q, s)
    target = torch.empty(rows, k + 1, V, dtype=torch.bfloat16, device=dev)
    m.head_logits_fp8(x, q, s, target, m.new_head_workspace(rows * (k + 1), H))
    base = target[:, :k].contiguous()
    w1, w2 = ((torch.randn(V, R, generator=g) * 0.1).bfloat16().to(dev) for _ in range(2))
    prev = torch.randint(0, V, (rows,), generator=g).to(dev)
    seeds = torch.arange(rows).to(dev)
    positions = torch.arange(k)[None].expand(rows, k).contiguous().to(dev)
    heat = torch.full((rows,), 0.3, device=dev)
    cache, tokens = torch.empty_like(base), torch.empty(rows, k, dtype=torch.int64, device=dev)
    m.sample_sequential(base, w1, w2, prev, seeds, positions, heat, cache, tokens,
                        m.new_workspace(rows, V, R, k))
    accepted = torch.empty(rows, k + 1, dtype=torch.int64, device=dev)
    n = torch.empty(rows, dtype=torch.int32, device=dev)
    m.greedy_accept(target, tokens, torch.full((rows,), k, dtype=torch.int32, device=dev), accepted, n,
                    m.new_verify_workspace(rows, k))
    # the drafted distribution's own log-probabilities of the drafted tokens
    d = dict(base=base, w1=w1, w2=w2, prev=prev, tokens=tokens, temperature=heat)
    lp, lse = score(d, None, dev)
    b = O.Block(base, w1, w2, prev, tokens, None, heat)
    near(lp, b.logprobs, 2 * b.off, "logprobs")
    # the loop samples from the rounded logits: a bf16 step of |z| / T each
    rounded = torch.log_softmax(cache.double() / 0.3, 2).gather(2, tokens[:, :, None])[:, :, 0]
    size = float(cache.double().abs().max()) / 0.3
    assert ((rounded - lp).abs() <= 2 * 3 * O.BF16 * size).all()
    # the accepted tokens, -1 after them, against the target's base logits
    d = dict(base=target, w1=w1, w2=w2, prev=prev, tokens=accepted, temperature=heat)
    alp, alse = score(d, None, dev)
    assert torch.equal(alp != 0, accepted >= 0) and torch.equal((accepted >= 0).sum(1).int(), n)
    adv = torch.where(accepted == torch.nn.functional.pad(tokens, (0, 1), value=-2), 1.0, -0.5)
    stats, grad = torch.empty(4, device=dev), torch.empty(rows, k + 1, device=dev)
    m.policy_loss(alp, alp, alp - 0.1, adv, accepted, None, V, stats, grad, beta=0.05)
    gb, g1, g2 = backward(d, None, alse, grad, dev)
    ob = O.Block(target, w1, w2, prev, accepted, None, heat)
    for (want, off), got, name in zip(ob.backward(grad), (gb, g1, g2), ("base", "w1", "w2")):
        near(got, want, off, name)
    norm = torch.empty(1, device=dev)
    want = float(torch.sqrt(g1.double().square().sum() + g2.double().square().sum()))
    m.clip_gradients([g1, g2], [g1, g2], want / 2, norm, m.new_clip_workspace(2))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    now = float(torch.sqrt(g1.double().square().sum() + g2.double().square().sum()))
    assert abs(now - want / 2) <= O.BF16 * want
