"""Gradient clipping on the GPU, through the C ABI, against binary64."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import markov_draft_sampling_step_amd as m  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m.lib()
    return torch.device("cuda:0")


def tensors(sizes, types, seed, dev):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, generator=g).to(t).to(dev) for n, t in zip(sizes, types)]


def check(grads, max_norm, in_place=False):
    before = [g.clone() for g in grads]
    out = grads if in_place else [torch.full_like(g, 3.0) for g in grads]
    norm = torch.full((1,), -1.0, device=grads[0].device if grads else "cuda")
    m.clip_gradients(grads, out, max_norm, norm, m.new_clip_workspace(grads))
    want = math.sqrt(sum(float((g.double().cpu() ** 2).sum()) for g in before))
    # the sum is in binary64: its root is a binary32 rounding from exact
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    by = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(before, out):
        exact = g.double() * by
        half = torch.finfo(g.dtype).eps / 2
        # the factor and the product in binary32, then the type's rounding
        off = exact.abs() * (half * (g.dtype != torch.float32) + 3 * 2.0 ** -24) + 2.0 ** -149
        assert ((o.double() - exact).abs() <= off).all()
        if by == 1.0:
            assert torch.equal(o, g)
    if not in_place:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    return norm


BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6, math.inf])
@pytest.mark.parametrize("sizes,types", [
    ([1], [BF]), ([1], [FP]), ([7, 0, 4097, 16384, 16385], [FP, BF, BF, FP, BF]),
    ([1000003, 5, 65536 * 3], [BF, FP, FP])])
def test_clip(dev, sizes, types, max_norm):
    for in_place in (False, True):
        check(tensors(sizes, types, len(sizes), dev), max_norm, in_place)


def test_many_tensors_take_several_launches(dev):
    sizes = [1 + (i * 37) % 900 for i in range(203)]
    check(tensors(sizes, [(BF, FP)[i % 2] for i in range(203)], 3, dev), 1.0)


def test_no_tensors(dev):
    check([], 1.0)
    check([torch.empty(0, device=dev)], 1.0)


def test_views_of_any_alignment(dev):
    for t in (BF, FP):
        flat = torch.randn(70000, generator=torch.Generator().manual_seed(4)).to(t).to(dev)
        for a, b in ((1, 2), (3, 40000), (5, 33001), (8, 8 + 32768), (2, 66667)):
            out = torch.full((70000,), 9.0, dtype=t, device=dev)
            norm = torch.empty(1, device=dev)
            m.clip_gradients([flat[a:b]], [out[a + 1:b + 1]], 0.25, norm, m.new_clip_workspace(1))
            other = torch.empty_like(flat[a:b])
            m.clip_gradients([flat[a:b].clone()], [other], 0.25, norm, m.new_clip_workspace(1))
            assert torch.equal(out[a + 1:b + 1], other)
            assert (out[:a + 1] == 9).all() and (out[b + 1:] == 9).all()


def test_large_and_small_values(dev):
    """Squares past binary32's range at either end."""
    check([torch.full((1000,), 1e30, device=dev), torch.full((10,), 1e-30, dtype=BF, device=dev)], 1.0)
    check([torch.full((1000,), 1e-30, device=dev)], 1e-33)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_not_finite_leaves_the_gradients(dev, bad):
    grads = tensors([5000, 300], [FP, BF], 5, dev)
    grads[1][7] = bad
    before = [g.clone() for g in grads]
    out, norm = [torch.zeros_like(g) for g in grads], torch.zeros(1, device=dev)
    for o in (out, grads):
        m.clip_gradients(grads, o, 0.1, norm, m.new_clip_workspace(grads))
        assert not math.isfinite(float(norm))
        assert all(torch.equal(x.nan_to_num(1, 2, 3), b.nan_to_num(1, 2, 3)) and torch.equal(x.isnan(), b.isnan())
                   for x, b in zip(o, before))


def test_repeats_bit_for_bit_and_in_a_graph(dev):
    grads = tensors([300001, 77, 120000], [FP, BF, BF], 6, dev)
    out, norm = [torch.zeros_like(g) for g in grads], torch.zeros(1, device=dev)
    space = m.new_clip_workspace(grads)
    m.clip_gradients(grads, out, 1.0, norm, space)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.clip_gradients(grads, out, 1.0, norm, space)
    for i in range(4):
        for g in grads:
            g.mul_(0.5 + i)
        graph.replay()
        torch.cuda.synchronize()
        again, n = [torch.zeros_like(g) for g in grads], torch.zeros(1, device=dev)
        m.clip_gradients(grads, again, 1.0, n, m.new_clip_workspace(grads))
        assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(again, out)), i


def test_two_streams_at_once(dev):
    sets = [tensors([50000 + s, 1234], [FP, BF], 7 + s, dev) for s in range(2)]
    outs = [[torch.zeros_like(g) for g in gs] for gs in sets]
    norms, spaces = [torch.zeros(1, device=dev) for _ in sets], [m.new_clip_workspace(gs) for gs in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            m.clip_gradients(sets[i], outs[i], 1.0, norms[i], spaces[i], stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        out, n = [torch.zeros_like(g) for g in sets[i]], torch.zeros(1, device=dev)
        m.clip_gradients(sets[i], out, 1.0, n, spaces[i])
        assert torch.equal(n, norms[i]) and all(torch.equal(a, b) for a, b in zip(out, outs[i]))


def test_empty_tensors_among_many(dev):
    """Empty tensors in the first group of launches, whose places no tensor of
    the next group takes; groups of nothing but empty ones."""
    for n, empty in ((70, (0, 5)), (200, range(0, 150, 3)), (130, range(64)), (64, (0,)), (128, range(40, 128))):
        sizes = [0 if i in empty else 1 + (i * 41) % 700 for i in range(n)]
        for in_place in (False, True):
            check(tensors(sizes, [(FP, BF)[i % 2] for i in range(n)], n, dev), 0.5, in_place)


def test_a_norm_past_binary32_is_not_finite(dev):
    """A sum of squares that binary64 holds and whose root binary32 does not."""
    for in_place in (False, True):
        grads = [torch.full((1000,), 1e38, device=dev), torch.ones(300, dtype=BF, device=dev)]
        before = [g.clone() for g in grads]
        out = grads if in_place else [torch.zeros_like(g) for g in grads]
        norm = torch.zeros(1, device=dev)
        m.clip_gradients(grads, out, 1.0, norm, m.new_clip_workspace(grads))
        assert float(norm) == math.inf
        assert all(torch.equal(o, b) for o, b in zip(out, before))


@pytest.mark.parametrize("max_norm", [2.0 ** -10, 2.0 ** -16, 1.0])
def test_a_factor_below_the_smallest_normal_number(dev, max_norm):
    for in_place in (False, True):
        # (a norm of 1.7e38: sqrt(777 / 3) 1e37 and 3 x 2e37)
        check([torch.linspace(-1e37, 1e37, 777, device=dev), torch.full((9,), 2e37, dtype=BF, device=dev)], max_norm,
              in_place)


def test_a_tensor_listed_twice(dev):
    """It counts twice; in place, where it would be scaled twice, it is refused."""
    a, b = tensors([500, 40], [FP, BF], 9, dev)
    norm, space = torch.zeros(1, device=dev), m.new_clip_workspace(3)
    out = [torch.zeros_like(x) for x in (a, b, a)]
    m.clip_gradients([a, b, a], out, 1.0, norm, space)
    want = math.sqrt(float(2 * a.double().square().sum() + b.double().square().sum()))
    assert abs(float(norm) - want) <= 2.0 ** -23 * want and torch.equal(out[0], out[2])
    before = a.clone()
    for grads, out in (([a, b, a], [a, b, a]), ([a, b, b], [a, out[1], out[1]])):
        with pytest.raises(ValueError, match="twice"):
            m.clip_gradients(grads, out, 1.0, norm, space)
    assert torch.equal(a, before)
    nothing = torch.empty(0, device=dev)
    m.clip_gradients([nothing, nothing], [nothing, nothing], 1.0, norm, space)
