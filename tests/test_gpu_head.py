"""The E4M3 head on the GPU, through the C ABI: the quantizers bit for bit,
the product against binary64 within a bf16 rounding and its fp32 sums."""

import numpy as np
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


def head(V, H, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, H, generator=g) * torch.exp(torch.randn(V, 1, generator=g))
    w[V // 3] = 0.0
    return w.bfloat16()


def states(n, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, generator=g)
    x[:, torch.randint(0, H, (2,), generator=g)] *= 30.0
    x[n // 2] = 0.0 if n > 2 else x[n // 2]
    return x.bfloat16()


def quantized(w, dev):
    V, H = w.shape
    q = torch.full((V, H), 0x55, dtype=torch.uint8, device=dev)
    s = torch.full((-(-V // 128), -(-H // 128)), -1.0, device=dev)
    m.quantize_head_fp8(w.to(dev), q, s)
    return q, s


def values_of(q):
    return q.cpu().view(torch.float8_e4m3fn).double().numpy()


def logits(x, q, s, dev, space=None, **kw):
    out = torch.full((*x.shape[:-1], q.shape[0]), 7.0, dtype=torch.bfloat16, device=dev)
    space = m.new_head_workspace(x.numel() // x.shape[-1], x.shape[-1]) if space is None else space
    m.head_logits_fp8(x.to(dev), q, s, out, space, **kw)
    return out


@pytest.mark.parametrize("V,H", [(1, 16), (8, 16), (130, 144), (128, 128), (384, 272), (4104, 1040), (129, 4096)])
def test_quantizer_is_exact(dev, V, H):
    w = head(V, H, V + H)
    q, s = quantized(w, dev)
    values, scales = O.quantize(w, 128)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(values_of(q), values)


def test_quantizer_extremes(dev):
    """The smallest and largest magnitudes, and blocks that hold a NaN or an infinity."""
    w = torch.zeros(128 * 6, 128)
    w[3, 5], w[4, 6] = 3.3895e38, -1e-30
    w[128:256] = torch.randn(128, 128, generator=torch.Generator().manual_seed(1)) * 1e-38
    w[256, 0] = 9.2e-41                         # a subnormal alone: the scale underflows to less than one step
    w[384 + 7, 3], w[512 + 9, 1], w[512, 0] = float("nan"), float("inf"), 1.0
    w = w.bfloat16()
    q, s = quantized(w, dev)
    s = s.cpu().numpy()[:, 0]
    values, scales = O.quantize(w[:384], 128)
    assert np.array_equal(s[:3], scales[:, 0]) and np.array_equal(values_of(q)[:384], values)
    assert np.isnan(s[3]) and np.isinf(s[4]) and s[5] == 0
    got = values_of(q)
    assert np.isnan(got[384:512]).all() and np.isnan(got[512 + 9, 1]) and got[512, 0] == 0 and not got[640:].any()


@pytest.mark.parametrize("n,V,H", [
    (1, 8, 16), (1, 4096, 512), (3, 136, 48), (5, 1000, 128), (6, 4096, 512), (16, 264, 272), (17, 520, 1040),
    (31, 2048, 384), (33, 256, 4096), (64, 1024, 640), (65, 648, 896), (127, 384, 256), (130, 1288, 144),
    (256, 1024, 512), (300, 808, 1296), (513, 1032, 208)])
def test_product(dev, n, V, H):
    w, x = head(V, H, 3), states(n, H, 4)
    q, s = quantized(w, dev)
    want, off = O.product(x, values_of(q), s.cpu().numpy())
    got = logits(x, q, s, dev).cpu().double().numpy()
    bad = np.abs(got - want) > off
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("n,V,H", [(200, 520, 272), (480, 264, 144), (2049, 136, 400), (4, 264, 16400)])
def test_product_more_shapes(dev, n, V, H):
    test_product(dev, n, V, H)


def test_offsets_past_32_bits(dev):
    """A head of more than 4 GiB, and logits of more than 4 GiB: the last entries
    against the formula, and the first against a call of their own."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    torch.manual_seed(13)
    V, H, n = 270008, 16016, 3
    w = torch.empty(V, H, dtype=torch.bfloat16, device=dev).normal_()
    q, s = quantized(w, dev)
    tail = V // 128 * 128
    values, scales = O.quantize(w[tail:].cpu(), 128)
    assert np.array_equal(values_of(q[tail:]), values) and np.array_equal(s[-1:].cpu().numpy(), scales)
    del w
    x = states(n, H, 14)
    out = logits(x, q, s, dev)
    want, off = O.product(x, values, scales)
    assert (np.abs(out[:, tail:].cpu().double().numpy() - want) <= off).all()
    assert torch.equal(out[:, :1024], logits(x, q[:1024], s[:8].contiguous(), dev))
    # 8200 x 270008 logits of short rows
    H, n = 64, 8200
    q, s = quantized(torch.empty(V, H, dtype=torch.bfloat16, device=dev).normal_(), dev)
    x = states(n, H, 15)
    out = logits(x, q, s, dev)
    want, off = O.product(x[-40:], values_of(q[tail:]), s[-1:].cpu().numpy())
    assert (np.abs(out[-40:, tail:].cpu().double().numpy() - want) <= off).all()


@pytest.mark.parametrize("n", [5, 20, 50, 70, 130, 160, 190, 224, 256])
def test_a_streamed_head_gives_the_same_logits(dev, n):
    """A head of more than 256 MiB (streamed past the caches) against its first
    rows alone (which are not)."""
    V, H = 16904, 16384
    g = torch.Generator(device=dev).manual_seed(22)
    q = torch.randint(0, 126, (V, H), dtype=torch.uint8, device=dev, generator=g)
    s = torch.rand(-(-V // 128), H // 128, device=dev, generator=g)
    x = states(n, H, 23).to(dev)
    part = logits(x, q[:8192], s[:64].contiguous(), dev)
    assert V * H > 256 << 20 and torch.equal(logits(x, q, s, dev)[:, :8192], part) and part.isfinite().all()


def test_two_products_at_once(dev):
    """Two streams, each with its own workspace."""
    q, s = quantized(head(8200, 1040, 16), dev)
    xs = [states(n, 1040, 17 + n).to(dev) for n in (7, 90)]
    spaces = [m.new_head_workspace(len(x), 1040) for x in xs]
    outs = [torch.zeros(len(x), 8200, dtype=torch.bfloat16, device=dev) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, ws, st in zip(xs, outs, spaces, streams):
            m.head_logits_fp8(x, q, s, o, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, logits(x, q, s, dev)) for x, o in zip(xs, outs))


def test_product_shapes_and_streams(dev):
    """[rows, k, H] states, a side stream, a reused workspace with a larger
    call before a smaller one, an output whose neighbours stay as they were."""
    q, s = quantized(head(520, 272, 5), dev)
    x = states(60, 272, 6).view(12, 5, 272)
    space = m.new_head_workspace(60, 272)
    first = logits(x, q, s, dev, space)
    assert first.shape == (12, 5, 520)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        small = logits(x[:2].contiguous(), q, s, dev, space)
    side.synchronize()
    assert torch.equal(small, first[:2])
    wide = torch.full((62 * 520,), 7.0, dtype=torch.bfloat16, device=dev)
    m.head_logits_fp8(x.view(60, 272).to(dev), q, s, wide[520:-520].view(60, 520), space)
    assert torch.equal(wide[520:-520].view_as(first), first)
    assert (wide[:520] == 7).all() and (wide[-520:] == 7).all()


def test_product_rows_do_not_depend_on_the_batch(dev):
    """A token's logits are the same whatever is computed beside it."""
    q, s = quantized(head(1032, 656, 7), dev)
    x = states(300, 656, 8)
    whole = logits(x, q, s, dev)
    for n in (1, 2, 16, 33, 64, 100, 129, 257):
        assert torch.equal(logits(x[:n].contiguous(), q, s, dev), whole[:n]), n
    # (whole blocks: the order of the sums differs between up to 64 tokens and more)
    q, s = quantized(head(1032, 640, 7), dev)
    x = states(300, 640, 8)
    for whole, few in ((300, (65, 129, 257)), (64, (1, 2, 16, 17, 33))):
        want = logits(x[:whole].contiguous(), q, s, dev)
        for n in few:
            assert torch.equal(logits(x[:n].contiguous(), q, s, dev), want[:n]), n


def test_nan_and_inf_states_stay_in_their_row(dev):
    q, s = quantized(head(264, 272, 9), dev)
    x = states(40, 272, 10)
    clean = logits(x, q, s, dev)
    x[7, 200], x[20, 0] = float("nan"), float("inf")
    got = logits(x, q, s, dev)
    assert got[7].isnan().all() and got[20].isnan().all()
    keep = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(got[keep], clean[keep])


def test_head_in_a_graph(dev):
    q, s = quantized(head(1032, 400, 11), dev)
    x = states(20, 400, 12).to(dev)
    space, out = m.new_head_workspace(20, 400), torch.zeros(20, 1032, dtype=torch.bfloat16, device=dev)
    m.head_logits_fp8(x, q, s, out, space)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.head_logits_fp8(x, q, s, out, space)
    for i in range(4):
        x.copy_(states(20, 400, 20 + i))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, logits(x, q, s, dev)), i
