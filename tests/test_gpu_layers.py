"""The operators between a drafter's layers and the loop in a run, as they are used
together: on the GPU, through the C ABI."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_oracle as O  # noqa: E402
import markov_draft_sampling_step_amd as m  # noqa: E402

BF, FP, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m.lib()
    return torch.device("cuda:0")


def test_a_serving_step(dev):
    """Norm to codes, the head's product, masks and penalties where the logits stand,
    the loop, verification of adjusted target logits, the accepted tokens counted:
    eagerly, and captured and replayed with other inputs and a state that goes on."""
    rows, k, V, H, R = 4, 3, 4104, 528, 32
    g = torch.Generator().manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, qs = torch.empty(V, H, dtype=torch.uint8, device=dev), torch.empty(-(-V // 128), -(-H // 128), device=dev)
    m.quantize_head_fp8((normal(V, H) * H ** -0.5).to(BF).to(dev), q, qs)
    w1, w2, weight = ((normal(*s) * 0.3).to(BF).to(dev) for s in ((V, R), (V, R), (H,)))
    x, r = ((normal(rows, k, H) * 4).to(BF).to(dev) for _ in range(2))
    total, base, cache = (torch.empty(rows, k, n, dtype=BF, device=dev) for n in (H, V, V))
    states = m.new_states_fp8(rows * k, H, dev)
    state = m.new_token_state(6, V, dev)
    want = O.State(6, V)
    slots = torch.tensor([2, 5, 0, 3], dtype=I32)
    prompt = torch.randint(0, V, (rows, 50), generator=g)
    m.count_tokens(state, prompt.to(dev), prompt_lengths=torch.full((rows,), 50, dtype=I32, device=dev), slots=slots.to(dev),
                   reset=True)
    want.count(prompt, prompt_lengths=torch.full((rows,), 50), slots=slots)
    allowed = torch.rand(rows, k + 1, V, generator=g) < 0.01
    allowed[2:] = True
    words = O.bits(allowed).to(dev)
    first = words[:, :k].contiguous()
    rates = dict(repetition=torch.tensor([1.5, 1.0, 2.0, 1.1]), frequency=torch.tensor([0.5, 0.0, 1.0, 0.0]),
                 presence=torch.tensor([0.0, 1.0, 0.5, 2.0]))
    on = {n: t.to(dev) for n, t in rates.items()}
    prev, seeds = torch.zeros(rows, dtype=torch.int64, device=dev), torch.arange(rows, device=dev)
    positions = torch.arange(k, device=dev).repeat(rows, 1)
    heat = torch.tensor([0.0, 0.8, 0.0, 1.0], device=dev)
    tokens, accepted = (torch.empty(rows, n, dtype=torch.int64, device=dev) for n in (k, k + 1))
    length, full = torch.empty(rows, dtype=I32, device=dev), torch.full((rows,), k, dtype=I32, device=dev)
    target = (normal(rows, k + 1, V) * 3).to(BF).to(dev)
    judged = torch.empty_like(target)
    ws, vs = m.new_workspace(rows, V, R, k), m.new_verify_workspace(rows, k)
    on_slots = slots.to(dev)

    def step():
        m.add_norm(x, r, weight, None, total, None, states=states, offset=1.0)
        m.head_logits_states(states, q, qs, base)
        m.adjust_logits(base, base, state=state, slots=on_slots, allowed=first, **on)
        m.sample_sequential(base, w1, w2, prev, seeds, positions, heat, cache, tokens, ws)
        m.adjust_logits(target, judged, state=state, slots=on_slots, drafted=tokens, allowed=words, **on)
        m.greedy_accept(judged, tokens, full, accepted, length, vs)
        m.count_tokens(state, accepted, lengths=length, slots=on_slots)

    def check():
        torch.cuda.synchronize()
        y, off, _ = O.norm(total.view(-1, H), weight, 1e-6, 1.0)
        O.check_codes(y, off, *states, H)
        drafted = tokens.cpu()
        value, slack, _ = O.adjust(target, state=want, slots=slots, drafted=drafted, allowed=allowed, **rates)
        O.close(judged, value, slack, BF)
        best = judged.cpu().float().argmax(2)
        for row in range(rows):
            n = 0
            while n < k and drafted[row, n] == best[row, n]:
                n += 1
            assert accepted[row, :n + 1].tolist() == [*drafted[row, :n].tolist(), int(best[row, n])]
            assert all(allowed[row, s, t] for s, t in enumerate(drafted[row].tolist()))
        want.count(accepted.cpu(), length.cpu(), slots=slots)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(state, want.tensors()))

    for _ in range(2):
        step()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_((normal(rows, k, H) * 4).to(BF))
        target.copy_((normal(rows, k + 1, V) * 3).to(BF))
        graph.replay()
        check()


@pytest.mark.parametrize("t", [BF, FP])
def test_a_training_step(dev, t):
    """Embeddings of blocks that are mostly the mask token, the norm, both gradients,
    the clip: against the formulas one after another, in binary64."""
    rows, k, V, H, scale = 120, 5, 300, 272, 8.0
    g = torch.Generator().manual_seed(2)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    tokens = torch.randint(0, V, (rows, k), generator=g)
    tokens[:, 1:] = V - 1
    tokens[::7, 2:] = -1
    table, weight = normal(V, H).to(t).to(dev), (0.2 * normal(H)).to(dev)
    residual, dy, dt = (normal(rows, k, H).to(t).to(dev) for _ in range(3))
    x, y, total = (torch.empty(rows, k, H, dtype=t, device=dev) for _ in range(3))
    inv, dw, dtable = torch.empty(rows, k, device=dev), torch.empty(H, device=dev), torch.empty_like(table)
    on = tokens.to(dev)
    m.embed(table, on, x, scale=scale)
    m.add_norm(x, residual, weight, y, total, inv, offset=1.0)
    m.add_norm_backward(dy, total, weight, inv, dt, dt, dw, m.new_norm_workspace(rows * k, H, dev), offset=1.0)
    m.embed_backward(dt, on, dtable, m.new_embed_workspace(rows * k, H, dev), scale=scale)
    norm = torch.empty(1, device=dev)
    grads = [dw, dtable]
    before = [p.clone() for p in grads]
    m.clip_gradients(grads, grads, 0.5, norm, m.new_clip_workspace(grads))
    value, off = O.embed(table, tokens, scale)
    O.close(x, value, off, t)
    h = O.added(x, residual)
    assert torch.equal(total.cpu(), h)
    flat = lambda a: a.reshape(rows * k, H)  # noqa: E731
    value, off, exact_inv = O.norm(flat(h), weight, 1e-6, 1.0)
    O.close(flat(y), value, off, t)
    g2 = torch.Generator().manual_seed(2)
    again = lambda *s: torch.randn(*s, generator=g2)  # noqa: E731
    torch.randint(0, V, (rows, k), generator=g2)
    again(V, H), again(H), again(rows, k, H), again(rows, k, H)
    first_dt = again(rows, k, H).to(t)   # (grad_x was written over it)
    (dx, dx_off), (want, want_off) = O.norm_backward(flat(dy), flat(h), weight, inv.view(-1), flat(first_dt), 1.0)
    O.close(flat(dt), dx, dx_off, t)
    O.close(before[0], want, want_off, FP)
    O.close(before[1], *O.embed_backward(dt, tokens, V, scale), t)
    size = math.sqrt(sum(float((p.double() ** 2).sum()) for p in before))
    assert abs(float(norm) - size) <= 2.0 ** -23 * size
    assert float(grads[1].float().norm()) < 0.51


def test_refusals_on_the_device(dev):
    """What only a device tensor can be refused for: its strides, its device, shapes that
    do not belong together, overlaps."""
    on = lambda *s, t=BF: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    x, w, i64 = on(4, 64), on(64), torch.int64
    every_other = on(4, 128)[:, ::2]
    refused = [
        (ValueError, "x: must be contiguous", lambda: m.add_norm(every_other, None, w, x, None, None)),
        (ValueError, "residual: must be contiguous", lambda: m.add_norm(x, every_other, w, on(4, 64), None, None)),
        (ValueError, "weight: shape", lambda: m.add_norm(x, None, on(63), on(4, 64), None, None)),
        (ValueError, "weight: must be a device", lambda: m.add_norm(x, None, w.cpu(), on(4, 64), None, None)),
        (ValueError, "inv: shape", lambda: m.add_norm(x, None, w, on(4, 64), None, on(5, t=FP))),
        (ValueError, "codes: shape", lambda: m.add_norm(x, None, w, None, None, None, states=m.new_states_fp8(5, 64, dev))),
        (m.MarkovError, "NULL", lambda: m.add_norm(x, None, w, None, on(4, 64), None)),
        (m.MarkovError, "SHAPE", lambda: m.add_norm(on(4, 40), None, on(40), on(4, 40), None, None)),
        (m.MarkovError, "VALUE", lambda: m.add_norm(x, None, w, on(4, 64), None, None, eps=0.0)),
        (m.MarkovError, "ALIGN", lambda: m.add_norm(on(4 * 64 + 1)[1:].view(4, 64), None, w, x, None, None)),
        (m.MarkovError, "WORKSPACE", lambda: m.add_norm_backward(x, on(4, 64), w, on(4, t=FP), None, on(4, 64), on(64),
                                                                 on(8, t=torch.uint8))),
        (TypeError, "grad_x: dtype", lambda: m.add_norm_backward(x, on(4, 64), w, on(4, t=FP), None, on(4, 64, t=FP), on(64),
                                                                 m.new_norm_workspace(4, 64, dev))),
        (ValueError, "out: shape", lambda: m.embed(on(9, 64), on(4, t=i64), on(5, 64))),
        (TypeError, "tokens: dtype", lambda: m.embed(on(9, 64), on(4, t=I32), on(4, 64))),
        (ValueError, "grad_out: shape", lambda: m.embed_backward(on(5, 64), on(4, t=i64), on(9, 64), m.new_embed_workspace(4, 64, dev))),
        (ValueError, "prompt: shape", lambda: m.count_tokens((on(2, 3, t=I32), on(2, 3, t=I32), on(2, 64, t=I32)), on(2, 5, t=i64))),
        (ValueError, "lengths: shape", lambda: m.count_tokens(m.new_token_state(2, 64, dev), on(2, 5, t=i64), on(3, t=I32))),
        (ValueError, "state: of 64 tokens", lambda: m.adjust_logits(on(2, 3, 72), on(2, 3, 72), state=m.new_token_state(2, 64, dev))),
        (ValueError, "drafted: shape", lambda: m.adjust_logits(on(2, 3, 64), on(2, 3, 64), drafted=on(2, 1, t=i64))),
        (ValueError, "bias starts: shape", lambda: m.adjust_logits(on(2, 3, 64), on(2, 3, 64),
                                                                   bias=(on(4, t=i64), on(4, t=FP), on(2, t=I32)))),
        (ValueError, "allowed: shape", lambda: m.adjust_logits(on(2, 3, 64), on(2, 3, 64), allowed=on(2, 3, 1, t=I32))),
        (TypeError, "logits: dtype", lambda: m.adjust_logits(on(2, 3, 64, t=torch.float16), on(2, 3, 64))),
        (m.MarkovError, "SHAPE", lambda: m.adjust_logits(on(2, 3, 60), on(2, 3, 60))),
        (ValueError, "codes: shape", lambda: m.head_logits_states(m.new_states_fp8(4, 128, dev), on(8, 64, t=torch.uint8),
                                                                  on(1, 1, t=FP), on(5, 8))),
    ]
    for error, text, call in refused:
        with pytest.raises(error, match=text):
            call()
    both = on(2, 2, 64)
    with pytest.raises(m.MarkovError, match="VALUE"):
        m.adjust_logits(both.view(-1)[:128].view(2, 1, 64), both.view(-1)[64:192].view(2, 1, 64))


def test_the_current_stream(dev):
    """Calls without a stream go to the one that is current, behind what it has to do."""
    side = torch.cuda.Stream()
    x, w, out = torch.zeros(64, 4096, dtype=BF, device=dev), torch.ones(4096, device=dev), torch.zeros(64, 4096, dtype=BF, device=dev)
    big = torch.empty(1 << 28, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            big.normal_()
        x.fill_(2.0)
        m.add_norm(x, None, w, out, None, None)
        m.add_norm(out, out, w, out, None, None)
    side.synchronize()
    assert (out == 1).all()
