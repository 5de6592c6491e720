"""Refusals of the E4M3 head, the scoring, the policy loss and the clip, on the
host: no call here reaches the GPU (the pointers are never dereferenced)."""

import ctypes
import math

import pytest

import markov_draft_sampling_step_amd as m

P = ctypes.c_void_p
A = [0x10000 * (i + 1) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(m.LIBRARY):
        from markov_draft_sampling_step_amd import build

        build.build()
    return m.lib()


def every_null_and_shift(call, n, aligned, optional=()):
    """Each pointer in turn NULL (unless optional), then each aligned one 2 off."""
    for i in range(n):
        p = list(A[:n])
        p[i] = 0
        if i not in optional:
            assert call(p) == -1, i
    for i in aligned:
        p = list(A[:n])
        p[i] += 2
        assert call(p) == -4, i


def test_quantize_head_refusals(lib):
    f = lambda p=A, v=256, h=256: lib.markov_quantize_head_fp8(P(p[0]), P(p[1]), P(p[2]), v, h, None)  # noqa: E731
    every_null_and_shift(lambda p: f(p), 3, (0, 1, 2))
    for v, h in ((0, 256), (-8, 256), (8, 0), (8, 8), (8, 24), (8, 1048592)):
        assert f(v=v, h=h) == -2, (v, h)
    assert f(v=0x7fff0008) == -8


def test_head_logits_refusals(lib):
    need = lib.markov_head_workspace_bytes(4, 256)
    assert need >= 4 * 256 + 4 * 2 * 4

    def f(p=A, t=4, v=256, h=256, ws=need):
        return lib.markov_head_logits_fp8(P(p[0]), P(p[1]), P(p[2]), P(p[3]), t, v, h, P(p[4]), ws, None)

    every_null_and_shift(lambda p: f(p), 5, (0, 1, 2, 3, 4))
    for t, v, h in ((0, 256, 256), (4, 0, 256), (4, 12, 256), (4, 256, 0), (4, 256, 40)):
        assert f(t=t, v=v, h=h) == -2, (t, v, h)
    assert f(t=65537) == -5
    assert f(v=0x7fff0008) == -8
    assert f(ws=need - 1) == -6
    for t, h in ((0, 256), (65537, 256), (4, 8), (4, 1048592)):
        assert lib.markov_head_workspace_bytes(t, h) == 0


def _shape(rows=2, vocab=4096, rank=32):
    return m.make_shape(rows, vocab, rank)


BAD_SHAPES = [(dict(rows=0), 3, -2), (dict(vocab=4100), 3, -2), (dict(vocab=0), 3, -2),
              (dict(vocab=0x7fff0008), 3, -8), (dict(vocab=0x1000008), 3, -8), (dict(rank=48), 3, -3), (dict(rank=8), 3, -3),
              (dict(rank=1024), 3, -3), ({}, 0, -2), (dict(rows=65537), 1, -5),
              (dict(rows=2), 32769, -5), (dict(rows=0x7fffffff), 0x7fffffff, -5)]


@pytest.mark.parametrize("shape,k,status", BAD_SHAPES)
def test_scoring_shapes(lib, shape, k, status):
    sh = _shape(**shape)
    assert lib.markov_score_workspace_bytes(ctypes.byref(sh), k) == 0
    assert _score(lib, sh=sh, k=k) == status
    assert _backward(lib, sh=sh, k=k) == status
    assert _loss(lib, sh=sh, k=k) == status


def _score(lib, p=A, sh=None, k=3, ws=1 << 40):
    sh = sh or _shape()
    return lib.markov_score_sequential(P(p[0]), P(p[1]), P(p[2]), P(p[3]), P(p[4]), P(p[5]), k, P(p[6]),
                                       P(p[7]), P(p[8]), None, ctypes.byref(sh), P(p[9]), ws)


def _backward(lib, p=A, sh=None, k=3, ws=1 << 40):
    sh = sh or _shape()
    return lib.markov_score_backward(P(p[0]), P(p[1]), P(p[2]), P(p[3]), P(p[4]), P(p[5]), k, P(p[6]),
                                     P(p[7]), P(p[8]), P(p[9]), P(p[10]), P(p[11]), None,
                                     ctypes.byref(sh), P(p[12]), ws)


def _loss(lib, p=A, sh=None, k=3, low=0.2, high=0.2, beta=0.1):
    sh = sh or _shape()
    return lib.markov_policy_loss(P(p[0]), P(p[1]), P(p[2]), P(p[3]), P(p[4]), P(p[5]), k, low, high, beta,
                                  P(p[6]), P(p[7]), None, ctypes.byref(sh))


def test_scoring_refusals(lib):
    need = lib.markov_score_workspace_bytes(ctypes.byref(_shape()), 3)
    assert need > 0
    every_null_and_shift(lambda p: _score(lib, p), 10, (0, 1, 2, 9), optional=(5, 6))
    every_null_and_shift(lambda p: _backward(lib, p), 13, (0, 1, 2, 9, 10, 11, 12), optional=(5, 6))
    assert _score(lib, ws=need - 1) == -6 and _backward(lib, ws=need - 1) == -6
    assert lib.markov_score_sequential(*[P(x) for x in A[:6]], 3, *[P(x) for x in A[:3]], None, None,
                                       P(A[0]), need) == -1


def test_policy_loss_refusals(lib):
    every_null_and_shift(lambda p: _loss(lib, p), 8, (), optional=(5,))
    for kw in (dict(low=-0.1), dict(high=-1e-9), dict(low=math.nan), dict(high=math.nan),
               dict(beta=math.nan), dict(beta=math.inf)):
        assert _loss(lib, **kw) == -9, kw


def test_clip_refusals(lib):
    def f(n=2, grads=A[:2], out=A[2:4], counts=(5, 6), types=(0, 1), max_norm=1.0, norm=A[5], space=A[6],
          ws=None):
        c = max(n, 0)
        arr = lambda t, v: (t * c)(*v[:c]) if v is not None else None  # noqa: E731
        return lib.markov_clip_gradients(arr(P, grads), arr(P, out), arr(ctypes.c_int64, counts),
                                         arr(ctypes.c_int32, types), n, max_norm, P(norm), P(space),
                                         lib.markov_clip_workspace_bytes(c) if ws is None else ws, None)

    assert f(n=-1) == -2 and lib.markov_clip_workspace_bytes(-1) == 0
    for name in ("grads", "out", "counts", "types"):
        assert f(**{name: None}) == -1, name
    assert f(norm=0) == -1 and f(space=0) == -1
    assert f(grads=[A[0], 0]) == -1 and f(out=[0, A[0]]) == -1
    assert f(counts=(5, -1)) == -2 and f(types=(0, 2)) == -2 and f(types=(-1, 0)) == -2
    assert f(max_norm=-1.0) == -9 and f(max_norm=math.nan) == -9
    assert f(grads=[A[0] + 1, A[1]]) == -4 and f(grads=[A[0], A[1] + 2]) == -4
    assert f(out=[A[2], A[3] + 2]) == -4 and f(space=A[6] + 8) == -4 and f(norm=A[5] + 2) == -4
    assert f(ws=lib.markov_clip_workspace_bytes(2) - 1) == -6


def test_python_checks(lib):
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        m.score_sequential(cpu, cpu[0], cpu[0], None, None, None, None, None, None, None)
    with pytest.raises(TypeError, match="w: dtype"):
        m.quantize_head_fp8(torch.zeros(8, 16), None, None)
    with pytest.raises(TypeError, match="dtype torch.float16"):
        m.clip_gradients([torch.zeros(4, dtype=torch.float16)], [None], 1.0, None, None)
    with pytest.raises(ValueError, match="1 gradients, 0 outputs"):
        m.clip_gradients([cpu], [], 1.0, None, None)
    with pytest.raises(m.MarkovError):
        m.new_score_workspace(2, 100, 32, 3)
    with pytest.raises(m.MarkovError):
        m.new_head_workspace(0, 128)


def test_head_launches_past_32_bits(lib):
    """2^16 tokens of 2^20 hidden values would take 8.6e9 threads to quantize."""
    f = lambda t, h: lib.markov_head_logits_fp8(*[P(x) for x in A[:4]], t, 256, h, P(A[4]), 1 << 40, None)  # noqa: E731
    assert f(65536, 1048576) == -2 and lib.markov_head_workspace_bytes(65536, 1048576) == 0
    # 16 threads for each 128 values: 2^32 of them are one too many
    assert f(65536, 524288) == -2 and lib.markov_head_workspace_bytes(65536, 524288) == 0
    assert lib.markov_head_workspace_bytes(65535, 524288) > 65535 * 524288


def test_sizes_past_32_bits_are_not_cut_off(lib, monkeypatch):
    """2^32 + 8 is not 8, in a size that is given or in a tensor's."""
    torch = pytest.importorskip("torch")
    big = 2 ** 32 + 8
    for call in (lambda: m.new_head_workspace(big, 256), lambda: m.new_head_workspace(8, big + 8),
                 lambda: m.new_score_workspace(big, 4096, 32, 1), lambda: m.new_score_workspace(2, big, 32, 1),
                 lambda: m.new_score_workspace(2, 4096, 2 ** 32 + 32, 1), lambda: m.new_score_workspace(2, 4096, 32, big),
                 lambda: m.new_score_workspace(2, 4096, 32, 8 - 2 ** 32), lambda: m.new_clip_workspace(big, "cpu"),
                 lambda: m.policy_loss(None, None, None, None, None, None, big, None, None)):
        with pytest.raises(ValueError, match="past a 32-bit integer"):
            call()
    monkeypatch.setattr(m, "_dev", lambda *a, **kw: None)   # (tensors of these sizes without memory)
    on = lambda *s: torch.empty(*s, device="meta")  # noqa: E731
    w1 = on(8, 16)
    for call in (lambda: m.quantize_head_fp8(on(big, 16), None, None), lambda: m.quantize_head_fp8(on(8, big + 8), None, None),
                 lambda: m.head_logits_fp8(on(big, 16), on(8, 16), None, None, None),
                 lambda: m.head_logits_fp8(on(2, 2 ** 31, 16), on(8, 16), None, None, None),
                 lambda: m.head_logits_fp8(on(8, 16), on(big, 16), None, None, None),
                 lambda: m.score_sequential(on(big, 1, 8), w1, w1, *[None] * 7),
                 lambda: m.score_sequential(on(1, big, 8), w1, w1, *[None] * 7),
                 lambda: m.score_backward(on(1, 1, big), w1, w1, *[None] * 10),
                 lambda: m.policy_loss(on(big, 1), None, None, None, None, None, 8, None, None),
                 lambda: m.policy_loss(on(1, big), None, None, None, None, None, 8, None, None)):
        with pytest.raises(ValueError, match="past a 32-bit integer"):
            call()
