"""The norm before the head, embeddings, the state of seen tokens and logit
adjustments in binary64 on the CPU, from their formulas, with the error that
binary32 arithmetic and the roundings to the outputs' types may leave. Shares no
code with the library."""

from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24        # half a binary32 step, relative
TINY = 2.0 ** -149    # the smallest binary32 number


def f64(t):
    return t.detach().cpu().double()


def rounded(value, off, dtype):
    """The tolerance of a value that is off by at most ``off`` before it is rounded
    to ``dtype``: half a step of what is rounded, a subnormal's half step at least."""
    if dtype == torch.float32:
        return off + U * (value.abs() + off) + TINY
    return off + 2.0 ** -8 * (value.abs() + off) + 2.0 ** -133


def added(x, residual):
    """x + residual rounded once to their type. (Where a binary32 sum is not exact, the
    smaller term is below 2^-16 of the larger, far from the middle between two bf16.)"""
    x = x.detach().cpu()
    if residual is None:
        return x
    return (x.float() + residual.detach().cpu().float()).to(x.dtype)


def norm(h, weight, eps, offset):
    """(y, its tolerance as binary32, inv) of h [n, H]."""
    h, w = f64(h), f64(weight) + offset
    inv = 1.0 / torch.sqrt((h * h).mean(1) + float(np.float32(eps)))
    y = h * inv[:, None] * w
    # inv, offset + weight and the two products are rounded; a product may be subnormal
    return y, 4.01 * U * y.abs() + TINY * (2 + w.abs()), inv


def e4m3_half_step(q):
    """Half the distance of neighbouring E4M3 values around |q| <= 448."""
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def check_codes(y, off, codes, scales, hidden):
    """Codes' values [n, 128 wide] and scales [wide, >= n] of y [n, H] known to ``off``."""
    n, wide = len(y), -(-hidden // 128)
    codes, scales = f64(codes.cpu().view(torch.float8_e4m3fn)), f64(scales)[:, :n].T
    assert codes.shape == (n, 128 * wide)
    assert not codes[:, hidden:].any()
    for b in range(wide):
        part, slack = y[:, 128 * b:min(hidden, 128 * b + 128)], off[:, 128 * b:min(hidden, 128 * b + 128)]
        top = part.abs().amax(1)
        # the largest magnitude as the kernel has it, and the quotient's rounding
        assert ((scales[:, b] - top / 448).abs() <= slack.amax(1) / 448 * 1.01 + 1.01 * U * top / 448 + TINY).all(), b
        s = scales[:, b:b + 1]
        q = torch.where(s > 0, part / s, 0.0)
        near = e4m3_half_step(q) + torch.where(s > 0, slack / s, 0.0) + 2 * U * q.abs()
        got = codes[:, 128 * b:128 * b + part.shape[1]]
        # (a subnormal scale is far from top / 448: the codes saturate)
        bad = (got - q.clamp(-448, 448)).abs() > near
        assert not bad.any(), (b, got[bad][:4], q[bad][:4])


def norm_backward(grad_y, h, weight, inv, grad_total, offset):
    """((grad_x, tolerance), (grad_weight, tolerance)), before the outputs' rounding."""
    d, h, w, inv = f64(grad_y), f64(h), f64(weight) + offset, f64(inv)[:, None]
    t = torch.zeros_like(h) if grad_total is None else f64(grad_total)
    n, hidden = h.shape
    xh, g = h * inv, d * w
    mean = (g * xh).mean(1, keepdim=True)
    mean_off = U * (4.01 * (g * xh).abs().mean(1, keepdim=True) + mean.abs())
    inner = g - xh * mean
    dx = inv * inner + t
    # g: the weight's sum and the product; xh, its product with the mean; the
    # difference, the product with inv, the sum with grad_total
    off = inv * (2.01 * U * g.abs() + xh.abs() * mean_off + 2.01 * U * (xh * mean).abs() + U * inner.abs())
    off = 1.01 * (off + U * (inv * inner).abs() + U * dx.abs()) + 4 * TINY * (1 + inv)
    terms = d * xh
    # at least min(n, 256) holders add their rows, up to 16 of a workgroup their sums, then
    # 32 shares of up to 1024 workgroups, and these shares
    adds = -(-n // 256) + 16 + 32 + 32
    dw_off = (adds + 2.01) * U * terms.abs().sum(0) * 1.01 + n * TINY
    return (dx, off), (terms.sum(0), dw_off)


def embed(table, tokens, scale):
    table, tokens = f64(table), tokens.cpu()
    live = (tokens >= 0) & (tokens < len(table))
    out = table[torch.where(live, tokens, 0)] * float(np.float32(scale))
    out = torch.where(live[..., None], out, 0.0)
    return out, U * out.abs() + TINY


def embed_backward(grad_out, tokens, vocab, scale):
    """(grad_table, tolerance), before the table type's rounding."""
    tokens, scale = tokens.cpu().reshape(-1), float(np.float32(scale))
    grad = f64(grad_out).reshape(len(tokens), -1)
    live = (tokens >= 0) & (tokens < vocab)
    out, mass = (torch.zeros(vocab, grad.shape[1], dtype=torch.float64) for _ in range(2))
    out.index_add_(0, tokens[live], grad[live])
    mass.index_add_(0, tokens[live], grad[live].abs())
    count = torch.bincount(tokens[live], minlength=vocab)[:, None]
    # up to 64 rows are added one after another; of these sums up to 17 one after
    # another, or every 16th, and these 16; then the scale's product
    adds = count.clamp(max=64) + count / 1024 + 34
    return out * scale, 1.01 * U * (adds * mass * abs(scale) + (out * scale).abs()) + 2 * TINY


def bits(truths):
    """bool [..., V] as int32 words [..., ceil(V / 32)], the lowest bit first."""
    a = truths.cpu().numpy()
    a = np.concatenate([a, np.zeros((*a.shape[:-1], -a.shape[-1] % 32), bool)], -1)
    return torch.from_numpy(np.packbits(a, axis=-1, bitorder="little").view(np.int32).copy())


class State:
    """What slots of a state hold, as truth values and whole numbers."""

    def __init__(self, slots, vocab):
        self.prompt = torch.zeros(slots, vocab, dtype=torch.bool)
        self.counts = torch.zeros(slots, vocab, dtype=torch.int32)

    def count(self, tokens, lengths=None, prompt_lengths=None, slots=None, reset=False):
        rows, n = tokens.shape
        at = [int(slots[r]) if slots is not None else r for r in range(rows)]
        for r in range(rows):
            if reset and 0 <= at[r] < len(self.counts):
                self.prompt[at[r]], self.counts[at[r]] = False, 0
        for r in range(rows):
            if not 0 <= at[r] < len(self.counts):
                continue
            for j in range(n if lengths is None else min(n, int(lengths[r]))):
                t = int(tokens[r, j])
                if 0 <= t < self.counts.shape[1]:
                    if prompt_lengths is not None and j < int(prompt_lengths[r]):
                        self.prompt[at[r], t] = True
                    else:
                        self.counts[at[r], t] += 1

    def tensors(self, device="cpu"):
        return tuple(t.to(device) for t in (bits(self.prompt), bits(self.counts > 0), self.counts))


def adjust(logits, state=None, slots=None, drafted=None, repetition=None, frequency=None, presence=None,
           bias=None, allowed=None):
    """(values, tolerance before the type's rounding, which logits are computed).
    ``state`` a State, ``allowed`` bool [rows, k, V]."""
    x = f64(logits).clone()
    rows, k, V = x.shape
    off, named = torch.zeros_like(x), torch.zeros_like(x, dtype=torch.bool)
    for r in range(rows):
        number = lambda t, other: other if t is None else float(t[r])  # noqa: E731
        rep, freq, pres = number(repetition, 1.0), number(frequency, 0.0), number(presence, 0.0)
        prompt, counts = torch.zeros(V, dtype=torch.bool), torch.zeros(V, dtype=torch.int64)
        at = int(slots[r]) if slots is not None else r
        if state is not None and 0 <= at < len(state.counts):
            prompt, counts = state.prompt[at], state.counts[at].long()
        entries = {}
        if bias is not None:
            for b in range(int(bias[2][r]), int(bias[2][r + 1])):
                if 0 <= int(bias[0][b]) < V:
                    entries[int(bias[0][b])] = float(bias[1][b])
        for s in range(k):
            count = counts.clone()
            for j in range(s if drafted is not None else 0):
                if 0 <= int(drafted[r, j]) < V:
                    count[int(drafted[r, j])] += 1
            seen, out = prompt | (count > 0), count > 0
            z, o = x[r, s], off[r, s]
            z[seen] = torch.where(z[seen] > 0, z[seen] / rep, z[seen] * rep)
            o[seen] += U * z[seen].abs()
            fall = freq * count[out].double()
            o[out] += U * (fall.abs() + (z[out] - fall).abs())
            z[out] -= fall
            z[out] -= pres
            o[out] += U * z[out].abs()
            named[r, s] = seen
            for t, value in entries.items():
                z[t] += value
                o[t] += U * abs(z[t])
                named[r, s, t] = True
            if allowed is not None:
                z[~allowed[r, s]] = -math.inf
                named[r, s][~allowed[r, s]] = True
    off = torch.where(x.isfinite(), off, 0.0)
    return x, 1.01 * off + 2 * TINY, named


def close(got, want, off, dtype):
    """got within the tolerance of want, infinities and NaN where it has them."""
    got = f64(got)
    plain = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    other = ~plain & ~want.isnan()
    assert torch.equal(got[other], want[other])
    tol = rounded(want, off, dtype)
    bad = plain & ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
