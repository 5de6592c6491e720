"""The operators between a drafter's layers and the loop, on the shapes they are used at.

- ``norm``: a residual added to hidden states and their root-mean-square norm,
  as bf16 or fp32 states or as the E4M3 codes and scales that the head's product
  reads; ``norm_grad``: its gradients;
- ``embed``: the embeddings of a block's tokens, scaled; ``embed_grad``: the
  gradient of the embedding table;
- ``count``: the tokens that a request has seen, as its slot of a state that is
  kept from step to step;
- ``adjust``: penalties for those tokens, biases and grammar masks on logits,
  before the loop draws from them or a verifier compares them.

The vocabularies, rows and steps are those of the five drafting workloads (4096
with 2 rows of 3 steps, 129280 with 1 and 16 rows of 5, 163840 with 64 rows of 5
and 256 rows of 8), with generic hidden sizes.
"""

import math

import torch

own = False
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TYPES = {"bf16": BF16, "fp32": F32}
EPS = 1e-6


# -- the cases ---------------------------------------------------------------------

def listed():
    return [
        # one request's block of 5 positions before the head: latency
        dict(name="norm_single", op="norm", tokens=5, hidden=7168, type="bf16", weight="bf16",
             residual=True, codes=True),
        # a training batch, with what its backward pass needs
        dict(name="norm_train", op="norm", tokens=16384, hidden=4096, type="bf16", weight="fp32",
             residual=True, codes=False),
        # a small batch in fp32, a hidden size that ends inside a block
        dict(name="norm_grad_small", op="norm_grad", tokens=80, hidden=1040, type="fp32",
             weight="fp32", through=False),
        # the training batch's way back, with the gradient of the residual stream
        dict(name="norm_grad_train", op="norm_grad", tokens=16384, hidden=4096, type="bf16",
             weight="fp32", through=True),
        # a training batch's embeddings
        dict(name="embed_train", op="embed", tokens=16384, vocab=163840, hidden=4096, type="bf16",
             scale=64.0, same=0.8),
        # the smallest block
        dict(name="embed_grad_tiny", op="embed_grad", tokens=6, vocab=4096, hidden=512, type="bf16",
             table="bf16", scale=1.0, same=0.5),
        # a training batch of blocks of 5: four of five tokens are the mask token
        dict(name="embed_grad_train", op="embed_grad", tokens=16384, vocab=163840, hidden=4096,
             type="bf16", table="bf16", scale=64.0, same=0.8),
        # one request that starts with its prompt
        dict(name="count_single", op="count", rows=1, length=300, vocab=129280),
        # 256 requests that start with their prompts
        dict(name="count_stress", op="count", rows=256, length=4096, vocab=163840),
        # one request's block, everything at once
        dict(name="adjust_single", op="adjust", rows=1, k=5, vocab=129280, type="bf16", place="out",
             history=2000, biases=16, allowed=0.01),
        # half of 64 requests answer in a grammar: what it forbids is struck out
        # where the logits stand
        dict(name="adjust_grammar", op="adjust", rows=64, k=5, vocab=163840, type="bf16",
             place="in", history=0, biases=0, allowed=0.01),
        # 256 requests x 8 positions, everything at once
        dict(name="adjust_stress", op="adjust", rows=256, k=8, vocab=163840, type="bf16",
             place="out", history=2000, biases=16, allowed=0.5),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "count", "adjust", "adjust"])
    types = ["bf16", "bf16", "fp32"]
    if op in ("norm", "norm_grad"):
        hidden = 16 * _log_uniform(rng, 2, 1024)
        case = dict(op=op, tokens=_log_uniform(rng, 1, min(65536, 16384 * 4096 // hidden)), hidden=hidden,
                    type=rng.choice(types), weight=rng.choice(["bf16", "fp32"]))
        if op == "norm":
            case.update(residual=rng.random() < 0.75, codes=rng.random() < 0.5)
        else:
            case.update(through=rng.random() < 0.5)
        return case
    if op in ("embed", "embed_grad"):
        hidden, vocab = 16 * _log_uniform(rng, 2, 448), 8 * _log_uniform(rng, 64, 20480)
        vocab = min(vocab, 8 * (163840 * 4096 // 8 // hidden))
        case = dict(op=op, tokens=_log_uniform(rng, 1, min(65536, 16384 * 4096 // hidden)), vocab=vocab,
                    hidden=hidden, type=rng.choice(types), scale=rng.choice([1.0, 64.0, 0.125]),
                    same=rng.choice([0.0, 0.5, 0.8, 1.0]))
        if op == "embed_grad":
            case["table"] = "fp32" if case["type"] == "fp32" else "bf16"
        return case
    vocab = 8 * _log_uniform(rng, 512, 20480)
    if op == "count":
        return dict(op=op, rows=_log_uniform(rng, 1, 256), length=_log_uniform(rng, 1, 4096), vocab=vocab)
    place = rng.choice(["out", "out", "in"])
    plain = place == "in"   # (what a second pass over the same logits leaves as it is)
    return dict(op=op, rows=_log_uniform(rng, 1, 128), k=rng.randint(1, 8), vocab=vocab,
                type=rng.choice(types), place=place, history=0 if plain else rng.choice([0, 1, 300, 5000]),
                biases=0 if plain else rng.choice([0, 1, 16, 500]), allowed=rng.choice([1.0, 0.99, 0.5, 0.001]))


def _blocks(n):
    return -(-n // 128)


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, size, w = case["tokens"] * case["hidden"], _size(case["type"]), _size(case["weight"])
        if op == "norm":
            total = case["residual"]
            out = n + 4 * case["tokens"] * _blocks(case["hidden"]) if case["codes"] else size * n + 4 * case["tokens"]
            return {"bytes": size * n * (1 + 2 * total) + out + w * case["hidden"], "flops": 6 * n}
        return {"bytes": size * n * (3 + case["through"]) + 4 * case["tokens"] + 2 * w * case["hidden"],
                "flops": 12 * n}
    if op == "embed":
        n = case["tokens"] * case["hidden"]
        return {"bytes": 2 * _size(case["type"]) * n + 8 * case["tokens"], "flops": n}
    if op == "embed_grad":
        n = case["tokens"] * case["hidden"]
        return {"bytes": _size(case["type"]) * n + 8 * case["tokens"] + _size(case["table"]) * case["vocab"] * case["hidden"],
                "flops": 2 * n}
    rows, v = case["rows"], case["vocab"]
    if op == "count":
        return {"bytes": rows * (8 * case["length"] + 4 * v + 2 * v // 8), "flops": rows * case["length"]}
    m = rows * case["k"]
    bits = rows * v // 4 + m * v // 8 if case["history"] else m * v // 8
    small = rows * (16 + 4 * min(case["history"], v) + 12 * case["biases"])
    if case["place"] == "in":   # half of the rows are masked
        return {"bytes": bits + int(m * v * _size(case["type"]) * 0.5 * (1 - case["allowed"])), "flops": m * v}
    return {"bytes": bits + small + 2 * m * v * _size(case["type"]), "flops": m * v}


# -- the inputs --------------------------------------------------------------------

def _words(bits):
    """Truth values [..., V] as 32-bit words [..., ceil(V / 32)], the lowest bit first."""
    v = bits.shape[-1]
    bits = torch.nn.functional.pad(bits, (0, -v % 32)).view(*bits.shape[:-1], -1, 32)
    place = torch.tensor([1 << i for i in range(31)] + [-(1 << 31)], dtype=torch.int64, device=DEV)
    return (bits * place).sum(-1).to(I32)


def _truths(words, v):
    """The truth values of words, [..., v]."""
    place = torch.arange(32, dtype=I32, device=DEV)
    return ((words[..., None] >> place) & 1).bool().flatten(-2)[..., :v]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    uniform = lambda *shape: torch.rand(*shape, generator=g, device=DEV)  # noqa: E731
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        n, h, t, w = case["tokens"], case["hidden"], TYPES[case["type"]], TYPES[case["weight"]]
        x = normal(n, h)
        x[:, torch.randint(0, h, (max(1, h // 256),), generator=g, device=DEV)] *= 20.0   # outlier channels
        s["weight"] = (1.0 + 0.2 * normal(h)).to(w)
        if op == "norm":
            s.update(x=x.to(t), residual=(3.0 * normal(n, h)).to(t) if case["residual"] else None)
            s["total"] = torch.empty(n, h, dtype=t, device=DEV) if case["residual"] else None
            if case["codes"]:
                s["codes"] = torch.zeros(n, 128 * _blocks(h), dtype=torch.uint8, device=DEV)
                s["scales"] = torch.zeros(_blocks(h), -(-n // 256) * 256, device=DEV)
            else:
                s.update(y=torch.empty(n, h, dtype=t, device=DEV), inv=torch.empty(n, device=DEV))
            return s
        s.update(total=x.to(t), grad_y=(normal(n, h) * 0.01).to(t),
                 grad_total=(normal(n, h) * 0.01).to(t) if case["through"] else None)
        s["inv"] = (s["total"].double().square().mean(1) + EPS).rsqrt().float()
        s.update(grad_x=torch.empty(n, h, dtype=t, device=DEV), grad_weight=torch.empty(h, dtype=w, device=DEV))
        if own:
            import markov_draft_sampling_step_amd as m_

            s["space"] = m_.new_norm_workspace(n, h)
        return s
    if op in ("embed", "embed_grad"):
        n, v, h, t = case["tokens"], case["vocab"], case["hidden"], TYPES[case["type"]]
        # frequent tokens have small numbers; `same` of them are the mask token
        tokens = (v * uniform(n) ** 3).long().clamp(max=v - 1)
        s["tokens"] = torch.where(uniform(n) < case["same"], v - 3, tokens)
        if op == "embed":
            s.update(table=normal(v, h).mul_(h ** -0.5).to(t), out=torch.empty(n, h, dtype=t, device=DEV))
            return s
        s.update(grad_out=(normal(n, h) * 0.01).to(t),
                 grad_table=torch.empty(v, h, dtype=TYPES[case["table"]], device=DEV))
        if own:
            import markov_draft_sampling_step_amd as m_

            s["space"] = m_.new_embed_workspace(n, h)
        return s
    rows, v = case["rows"], case["vocab"]
    if op == "count":
        n = case["length"]
        s["tokens"] = (v * uniform(rows, n) ** 3).long().clamp(max=v - 1)
        s["lengths"] = (n * (0.25 + 0.75 * uniform(rows))).long().clamp(min=1).to(I32)
        s["prompts"] = (s["lengths"] * uniform(rows)).to(I32)
        s["slots"] = torch.randperm(rows, generator=g, device=DEV).to(I32)
        words = -(-v // 32)
        s["state"] = (torch.full((rows, words), -1, dtype=I32, device=DEV),
                      torch.full((rows, words), -1, dtype=I32, device=DEV),
                      torch.full((rows, v), 7, dtype=I32, device=DEV))
        return s
    k, t = case["k"], TYPES[case["type"]]
    s["logits"] = torch.randn(rows, k, v, generator=g, device=DEV).mul_(3.0).to(t)
    s["out"] = s["logits"] if case["place"] == "in" else torch.empty_like(s["logits"])
    for name in ("state", "slots", "drafted", "repetition", "frequency", "presence", "bias", "allowed"):
        s[name] = None
    if case["history"]:
        counts = torch.zeros(rows, v, dtype=I32, device=DEV)
        prompt = torch.zeros(rows, v, dtype=torch.bool, device=DEV)
        n = case["history"]
        old = (v * uniform(rows, n) ** 3).long().clamp(max=v - 1)
        prompt.scatter_(1, old[:, :n // 2], True)
        counts.scatter_add_(1, old[:, n // 2:], torch.ones(rows, n - n // 2, dtype=I32, device=DEV))
        s["state"] = (_words(prompt), _words(counts > 0), counts)
        s["slots"] = torch.randperm(rows, generator=g, device=DEV).to(I32)
        s["drafted"] = (v * uniform(rows, k) ** 3).long().clamp(max=v - 1)
        s["repetition"], s["frequency"], s["presence"] = 1.0 + 0.3 * uniform(rows), 0.5 * uniform(rows), uniform(rows)
    if case["biases"]:
        n = min(case["biases"], v)
        start = torch.randint(0, v, (rows, 1), generator=g, device=DEV)
        step = v // n   # (every row's tokens are different ones)
        s["bias"] = (((start + step * torch.arange(n, device=DEV)) % v).flatten(), 4.0 * normal(rows * n),
                     n * torch.arange(rows + 1, dtype=I32, device=DEV))
    if case["allowed"] < 1:
        allowed = torch.rand(rows, k, v, generator=g, device=DEV) < case["allowed"]
        allowed[rows // 2 + 1:] = True   # the others answer freely
        s["allowed"] = torch.stack([_words(a) for a in allowed])
    return s


# -- one pass ----------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import markov_draft_sampling_step_amd as m_

    case = s["case"]
    op = case["op"]
    if op == "norm":
        if case["codes"]:
            m_.add_norm(s["x"], s["residual"], s["weight"], None, s["total"], None,
                        states=(s["codes"], s["scales"]), eps=EPS)
            return _coded(s, s["codes"].view(torch.float8_e4m3fn), s["scales"], s["total"])
        m_.add_norm(s["x"], s["residual"], s["weight"], s["y"], s["total"], s["inv"], eps=EPS)
        return dict(y=s["y"], total=s["total"], inv=s["inv"])
    if op == "norm_grad":
        m_.add_norm_backward(s["grad_y"], s["total"], s["weight"], s["inv"], s["grad_total"],
                             s["grad_x"], s["grad_weight"], s["space"])
        return dict(grad_x=s["grad_x"], grad_weight=s["grad_weight"])
    if op == "embed":
        m_.embed(s["table"], s["tokens"], s["out"], scale=case["scale"])
        return s["out"]
    if op == "embed_grad":
        m_.embed_backward(s["grad_out"], s["tokens"], s["grad_table"], s["space"], scale=case["scale"])
        return s["grad_table"]
    if op == "count":
        m_.count_tokens(s["state"], s["tokens"], lengths=s["lengths"], prompt_lengths=s["prompts"],
                        slots=s["slots"], reset=True)
        return list(s["state"])
    m_.adjust_logits(s["logits"], s["out"], state=s["state"], slots=s["slots"], drafted=s["drafted"],
                     repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                     bias=s["bias"], allowed=s["allowed"])
    return s["out"]


def _coded(s, codes, scales, total):
    """What is returned of codes [tokens, ...] and scales [blocks, ...] that may end in padding."""
    n, h = s["x"].shape
    return dict(codes=codes[:, :h], scales=scales[:, :n], total=total)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float()
        total = None
        if s["residual"] is not None:
            total = (h + s["residual"].float()).to(s["x"].dtype)
            h = total.float()
        inv = (h.square().mean(1) + EPS).rsqrt()
        y = h * inv[:, None] * s["weight"].float()
        if not case["codes"]:
            return dict(y=y.to(s["x"].dtype), total=total, inv=inv)
        n, wide = len(y), _blocks(y.shape[1])
        pad = torch.nn.functional.pad(y, (0, wide * 128 - y.shape[1])).view(n, wide, 128)
        # a true quotient: by a plain number it would be a product with 1/448
        scales = pad.abs().amax(2) / torch.full((1, 1), 448.0, device=DEV)
        q = torch.where(scales[:, :, None] > 0, pad / scales[:, :, None], 0.0)
        return _coded(s, q.view(n, -1).to(torch.float8_e4m3fn), scales.T.contiguous(), total)
    if op == "norm_grad":
        g = s["grad_y"].float()
        xh = s["total"].float() * s["inv"][:, None]
        grad_weight = (g * xh).sum(0)
        g = g * s["weight"].float()
        d = s["inv"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["grad_total"] is not None:
            d += s["grad_total"].float()
        return dict(grad_x=d.to(s["total"].dtype), grad_weight=grad_weight.to(s["weight"].dtype))
    if op == "embed":
        return (s["table"][s["tokens"]].float() * case["scale"]).to(s["table"].dtype)
    if op == "embed_grad":
        order = torch.argsort(s["tokens"], stable=True)
        table = torch.zeros(s["grad_table"].shape, device=DEV)
        table.index_add_(0, s["tokens"][order], s["grad_out"][order].float())
        return (table * case["scale"]).to(s["grad_table"].dtype)
    if op == "count":
        n, v = s["tokens"].shape[1], case["vocab"]
        at = torch.arange(n, device=DEV)[None, :]
        inside, prompt = at < s["lengths"][:, None], at < s["prompts"][:, None]
        seen = torch.zeros(case["rows"], v, dtype=I32, device=DEV)
        seen.scatter_add_(1, s["tokens"], (inside & prompt).to(I32))
        fresh = torch.zeros(case["rows"], v, dtype=I32, device=DEV)
        fresh.scatter_add_(1, s["tokens"], (inside & ~prompt).to(I32))
        back = torch.empty_like(s["slots"])
        back[s["slots"].long()] = torch.arange(case["rows"], dtype=I32, device=DEV)
        seen, fresh = seen[back.long()], fresh[back.long()]
        return [_words(seen > 0), _words(fresh > 0), fresh]
    logits = s["logits"]
    rows, k, v = logits.shape
    if case["place"] == "in":
        logits.masked_fill_(~_truths(s["allowed"], v), -math.inf) if s["allowed"] is not None else None
        return logits
    x = logits.float()
    if s["state"] is not None:
        slots = s["slots"].long()
        old, counts = _truths(s["state"][0][slots], v), s["state"][2][slots].clone()
        for i in range(k):
            z, before = x[:, i], counts > 0
            rep = s["repetition"][:, None]
            z = torch.where(old | before, torch.where(z > 0, z / rep, z * rep), z)
            z = z - s["frequency"][:, None] * counts
            x[:, i] = z - s["presence"][:, None] * before
            counts.scatter_add_(1, s["drafted"][:, i:i + 1], torch.ones(rows, 1, dtype=I32, device=DEV))
    if s["bias"] is not None:
        tokens, values, _ = s["bias"]
        x.view(rows, k, v).scatter_add_(2, tokens.view(rows, 1, -1).expand(rows, k, -1),
                                        values.view(rows, 1, -1).expand(rows, k, -1))
    if s["allowed"] is not None:
        for i in range(k):
            x[:, i].masked_fill_(~_truths(s["allowed"][:, i], v), -math.inf)
    return x.to(logits.dtype)


# -- in 64 bits --------------------------------------------------------------------

def _nearest_e4m3(y):
    """The E4M3 value nearest to each binary64 value (ties to even)."""
    exponent = torch.frexp(y.abs().clamp(min=2.0 ** -9))[1] - 1
    step = torch.ldexp(torch.ones_like(y), exponent.clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = None
        h = s["x"].double()
        if s["residual"] is not None:
            total = h + s["residual"].double()
            h = total.to(s["x"].dtype).double()   # what is normalised is the sum as it is kept
        inv = 1.0 / torch.sqrt((h ** 2).sum(1) / h.shape[1] + EPS)
        y = torch.einsum("nh,n,h->nh", h, inv, s["weight"].double())
        if not case["codes"]:
            return dict(y=y, total=total, inv=inv)
        codes, scales = torch.empty_like(y), []
        for j in range(0, case["hidden"], 128):
            part = y[:, j:j + 128]
            scale = (part.abs().amax(1) / 448.0).float().double()   # a scale is a binary32 number
            scales.append(scale)
            codes[:, j:j + 128] = torch.where(scale[:, None] > 0, _nearest_e4m3(part / scale[:, None]), 0.0)
        return dict(codes=codes, scales=torch.stack(scales), total=total)
    if op == "norm_grad":
        h, w = s["total"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        # (the norm of a row as it was kept, in fp32: the gradients are those at this value)
        inv = s["inv"].double()
        with torch.no_grad():
            mean = (h ** 2).mean(1) + EPS
        live = inv * torch.sqrt(mean / ((h ** 2).mean(1) + EPS))
        y = h * live[:, None] * w
        y.backward(s["grad_y"].double())
        grad = h.grad
        if s["grad_total"] is not None:
            grad = grad + s["grad_total"].double()
        return dict(grad_x=grad, grad_weight=w.grad)
    if op == "embed":
        return torch.index_select(s["table"], 0, s["tokens"]).double() * case["scale"]
    if op == "embed_grad":
        out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device=DEV)
        tokens, order = torch.sort(s["tokens"])
        names, many = torch.unique_consecutive(tokens, return_counts=True)
        at = 0
        few = many <= 64
        # a token with many rows by a sum of its own, the others one rank at a time
        starts = torch.cumsum(many, 0) - many
        for t, a, c in zip(names[~few].tolist(), starts[~few].tolist(), many[~few].tolist()):
            for at in range(a, a + c, 4096):
                out[t] += s["grad_out"][order[at:min(at + 4096, a + c)]].double().sum(0)
        for r in range(int(many[few].max()) if bool(few.any()) else 0):
            has = few & (many > r)
            out[names[has]] += s["grad_out"][order[starts[has] + r]].double()
        return out.mul_(case["scale"])
    rows, v = case["rows"], case["vocab"]
    if op == "count":
        states = [torch.zeros_like(x) for x in s["state"]]
        for r in range(rows):
            p, n, at = int(s["prompts"][r]), int(s["lengths"][r]), int(s["slots"][r])
            states[0][at] = _words(torch.bincount(s["tokens"][r, :min(p, n)], minlength=v) > 0)
            fresh = torch.bincount(s["tokens"][r, min(p, n):n], minlength=v)
            states[1][at], states[2][at] = _words(fresh > 0), fresh.to(I32)
        return states
    out = s["logits"].double()
    k = case["k"]
    for r in range(rows):
        for i in range(k):
            x = out[r, i]
            if s["state"] is not None:
                at = int(s["slots"][r])
                count = s["state"][2][at].double()
                if i:
                    count = count + torch.bincount(s["drafted"][r, :i], minlength=v).double()
                seen = (count > 0) | _truths(s["state"][0][at], v)
                rep, freq, pres = (float(s[n][r]) for n in ("repetition", "frequency", "presence"))
                x[seen] = torch.where(x[seen] > 0, x[seen] / rep, x[seen] * rep)
                x -= freq * count + pres * (count > 0)
            if s["bias"] is not None:
                a, b = int(s["bias"][2][r]), int(s["bias"][2][r + 1])
                x[s["bias"][0][a:b]] += s["bias"][1][a:b].double()
            if s["allowed"] is not None:
                x[~_truths(s["allowed"][r, i], v)] = -math.inf
    return out
