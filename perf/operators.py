"""The training and head operators on the shapes they are used at.

Four operators around the draft-sampling loop:

- ``product``: the base logits of every draft position from bf16 hidden
  states and an E4M3 head with one scale for each block of 128 x 128 (the
  activations are quantized within the call, one scale per 128 values);
- ``quantize``: that head's E4M3 codes and scales from its bf16 weights;
- ``train``: a clipped policy loss with a KL term over drafted tokens, forward
  and backward: the tokens' log-probabilities under the corrected logits
  (base + w1[previous] . w2, output transform, temperature), the loss and its
  gradient, and the gradients of the base logits, w1 and w2;
- ``clip``: the norm over many gradients, and the clipped gradients.

The shapes are those of the five drafting workloads (4096 x 32 with 2 rows of
3 steps, 129280 x 256 with 1 and 16 rows of 5, 163840 x 256 with 64 rows of 5
and 256 rows of 8), with generic hidden sizes for the head.
"""

import math

import torch

own = False
DEV = "cuda"


# -- the cases ---------------------------------------------------------------------

def listed():
    return [
        # a handful of positions against a small head: the call's latency
        dict(name="product_tiny", op="product", rows=6, vocab=4096, hidden=512),
        # one request's block of 5 positions: the head streams past 5 tokens
        dict(name="product_single", op="product", rows=5, vocab=129280, hidden=7168),
        # 64 requests x 5 positions: a serving batch
        dict(name="product_large", op="product", rows=320, vocab=163840, hidden=4096),
        # 256 requests x 8 positions: the compute-bound end
        dict(name="product_stress", op="product", rows=2048, vocab=163840, hidden=4096),
        # a head whose vocabulary and hidden size both end inside a block
        dict(name="quantize_ragged", op="quantize", vocab=4104, hidden=1040),
        # a whole head, once when a model is loaded
        dict(name="quantize_head", op="quantize", vocab=163840, hidden=4096),
        # the smallest workload: the step's launches and latency
        dict(name="train_tiny", op="train", rows=2, k=3, vocab=4096, rank=32, softcap=0.0,
             masked=0.0, cold=0.0),
        # 16 requests x 5 positions: the tables dominate
        dict(name="train_small", op="train", rows=16, k=5, vocab=129280, rank=256, softcap=0.0,
             masked=0.0, cold=0.0),
        # 64 x 5 with the soft cap
        dict(name="train_large", op="train", rows=64, k=5, vocab=163840, rank=256, softcap=30.0,
             masked=0.0, cold=0.0),
        # 256 x 8, half of the rows drafted greedily, a quarter of each
        # vocabulary row masked out
        dict(name="train_stress", op="train", rows=256, k=8, vocab=163840, rank=256, softcap=0.0,
             masked=0.25, cold=0.5),
        # a few small gradients of both types: the call's latency
        dict(name="clip_tiny", op="clip", count=6, most=4097, types="mixed", max_norm=0.01),
        # gradients from one element to two tables' size, ragged, both types
        dict(name="clip_model", op="clip", count=40, most=41943040, types="mixed", max_norm=1.0),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["product", "quantize", "train", "train", "clip"])
    if op == "product":
        vocab = 8 * _log_uniform(rng, 512, 20480)
        hidden = 16 * _log_uniform(rng, 8, 448)
        most = min(2048, 2048 * 163840 * 4096 // (vocab * hidden))
        return dict(op=op, rows=_log_uniform(rng, 1, most), vocab=vocab, hidden=hidden)
    if op == "quantize":
        vocab = 8 * _log_uniform(rng, 1, 20480)
        return dict(op=op, vocab=vocab, hidden=16 * _log_uniform(rng, 1, 256))
    if op == "train":
        rank = rng.choice([16, 32, 64, 128, 256, 512])
        k = rng.randint(1, 8)
        return dict(op=op, rows=_log_uniform(rng, 1, 128 if rank == 512 else 256), k=k, vocab=8 * _log_uniform(rng, 512, 20480),
                    rank=rank, softcap=rng.choice([0.0, 15.0, 30.0]),
                    masked=rng.choice([0.0, 0.0, 0.25, 0.75]), cold=rng.choice([0.0, 0.5]))
    return dict(op=op, count=rng.randint(1, 40), most=_log_uniform(rng, 16, 41943040),
                types=rng.choice(["bf16", "fp32", "mixed"]), max_norm=rng.choice([0.25, 1.0, 1e6]))


def _blocks(n):
    return -(-n // 128)


def _clip_sizes(case):
    """Element counts from one to ``most``, spread over their logarithm."""
    n, most = case["count"], case["most"]
    sizes = [max(1, int(most ** (i / max(1, n - 1)))) for i in range(n)]
    sizes[-1] = most
    return sizes


def _clip_types(case):
    kinds = {"bf16": [torch.bfloat16], "fp32": [torch.float32],
             "mixed": [torch.bfloat16, torch.float32]}[case["types"]]
    return [kinds[(i + case["count"] - 1) % len(kinds)] for i in range(case["count"])]


def work(case):
    if case["op"] == "product":
        m, v, h = case["rows"], case["vocab"], case["hidden"]
        return {"bytes": 2 * m * h + v * h + 4 * _blocks(v) * _blocks(h) + 2 * m * v,
                "flops": 2 * m * v * h}
    if case["op"] == "quantize":
        v, h = case["vocab"], case["hidden"]
        return {"bytes": 3 * v * h + 4 * _blocks(v) * _blocks(h), "flops": 3 * v * h}
    if case["op"] == "train":
        m, v, r = case["rows"] * case["k"], case["vocab"], case["rank"]
        # base read and its gradient written, w2 and its gradient, w1's rows
        # and its whole gradient; three products and the softmax
        return {"bytes": 4 * m * v + 4 * v * r + 2 * v * r + 2 * m * r,
                "flops": 6 * m * v * r + 12 * m * v}
    total = sum(n * (2 if t == torch.bfloat16 else 4)
                for n, t in zip(_clip_sizes(case), _clip_types(case)))
    return {"bytes": 2 * total, "flops": 3 * sum(_clip_sizes(case))}


# -- the inputs --------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "product":
        m, v, h = case["rows"], case["vocab"], case["hidden"]
        x = normal(m, h)
        x[:, torch.randint(0, h, (max(1, h // 256),), generator=g, device=DEV)] *= 20.0  # outlier channels
        w, ws = _quantize(normal(v, h) * h ** -0.5, 128)
        s = dict(case=case, x=x.to(torch.bfloat16), w=w.view(torch.uint8), ws=ws,
                 out=torch.empty(m, v, dtype=torch.bfloat16, device=DEV))
        if own:
            import markov_draft_sampling_step_amd as m_

            s["space"] = m_.new_head_workspace(m, h)
        return s
    if case["op"] == "quantize":
        v, h = case["vocab"], case["hidden"]
        w = normal(v, h)
        w *= h ** -0.5
        return dict(case=case, w=w.to(torch.bfloat16),
                    q=torch.empty(v, h, dtype=torch.uint8, device=DEV),
                    qs=torch.empty(_blocks(v), _blocks(h), device=DEV))
    if case["op"] == "clip":
        grads = []
        for n, t in zip(_clip_sizes(case), _clip_types(case)):
            grads.append((normal(n) * 1e-3).to(t))
        s = dict(case=case, grads=grads, out=[torch.empty_like(x) for x in grads],
                 norm=torch.empty(1, device=DEV))
        if own:
            import markov_draft_sampling_step_amd as m_

            s["space"] = m_.new_clip_workspace(grads)
        return s
    rows, k, v, r = case["rows"], case["k"], case["vocab"], case["rank"]
    integers = lambda high, *shape: torch.randint(0, high, shape, generator=g, device=DEV)  # noqa: E731
    s = dict(case=case, w1=(normal(v, r) * 0.02).to(torch.bfloat16),
             w2=(normal(v, r) * 0.02).to(torch.bfloat16))
    base = normal(rows, k, v).mul_(3.0)
    if case["masked"]:
        base[torch.rand(rows, k, v, generator=g, device=DEV) < case["masked"]] = -math.inf
    s["tokens"] = integers(v, rows, k)
    # a drafted token had mass: its logit is one of the row's larger ones
    base.scatter_(2, s["tokens"][:, :, None], normal(rows, k, 1).abs() * 3.0 + 2.0)
    s["base"] = base.to(torch.bfloat16)
    del base
    s["prev"] = integers(v, rows)
    s["lengths"] = torch.where(torch.rand(rows, generator=g, device=DEV) < 0.25,
                               integers(k + 1, rows), torch.full((rows,), k, device=DEV)).to(torch.int32)
    if rows == 1:
        s["lengths"].fill_(k)
    s["temperature"] = torch.where(torch.rand(rows, generator=g, device=DEV) < case["cold"],
                                   0.0, 0.6 + 0.6 * torch.rand(rows, generator=g, device=DEV))
    # what the drafter gave when it drafted and what a reference gives: near
    # the present policy
    now = _score(s)[0]
    s["old"] = now + 0.2 * normal(rows, k)
    s["ref"] = now + 0.3 * normal(rows, k)
    s["advantages"] = normal(rows, k) + 0.25
    for name, shape in (("logprobs", (rows, k)), ("lse", (rows, k)), ("grad_logprobs", (rows, k)),
                        ("stats", (4,))):
        s[name] = torch.empty(*shape, device=DEV)
    for name, like in (("grad_base", "base"), ("grad_w1", "w1"), ("grad_w2", "w2")):
        s[name] = torch.empty_like(s[like])
    if own:
        import markov_draft_sampling_step_amd as m_

        s["space"] = m_.new_score_workspace(rows, v, r, k, softcap=case["softcap"])
    return s


CLIP_LOW, CLIP_HIGH, BETA = 0.2, 0.28, 0.05


# -- one pass ----------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import markov_draft_sampling_step_amd as m_

    case = s["case"]
    if case["op"] == "product":
        m_.head_logits_fp8(s["x"], s["w"], s["ws"], s["out"], s["space"])
        return s["out"]
    if case["op"] == "quantize":
        m_.quantize_head_fp8(s["w"], s["q"], s["qs"])
        return dict(codes=s["q"].view(torch.float8_e4m3fn), scales=s["qs"])
    if case["op"] == "clip":
        m_.clip_gradients(s["grads"], s["out"], case["max_norm"], s["norm"], s["space"])
        return dict(norm=s["norm"], grads=s["out"])
    m_.score_sequential(s["base"], s["w1"], s["w2"], s["prev"], s["tokens"], s["lengths"],
                        s["temperature"], s["logprobs"], s["lse"], s["space"],
                        softcap=case["softcap"])
    m_.policy_loss(s["logprobs"], s["old"], s["ref"], s["advantages"], s["tokens"], s["lengths"],
                   case["vocab"], s["stats"], s["grad_logprobs"], clip_low=CLIP_LOW,
                   clip_high=CLIP_HIGH, beta=BETA)
    m_.score_backward(s["base"], s["w1"], s["w2"], s["prev"], s["tokens"], s["lengths"],
                      s["temperature"], s["lse"], s["grad_logprobs"], s["grad_base"], s["grad_w1"],
                      s["grad_w2"], s["space"], softcap=case["softcap"])
    return {n: s[n] for n in ("logprobs", "lse", "stats", "grad_logprobs", "grad_base", "grad_w1",
                              "grad_w2")}


def _quantize(x, height):
    """E4M3 codes and the scales of blocks of ``height`` x 128, |block|max / 448."""
    x = x.float()
    n, h = x.shape
    tall, wide = -(-n // height), _blocks(h)
    pad = torch.zeros(tall * height, wide * 128, device=x.device)
    pad[:n, :h] = x
    pad = pad.view(tall, height, wide, 128)
    # a true quotient: by a plain number it would be a product with 1/448
    scales = pad.abs().amax((1, 3)) / torch.full((1, 1), 448.0, device=x.device)
    q = torch.where(scales[:, None, :, None] > 0, pad / scales[:, None, :, None], 0.0)
    codes = q.reshape(tall * height, wide * 128)[:n, :h].to(torch.float8_e4m3fn)
    return codes.contiguous(), scales


def _dequantize(codes, scales, height):
    n, h = codes.shape
    return codes.float() * scales.repeat_interleave(height, 0)[:n].repeat_interleave(128, 1)[:, :h]


def _embed(s):
    """The feeding token of each step (the previous one) and its w1 row."""
    fed = torch.cat([s["prev"][:, None], s["tokens"][:, :-1]], 1)
    return fed, s["w1"][fed].float()


def _valid(s):
    k = s["case"]["k"]
    return torch.arange(k, device=DEV)[None, :] < s["lengths"][:, None]


def _heat(s):
    return torch.where(s["temperature"] == 0, 1.0, s["temperature"])


def _score(s):
    """(log-probabilities, log-sum-exps, tempered logits, slope of the transform)."""
    rows, k, v = s["base"].shape
    cap = s["case"]["softcap"]
    _, emb = _embed(s)
    z = (emb.view(rows * k, -1) @ s["w2"].float().T).view(rows, k, v)
    z += s["base"]
    slope = None
    if cap > 0:
        z = torch.tanh(z / cap)
        slope = 1 - z * z
        z *= cap
    z /= _heat(s)[:, None, None]
    top = z.amax(2, keepdim=True)
    lse = top[:, :, 0] + torch.exp(z - top).sum(2).log()
    valid = _valid(s)
    logp = torch.where(valid, z.gather(2, s["tokens"][:, :, None])[:, :, 0] - lse, 0.0)
    return logp, torch.where(valid, lse, 0.0), z, slope


def _policy(s, logp):
    """The loss's parts and the gradient of the log-probabilities (64 bits inside)."""
    valid = _valid(s)
    n = valid.sum().clamp(min=1).double()
    ratio = torch.exp(logp.double() - s["old"])
    adv = s["advantages"].double()
    free, held = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    gap = s["ref"].double() - logp
    kl = torch.expm1(gap) - gap
    clipped = valid & (held < free)
    mean = lambda x: torch.where(valid, x, 0.0).sum() / n  # noqa: E731
    surrogate, kl_mean = mean(torch.minimum(free, held)), mean(kl)
    grad = (torch.where(clipped, 0.0, -free) - BETA * torch.expm1(gap)) / n
    stats = torch.stack([BETA * kl_mean - surrogate, surrogate, kl_mean, clipped.sum() / n])
    return stats.float(), torch.where(valid, grad, 0.0).float()


def _run_plain(s):
    case = s["case"]
    if case["op"] == "product":
        x = _dequantize(*_quantize(s["x"], 1), 1)
        w = _dequantize(s["w"].view(torch.float8_e4m3fn), s["ws"], 128)
        return (x @ w.T).to(torch.bfloat16)
    if case["op"] == "quantize":
        codes, scales = _quantize(s["w"], 128)
        return dict(codes=codes, scales=scales)
    if case["op"] == "clip":
        total = torch.stack([x.double().square().sum() for x in s["grads"]]).sum()
        norm = total.sqrt()
        by = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0).float()
        return dict(norm=norm.float().view(1), grads=[(x.float() * by).to(x.dtype) for x in s["grads"]])
    rows, k, v = s["base"].shape
    logp, lse, z, slope = _score(s)
    stats, grad = _policy(s, logp)
    d = torch.exp(z - lse[:, :, None]).neg_()
    del z
    d.scatter_add_(2, s["tokens"][:, :, None], torch.ones(rows, k, 1, device=DEV))
    d *= (grad / _heat(s)[:, None])[:, :, None]
    d = torch.where(_valid(s)[:, :, None], d, 0.0)
    if slope is not None:
        d *= slope
    fed, emb = _embed(s)
    flat = d.view(rows * k, v)
    grad_w2 = flat.T @ emb.view(rows * k, -1)
    grad_w1 = torch.zeros(s["w1"].shape, device=DEV)
    grad_w1.index_add_(0, fed.view(-1), flat @ s["w2"].float())
    return dict(logprobs=logp, lse=lse, stats=stats, grad_logprobs=grad,
                grad_base=d.to(torch.bfloat16), grad_w1=grad_w1.to(torch.bfloat16),
                grad_w2=grad_w2.to(torch.bfloat16))


# -- in 64 bits --------------------------------------------------------------------

def _nearest_e4m3(y):
    """The E4M3 value nearest to each binary64 value (ties to even)."""
    exponent = torch.frexp(y.abs().clamp(min=2.0 ** -9))[1] - 1
    step = torch.ldexp(torch.ones_like(y), exponent.clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _blocks64(x, height):
    """(scales, values of the codes) of blocks of ``height`` x 128 in 64 bits."""
    n, h = x.shape
    values, scales = torch.empty_like(x), []
    for j in range(0, h, 128):
        part = x[:, j:j + 128]
        top = part.abs().amax(1)
        if height > 1:
            top = torch.nn.functional.pad(top, (0, -n % height)).view(-1, height).amax(1)
        scale = (top / 448.0).float().double()   # a scale is a binary32 number
        scales.append(scale)
        of_row = scale.repeat_interleave(height)[:n, None]
        # a code is the nearest to the quotient as a binary32 number
        values[:, j:j + 128] = torch.where(of_row > 0, _nearest_e4m3((part / of_row).float().double()), 0.0)
    return torch.stack(scales, 1), values


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        scales, x = _blocks64(s["x"].double(), 1)
        out = torch.zeros(case["rows"], case["vocab"], dtype=torch.float64, device=DEV)
        for b, j in enumerate(range(0, case["hidden"], 128)):
            w = s["w"].view(torch.float8_e4m3fn)[:, j:j + 128].to(torch.float64)
            by = s["ws"][:, b].double().repeat_interleave(128)[:case["vocab"]]
            out += (x[:, j:j + 128] @ w.T) * scales[:, b, None] * by[None, :]
        return out
    if case["op"] == "quantize":
        scales, values = _blocks64(s["w"].double(), 128)
        return dict(codes=values, scales=scales)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float((x.double() ** 2).sum()) for x in s["grads"]))
        by = min(1.0, case["max_norm"] / (norm + 1e-6))
        return dict(norm=torch.tensor([norm], dtype=torch.float64),
                    grads=[x.double() * by for x in s["grads"]])
    rows, k, v = s["base"].shape
    base, w1, w2 = (s[n].double().requires_grad_(True) for n in ("base", "w1", "w2"))
    fed = torch.cat([s["prev"][:, None], s["tokens"][:, :-1]], 1).reshape(-1)
    logits = base.view(rows * k, v) + w1[fed] @ w2.T
    if case["softcap"] > 0:
        logits = torch.tanh(logits / case["softcap"]) * case["softcap"]
    heat = s["temperature"].double()
    heat = torch.where(heat == 0, torch.ones_like(heat), heat).repeat_interleave(k)
    logits = logits / heat[:, None]
    lse = torch.logsumexp(logits, 1)
    logp = (logits.gather(1, s["tokens"].view(-1, 1))[:, 0] - lse).view(rows, k)
    del logits
    logp.retain_grad()
    keep = torch.arange(k, device=DEV)[None, :] < s["lengths"][:, None]
    count = max(1, int(keep.sum()))
    kept = torch.masked_select(logp, keep)
    old, ref, adv = (torch.masked_select(s[n].double(), keep) for n in ("old", "ref", "advantages"))
    ratio = (kept - old).exp()
    held = torch.minimum(torch.maximum(ratio, torch.tensor(1 - CLIP_LOW, device=DEV, dtype=torch.float64)),
                         torch.tensor(1 + CLIP_HIGH, device=DEV, dtype=torch.float64))
    surrogate = torch.minimum(ratio * adv, held * adv).sum() / count
    kl = ((ref - kept).exp() - (ref - kept) - 1).sum() / count
    loss = BETA * kl - surrogate
    loss.backward()
    share = (held * adv < ratio * adv).sum() / count
    stats = torch.stack([loss.detach(), surrogate.detach(), kl.detach(), share.double()])
    return dict(logprobs=torch.where(keep, logp, 0.0).detach(),
                lse=torch.where(keep, lse.view(rows, k), 0.0).detach(), stats=stats,
                grad_logprobs=torch.where(keep, logp.grad, 0.0), grad_base=base.grad,
                grad_w1=w1.grad, grad_w2=w2.grad)
