"""The operators around the ZeRO-1 shard step, as a training program calls them, with their plain forms.

  muon_step     momentum, Newton-Schulz orthogonalisation and the fp32 master / bf16 weight update of a list of
                same-shaped matrices (the update Muon gives hidden matrices, beside AdamW for the others)
  ortho         the orthogonalisation alone
  embed         embedding lookup with scaling, and its gradient summed in fp32 by sorted tokens
  policy        clipped policy loss with a KL term over a logits matrix, loss and gradient
  preference    paired log-ratio preference loss over a logits matrix, loss and gradient

`own` False: elementary torch operations in fp32.  `own` True: the calls of mixed_precision_zero_amd.ops.
"""
import math

import numpy as np
import torch

own = False

NS_STEPS = 5
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
EPS = 1e-7
LR, WEIGHT_DECAY, MOMENTUM, CLIP = 3e-4, 0.1, 0.95, 1.0
BETA = 0.1                       # preference temperature
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # two small matrices of a toy model: a step of launches
        dict(name="muon_step_64x256", op="muon_step", batch=2, rows=64, cols=256),
        # the MLP matrices of eight layers of a 135M model
        dict(name="muon_step_8x1536x576", op="muon_step", batch=8, rows=1536, cols=576),
        # the attention matrices of one 1.7B layer
        dict(name="muon_step_4x2048x2048", op="muon_step", batch=4, rows=2048, cols=2048),
        # a tall matrix with odd sides
        dict(name="ortho_1x1537x333_f32", op="ortho", batch=1, rows=1537, cols=333, type="f32"),
        # one 7B MLP matrix, the largest
        dict(name="ortho_1x4096x11008_bf16", op="ortho", batch=1, rows=4096, cols=11008, type="bf16"),
        # a toy vocabulary and one short sequence
        dict(name="embed_33x64_v256_f32", op="embed", tokens=33, dim=64, vocab=256, type="f32", accumulate=False),
        # one micro-batch of a 135M model
        dict(name="embed_8192x576_v49152_bf16", op="embed", tokens=8192, dim=576, vocab=49152, type="bf16", accumulate=False),
        # a long micro-batch of a 1.7B model, summed onto the fp32 accumulator of earlier ones
        dict(name="embed_65536x2048_v49152_bf16_acc", op="embed", tokens=65536, dim=2048, vocab=49152, type="bf16", accumulate=True),
        # a toy vocabulary
        dict(name="policy_24x1000_f32", op="policy", tokens=24, vocab=1000, type="f32"),
        # one micro-batch over the 49152 vocabulary
        dict(name="policy_4096x49152_bf16", op="policy", tokens=4096, vocab=49152, type="bf16"),
        # three pairs of short answers, fp32 logits, a padded vocabulary of odd size
        dict(name="preference_3x77_v32001_f32", op="preference", pairs=3, length=77, vocab=32001, type="f32"),
        # eight pairs of long answers over the 32000 vocabulary
        dict(name="preference_8x512_v32000_bf16", op="preference", pairs=8, length=512, vocab=32000, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("muon_step", "ortho", "embed", "policy", "preference"))
    kind = rng.choice(("f32", "bf16", "f16"))
    if op in ("muon_step", "ortho"):
        rows, cols = _log(rng, 16, 8192), _log(rng, 16, 8192)
        if rng.random() < 0.5:               # the usual multiples
            rows, cols = -(-rows // 64) * 64, -(-cols // 64) * 64
        batch = _log(rng, 1, 16)
        while batch > 1 and batch * rows * cols * min(rows, cols) > 4096 * 4096 * 4096:
            batch -= 1
        while rows * cols * min(rows, cols) > 4096 * 4096 * 8192:
            rows, cols = rows // 2 + 1, cols // 2 + 1
        case = dict(op=op, batch=batch, rows=rows, cols=cols)
        if op == "ortho":
            case["type"] = rng.choice(("f32", "bf16"))
        return case
    if op == "embed":
        vocab, dim, tokens = _log(rng, 200, 60000), _log(rng, 16, 4096), _log(rng, 1, 65536)
        if rng.random() < 0.6:
            dim = -(-dim // 64) * 64
        while vocab * dim > 49152 * 2048 or tokens * dim > 65536 * 2048:
            dim = dim // 2 + 1
        return dict(op=op, tokens=tokens, dim=dim, vocab=vocab, type=kind, accumulate=rng.random() < 0.5)
    vocab = _log(rng, 200, 60000)
    if rng.random() < 0.6:
        vocab = -(-vocab // 64) * 64
    if op == "policy":
        tokens = min(_log(rng, 1, 8192), 4096 * 49152 // (vocab * (BYTES[kind] // 2)))
        return dict(op=op, tokens=tokens, vocab=vocab, type=kind)
    pairs, length = _log(rng, 1, 32), _log(rng, 1, 1024)
    length = max(1, min(length, 8 * 512 * 32000 // (pairs * vocab * (BYTES[kind] // 2))))
    return dict(op=op, pairs=pairs, length=length, vocab=vocab, type=kind)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _gradient(g, b, m, n):
    """Matrices with the spectrum of a gradient: a few strong directions over a broad floor."""
    r = min(8, m, n)
    x = torch.randn(b, m, n, generator=g, device="cuda")
    u = torch.randn(b, m, r, generator=g, device="cuda")
    v = torch.randn(b, r, n, generator=g, device="cuda")
    return (x + torch.bmm(u, v)) * 1e-3


def _rank(tokens, vocab, g):
    """Token ids with the skew of text: id = floor(V u^3)."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    return (u * u * u * vocab).long().clamp_(max=vocab - 1)


def _logits(g, n, vocab, kind):
    x = torch.empty(n, vocab, device="cuda", dtype=TYPES[kind])
    for at in range(0, n, 1024):
        k = min(1024, n - at)
        x[at:at + k] = torch.randn(k, vocab, generator=g, device="cuda") * 2.0
    return x


def _logp_of(x, y):
    """log-probability of the targets in fp32, in pieces (negative targets: that of id 0)."""
    out = torch.empty(x.shape[0], device="cuda")
    for at in range(0, x.shape[0], 1024):
        z = x[at:at + 1024].float()
        out[at:at + 1024] = z.gather(1, y[at:at + 1024].clamp(min=0)[:, None])[:, 0] - z.logsumexp(1)
    return out


def _loss_scale(case):
    """fp16 gradients are trained with a scaled loss, so that they do not underflow."""
    return 4096.0 if case["type"] == "f16" else 1.0


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("muon_step", "ortho"):
        b, m, n = case["batch"], case["rows"], case["cols"]
        grad = _gradient(g, b, m, n)
        if op == "ortho":
            s["grad"] = grad.to(TYPES[case["type"]])
            s["ortho"] = torch.empty(b, m, n, device="cuda", dtype=torch.bfloat16)
            if own:
                from mixed_precision_zero_amd import ops
                s["plan"] = ops.z1_muon_create([(m, n)] * b, list(s["grad"].unbind(0)), ortho=list(s["ortho"].unbind(0)),
                                               ns_steps=NS_STEPS, coeffs=(NS_A, NS_B, NS_C), eps=EPS)
            return s
        s["grad"] = grad
        s["momentum"] = _gradient(g, b, m, n) * 4.0
        s["master"] = torch.randn(b, m, n, generator=g, device="cuda") * 0.02
        s["weights"] = s["master"].to(torch.bfloat16)
        s["S"] = grad.double().square().sum().reshape(1)
        s["lr_scale"] = 0.2 * math.sqrt(max(m, n))
        if own:
            from mixed_precision_zero_amd import ops
            parts = {k: list(s[k].unbind(0)) for k in ("momentum", "master", "weights")}
            s["plan"] = ops.z1_muon_create([(m, n)] * b, list(grad.unbind(0)), **parts, lr_scale=[s["lr_scale"]] * b,
                                           ns_steps=NS_STEPS, coeffs=(NS_A, NS_B, NS_C), eps=EPS)
        return s
    t = TYPES[case["type"]]
    if op == "embed":
        n, d, v = case["tokens"], case["dim"], case["vocab"]
        s["weight"] = (torch.randn(v, d, generator=g, device="cuda") * 0.02).to(t)
        s["ids"] = _rank(n, v, g)
        if n > 8:
            s["ids"][torch.rand(n, generator=g, device="cuda") < 0.03] = -1      # padding
        s["dout"] = (torch.randn(n, d, generator=g, device="cuda") * 1e-3).to(t)
        s["scale"] = math.sqrt(d)
        s["out"] = torch.empty(n, d, device="cuda", dtype=t)
        s["dweight"] = torch.randn(v, d, generator=g, device="cuda") * 1e-2 if case["accumulate"] else torch.empty(v, d, device="cuda")
        if own:
            from mixed_precision_zero_amd import ops
            s["workspace"] = torch.empty(ops.z1_embed_grad_workspace(n, v, d), device="cuda", dtype=torch.uint8)
        return s
    v = case["vocab"]
    if op == "policy":
        n = case["tokens"]
    else:
        # answers of unequal length, one after another: chosen, rejected, chosen, ...
        mean = -(-3 * case["length"] // 4)
        cuts = torch.arange(2 * case["pairs"] + 1, device="cuda") * mean
        cuts[1:-1] += torch.randint(-(mean // 4), mean // 4 + 1, (2 * case["pairs"] - 1,), generator=g, device="cuda")
        s["cu_seqlens"] = cuts
        n = int(s["cu_seqlens"][-1])
    x = s["logits"] = _logits(g, n, v, case["type"])
    y = _rank(n, v, g)
    y[torch.rand(n, generator=g, device="cuda") < 0.1] = -100                   # prompt tokens
    s["targets"] = y
    s["dlogits"] = torch.empty_like(x)
    now = _logp_of(x, y)
    noise = lambda w: w * torch.randn(n, generator=g, device="cuda")  # noqa: E731
    f = dict(device="cuda", dtype=torch.float32)
    s["logp"], s["lse"], s["loss"] = torch.empty(n, **f), torch.empty(n, **f), torch.empty(1, **f)
    if op == "policy":
        s["ref_logp"], s["old_logp"] = now + noise(0.2), now + noise(0.2)
        s["advantages"] = torch.randn(n, generator=g, device="cuda") + 0.5
        s["scale"] = _loss_scale(case) / n
        s["token_loss"] = torch.empty(n, **f)
    else:
        # a policy that has moved towards the chosen answers
        which = torch.searchsorted(cuts[1:].contiguous(), torch.arange(n, device="cuda"), right=True)
        s["ref_logp"] = now - min(0.3, 15.0 / mean) * (1.0 - 2.0 * (which % 2)) + noise(0.2)
        s["dlogp"] = torch.empty(n, **f)
        s["pair_loss"], s["margins"] = torch.empty(case["pairs"], **f), torch.empty(case["pairs"], **f)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    return {"muon_step": _muon_step, "ortho": _ortho, "embed": _embed, "policy": _policy, "preference": _preference}[s["case"]["op"]](s)


def _newton_schulz(u):
    x = u.float()
    x = x.mT.contiguous() if u.shape[1] > u.shape[2] else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + EPS).float()
    for _ in range(NS_STEPS):
        a = torch.matmul(x, x.mT.contiguous())
        x = NS_A * x + torch.matmul(NS_B * a + NS_C * torch.matmul(a, a), x)
    return x.mT if u.shape[1] > u.shape[2] else x


def _ortho(s):
    if own:
        from mixed_precision_zero_amd import ops
        ops.z1_muon_orthogonalize(s["plan"])
        return dict(ortho=s["ortho"])
    s["ortho"].copy_(_newton_schulz(s["grad"]))
    return dict(ortho=s["ortho"])


def _muon_step(s):
    if own:
        from mixed_precision_zero_amd import ops
        ops.z1_muon_step(s["plan"], lr=LR, momentum=MOMENTUM, weight_decay=WEIGHT_DECAY, nesterov=True, clip=CLIP, d_S=s["S"])
    else:
        c = (CLIP / (s["S"].sqrt() + 1e-6)).clamp(max=1.0).float()
        grad = c * s["grad"]
        s["momentum"].mul_(MOMENTUM).add_(grad)
        o = _newton_schulz(grad + MOMENTUM * s["momentum"])
        s["master"].mul_(1.0 - LR * WEIGHT_DECAY).sub_((LR * s["lr_scale"]) * o)
        s["weights"].copy_(s["master"])
    return dict(momentum=s["momentum"], master=s["master"], weights=s["weights"])


def _embed(s):
    if own:
        from mixed_precision_zero_amd import ops
        ops.z1_embed_lookup(s["weight"], s["ids"], s["out"], scale=s["scale"])
        ops.z1_embed_grad(s["ids"], s["dout"], s["dweight"], scale=s["scale"], accumulate=s["case"]["accumulate"], workspace=s["workspace"])
        return dict(out=s["out"], dweight=s["dweight"])
    here = s["ids"] >= 0
    at = s["ids"].clamp(min=0)
    s["out"].copy_(s["weight"][at].float() * s["scale"] * here[:, None])
    if not s["case"]["accumulate"]:
        s["dweight"].zero_()
    s["dweight"].index_add_(0, at, s["dout"].float() * s["scale"] * here[:, None])
    return dict(out=s["out"], dweight=s["dweight"])


def _log_softmax(s):
    """fp32 shifted logits, their logsumexp, the targets' log-probabilities and the mask of rows that count."""
    z = s["logits"].float()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    here = s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    logp = torch.where(here, (z.gather(1, at) - top - torch.log(total))[:, 0], torch.zeros_like(top[:, 0]))
    return e, total, logp, here, at


def _dlogits(s, e, total, at, d):
    """d of each row's log-probability, through log-softmax, in the logits' type."""
    p = e.mul_((-d[:, None]) / total)
    p.scatter_add_(1, at, d[:, None])
    s["dlogits"].copy_(p)


def _policy(s):
    if own:
        from mixed_precision_zero_amd import ops
        ops.z1_policy_loss(s["logits"], s["targets"], s["old_logp"], s["advantages"], ref_logp=s["ref_logp"], clip_low=CLIP_LOW,
                           clip_high=CLIP_HIGH, kl_coef=KL, scale=s["scale"], loss=s["loss"], token_loss=s["token_loss"],
                           logp=s["logp"], dlogits=s["dlogits"])
        return {k: s[k] for k in ("loss", "token_loss", "logp", "dlogits")}
    e, total, logp, here, at = _log_softmax(s)
    ratio = torch.exp(logp - s["old_logp"])
    adv = s["advantages"]
    near = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    gap = s["ref_logp"] - logp
    token = torch.maximum(-ratio * adv, -near * adv) + KL * (torch.expm1(gap) - gap)
    token = torch.where(here, token, torch.zeros_like(token))
    through = (ratio == near) | (ratio * adv < near * adv)
    d = torch.where(through, -ratio * adv, torch.zeros_like(adv)) - KL * torch.expm1(gap)
    _dlogits(s, e, total, at, torch.where(here, d * s["scale"], torch.zeros_like(d)))
    loss = (token.double().sum() * s["scale"]).float().reshape(1)
    return dict(loss=loss, token_loss=token, logp=logp, dlogits=s["dlogits"])


def _preference(s):
    scale = _loss_scale(s["case"]) / s["case"]["pairs"]
    if own:
        from mixed_precision_zero_amd import ops
        ops.z1_token_logprob(s["logits"], s["targets"], s["logp"], s["lse"])
        ops.z1_preference_loss(s["logp"], s["ref_logp"], s["targets"], s["cu_seqlens"], beta=BETA, scale=scale, loss=s["loss"],
                               pair_loss=s["pair_loss"], margins=s["margins"], dlogp=s["dlogp"])
        ops.z1_logprob_grad(s["logits"], s["targets"], s["lse"], s["dlogp"], s["dlogits"])
        return {k: s[k] for k in ("loss", "pair_loss", "margins", "dlogits")}
    e, total, logp, here, at = _log_softmax(s)
    cu = s["cu_seqlens"]
    diff = torch.where(here, logp - s["ref_logp"], torch.zeros_like(logp)).double()
    run_sum = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), diff.cumsum(0)])
    sums = run_sum[cu[1:]] - run_sum[cu[:-1]]
    margins = BETA * (sums[0::2] - sums[1::2])
    pair = torch.log1p(torch.exp(-margins.abs())) + (-margins).clamp(min=0)
    dm = -scale * BETA / (1.0 + torch.exp(margins))
    which = torch.searchsorted(cu[1:].contiguous(), torch.arange(logp.numel(), device="cuda"), right=True)
    sign = 1.0 - 2.0 * (which % 2).double()
    d = torch.where(here, (dm[which // 2] * sign).float(), torch.zeros_like(logp))
    _dlogits(s, e, total, at, d)
    return dict(loss=(pair.sum() * scale).float().reshape(1), pair_loss=pair.float(), margins=margins.float(), dlogits=s["dlogits"])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _distinct(tokens, vocab):
    """Expected number of different ids among `tokens` draws of floor(V u^3)."""
    edge = (np.arange(vocab + 1) / vocab) ** (1.0 / 3.0)
    return float((1.0 - (1.0 - np.diff(edge)) ** tokens).sum())


def work(case):
    op = case["op"]
    if op in ("muon_step", "ortho"):
        b, m, n = case["batch"], case["rows"], case["cols"]
        k, w = min(m, n), max(m, n)
        # X X^T and its square are symmetric: half of each is enough
        flops = b * NS_STEPS * (3.0 * k * k * w + 1.0 * k * k * k)
        each = 22 if op == "muon_step" else BYTES[case["type"]] + 2
        return dict(bytes=b * m * n * each, flops=flops)
    e = BYTES[case["type"]]
    if op == "embed":
        t, d, v = case["tokens"], case["dim"], case["vocab"]
        rows = _distinct(t, v)
        dw = 8 * rows * d if case["accumulate"] else 4 * v * d
        return dict(bytes=16 * t + 2 * t * d * e + rows * d * e + dw, flops=3.0 * t * d)
    v = case["vocab"]
    n = case["tokens"] if op == "policy" else 2 * case["pairs"] * -(-3 * case["length"] // 4)
    return dict(bytes=n * v * e * 2.0 + 30 * n, flops=8.0 * n * v)


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def _exact_orthogonal(u):
    """q = p(p(...p(u / |u|))) with p(x) = a x + b (x x') x + c (x x')^2 x, one matrix at a time."""
    out = torch.empty_like(u)
    for i in range(u.shape[0]):
        flip = u.shape[1] > u.shape[2]
        x = u[i].t().contiguous() if flip else u[i].clone()
        x /= x.norm() + EPS
        for _ in range(NS_STEPS):
            gram = x @ x.t()
            y = gram @ x
            x = NS_A * x + NS_B * y + NS_C * (gram @ y)
        out[i] = x.t() if flip else x
    return out


def _exact_rows(x, y):
    """Log-probabilities of the targets (0 where there is none), from the definition."""
    logz = torch.stack([torch.logsumexp(x[i:i + 512].double(), 1) if i + 512 <= x.shape[0] else
                        torch.nn.functional.pad(torch.logsumexp(x[i:].double(), 1), (0, i + 512 - x.shape[0]))
                        for i in range(0, x.shape[0], 512)]).reshape(-1)[:x.shape[0]]
    at = torch.arange(x.shape[0], device=x.device)
    logp = x[at, y.clamp(min=0)].double() - logz
    return torch.where(y >= 0, logp, torch.zeros_like(logp)), logz


def _exact_dlogits(x, y, logz, d):
    """d_r (1[v = y_r] - p_rv)"""
    g = torch.empty(x.shape, device=x.device, dtype=torch.float64)
    for i in range(0, x.shape[0], 512):
        g[i:i + 512] = -d[i:i + 512, None] * torch.exp(x[i:i + 512].double() - logz[i:i + 512, None])
    at = torch.arange(x.shape[0], device=x.device)
    g[at, y.clamp(min=0)] += d
    return g


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "ortho":
        return dict(ortho=_exact_orthogonal(s["grad"].double()))
    if op == "muon_step":
        c = min(1.0, CLIP / (math.sqrt(float(s["S"])) + 1e-6))
        grad = s["grad"].double() * c
        mom = MOMENTUM * s["momentum"].double() + grad
        q = _exact_orthogonal(grad + MOMENTUM * mom)
        master = s["master"].double() * (1.0 - LR * WEIGHT_DECAY) - LR * s["lr_scale"] * q
        return dict(momentum=mom, master=master, weights=master)
    if op == "embed":
        keep = s["ids"] >= 0
        out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        out[keep] = s["weight"].double()[s["ids"][keep]] * s["scale"]
        dw = s["dweight"].double() if case["accumulate"] else torch.zeros(s["dweight"].shape, device="cuda", dtype=torch.float64)
        order = torch.argsort(s["ids"][keep], stable=True)
        dw.index_put_((s["ids"][keep][order],), s["dout"][keep][order].double() * s["scale"], accumulate=True)
        return dict(out=out, dweight=dw)
    x, y = s["logits"], s["targets"]
    logp, logz = _exact_rows(x, y)
    if op == "policy":
        adv, scale = s["advantages"].double(), s["scale"]
        ratio = torch.exp(logp - s["old_logp"].double())
        inside = (ratio >= 1.0 - CLIP_LOW) & (ratio <= 1.0 + CLIP_HIGH)
        lower = torch.minimum(ratio * adv, ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv)
        gap = s["ref_logp"].double() - logp
        token = (-lower + KL * (torch.expm1(gap) - gap)) * (y >= 0)
        moves = inside | (ratio * adv <= lower)
        d = (-(ratio * adv) * moves - KL * torch.expm1(gap)) * scale * (y >= 0)
        return dict(loss=(token.sum() * scale).reshape(1), token_loss=token, logp=logp, dlogits=_exact_dlogits(x, y, logz, d))
    cu = s["cu_seqlens"].tolist()
    scale, pair, margins, d = _loss_scale(case) / case["pairs"], [], [], torch.zeros_like(logp)
    diff = (logp - s["ref_logp"].double()) * (y >= 0)
    for p in range(case["pairs"]):
        a, b, c = cu[2 * p], cu[2 * p + 1], cu[2 * p + 2]
        z = BETA * (diff[a:b].sum() - diff[b:c].sum())
        margins.append(z)
        pair.append(-torch.nn.functional.logsigmoid(z))
        slope = -BETA * scale * torch.sigmoid(-z)
        d[a:b], d[b:c] = slope, -slope
    d = d * (y >= 0)
    pair, margins = torch.stack(pair), torch.stack(margins)
    return dict(loss=(pair.sum() * scale).reshape(1), pair_loss=pair, margins=margins, dlogits=_exact_dlogits(x, y, logz, d))
