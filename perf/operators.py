"""The operators that score sampled tokens and learn from them, as measured cases.

Four operators over decoder logits [rows, V] (row = one canvas position) and
the tokens that the sampler committed there:

  logprobs    log-probability of each row's token and entropy of the tempered
              softmax; direction "back": the gradient of both for the logits
  policy      clipped policy loss with a KL term and an entropy bonus, with
              the gradient for the logits
  preference  preference loss over pairs of sequences (paired log ratios),
              with the gradient for the logits
  lmhead      log-probability and entropy from hidden states and the LM head

Each is there twice: in elementary torch operations, and (`own`) as the calls
of this package.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

CLIP_LOW, CLIP_HIGH = 0.2, 0.28
KL_COEF, ENTROPY_COEF = 0.04, 0.01
BETA, SMOOTHING, MARGIN = 0.1, 0.05, 0.02


def listed():
    return [
        # the tiny sampler configuration: one canvas of 16 positions, latency only
        {"name": "logprobs_tiny", "op": "logprobs", "dir": "forward", "rows": 16, "V": 1024,
         "dtype": "f32", "ignored": 0, "banned": 0, "row_temps": False},
        # one canvas of the model card's shape, scored once
        {"name": "logprobs_canvas", "op": "logprobs", "dir": "forward", "rows": 256, "V": 262144,
         "dtype": "bf16", "ignored": 0, "banned": 0, "row_temps": False},
        # the same canvas, gradients of a caller's own loss coming back
        {"name": "logprobs_back_canvas", "op": "logprobs", "dir": "back", "rows": 256, "V": 262144,
         "dtype": "bf16", "ignored": 16, "banned": 0, "row_temps": False},
        # a policy step on the tiny configuration
        {"name": "policy_tiny", "op": "policy", "rows": 16, "V": 1024, "dtype": "f32",
         "ignored": 1, "banned": 0, "row_temps": False},
        # fp32 logits of an odd vocabulary, some ids banned with -inf, an odd number of rows
        {"name": "policy_ragged", "op": "policy", "rows": 1111, "V": 32003, "dtype": "f32",
         "ignored": 111, "banned": 500, "row_temps": True},
        # a policy step on one canvas
        {"name": "policy_canvas", "op": "policy", "rows": 256, "V": 262144, "dtype": "bf16",
         "ignored": 0, "banned": 0, "row_temps": False},
        # the small-batch serving shape, eight canvases, committed at different steps
        {"name": "policy_batch", "op": "policy", "rows": 2048, "V": 262144, "dtype": "bf16",
         "ignored": 128, "banned": 0, "row_temps": True},
        # three short answer pairs of a small vocabulary
        {"name": "preference_short", "op": "preference", "pairs": 3, "length": 40, "V": 32000,
         "dtype": "bf16", "ignored": 5, "banned": 0, "average": False},
        # four pairs of canvases of ragged lengths
        {"name": "preference_canvas", "op": "preference", "pairs": 4, "length": 256, "V": 262144,
         "dtype": "bf16", "ignored": 40, "banned": 0, "average": False},
        # a few positions scored from hidden states (the weight's bytes bound it)
        {"name": "lmhead_few", "op": "lmhead", "rows": 24, "V": 262144, "d": 2560},
        # one canvas scored from hidden states
        {"name": "lmhead_canvas", "op": "lmhead", "rows": 256, "V": 262144, "d": 2560},
        # eight canvases scored from hidden states
        {"name": "lmhead_batch", "op": "lmhead", "rows": 2048, "V": 262144, "d": 2560},
    ]


def _between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "policy", "policy", "preference", "lmhead"])
    if op == "lmhead":
        d = 8 * _between(rng, 8, 512)
        V = _between(rng, 1000, 262144)
        if rng.random() < 0.5:
            V -= V % 256
        return {"op": op, "rows": _between(rng, 1, 2048), "V": V, "d": min(d, 2560)}
    V = _between(rng, 1000, 262144)
    if rng.random() < 0.5:
        V -= V % 64
    dtype = rng.choice(["bf16", "f32"])
    most = min(4096, 2048 * 262144 // V // (2 if dtype == "f32" else 1))
    case = {"op": op, "V": V, "dtype": dtype, "banned": rng.choice([0, 0, 1, V // 10])}
    if op == "preference":
        case["pairs"] = _between(rng, 1, 16)
        case["length"] = _between(rng, 1, max(2, min(512, most // (2 * case["pairs"]))))
        case["ignored"] = rng.choice([0, case["length"] // 3])
        case["average"] = rng.random() < 0.3
        return case
    case["rows"] = _between(rng, 1, most)
    case["ignored"] = rng.choice([0, case["rows"] // 8])
    case["row_temps"] = rng.random() < 0.5
    if op == "logprobs":
        case["dir"] = rng.choice(["forward", "back"])
    return case


def _lengths(case):
    """Row counts of the 2 * pairs sequences: ragged, `length` the longest."""
    n, most = 2 * case["pairs"], case["length"]
    return [most - (i * 37 + i * i * 11) % max(1, most // 2 + 1) for i in range(n)]


def _rows(case):
    return sum(_lengths(case)) if case["op"] == "preference" else case["rows"]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    rows, V = _rows(case), case["V"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def integers(hi, n):
        return torch.randint(0, hi, (n,), generator=g, device=dev)

    s = {"case": case, "temperature": 0.7}
    if case["op"] == "lmhead":
        d = case["d"]
        weight = torch.empty((V, d), dtype=torch.bfloat16, device=dev)
        weight.normal_(0.0, 2.0 / math.sqrt(d), generator=g)
        tokens = integers(V, rows)
        # confident rows point along their token's row of the head
        pull = torch.where(uniform(rows) < 0.5, 3.0, 0.5)
        hidden = normal(rows, d) + pull[:, None] * weight[tokens].float()
        s |= {"hidden": hidden.to(torch.bfloat16), "weight": weight,
              "tokens": tokens.to(torch.int32)}
        return s

    # N(0, 1) logits with one boosted id per row, as a decoder's canvas has
    # them: a confident part of the rows, an open part
    logits = torch.empty((rows, V), dtype=torch.bfloat16 if case["dtype"] == "bf16"
                         else torch.float32, device=dev)
    logits.normal_(generator=g)
    top = integers(V, rows)
    boost = torch.where(uniform(rows) < 0.5, 12.0 + 8.0 * uniform(rows), 4.0 * uniform(rows))
    at = torch.arange(rows, device=dev)
    logits[at, top] += boost.to(logits.dtype)
    tokens = torch.where(uniform(rows) < 0.8, top, integers(V, rows))
    if case["banned"]:
        kept = logits[at, tokens], logits[at, top]
        logits[:, integers(V, case["banned"])] = -math.inf
        logits[at, tokens], logits[at, top] = kept
    if case.get("row_temps"):
        s["temperature"] = 0.8 - 0.4 * torch.floor(48.0 * uniform(rows)) / 47.0
    temp = s["temperature"]
    # what the policy gave these tokens when they were drawn, and a reference model
    each = temp if torch.is_tensor(temp) else torch.full((rows,), temp, device=dev)
    lse = torch.cat([torch.logsumexp(c.float() / t[:, None], 1)
                     for c, t in zip(logits.split(512), each.split(512))])
    now = logits[at, tokens].float() / each - lse
    tokens = tokens.to(torch.int32)
    if case["ignored"]:
        tokens[torch.randperm(rows, generator=g, device=dev)[:case["ignored"]]] = -1
    s |= {"logits": logits, "tokens": tokens}
    if case["op"] == "logprobs":
        if case["dir"] == "back":
            s |= {"d_logprobs": normal(rows) / rows, "d_entropies": 0.1 * normal(rows) / rows}
    elif case["op"] == "policy":
        s |= {"old": now + 0.15 * normal(rows), "ref": now + 0.3 * normal(rows),
              "advantages": normal(rows), "weights": 0.5 + uniform(rows), "scale": 1.0 / rows}
    else:
        lengths = torch.tensor(_lengths(case))
        offsets = torch.zeros(len(lengths) + 1, dtype=torch.int32)
        offsets[1:] = torch.cumsum(lengths, 0)
        seq = torch.repeat_interleave(torch.arange(len(lengths)), lengths).to(dev)
        kept = torch.where(tokens >= 0, now + 0.1 * normal(rows), torch.zeros_like(now))
        ref = torch.zeros(len(lengths), dtype=torch.float64, device=dev)
        ref.index_add_(0, seq, kept.double())
        if case["average"]:
            n = torch.zeros_like(ref).index_add_(0, seq, (tokens >= 0).double())
            ref = ref / n.clamp(min=1.0)
        s |= {"offsets": offsets.to(dev), "ref": ref.float(), "scale": 1.0 / case["pairs"]}
    return s


# -- the operators in elementary torch operations ------------------------------


def _softmax_rows(z, temperature, tokens):
    """y = z / T, softmax p, log-partition, log p of the token, entropy (rows of fp32)."""
    t = temperature[:, None] if torch.is_tensor(temperature) else temperature
    y = z.float() / t
    m = y.max(1, keepdim=True).values
    e = torch.exp(y - m)
    total = e.double().sum(1, keepdim=True)
    p = e / total.float()
    shift = torch.log(total)
    a = tokens.clamp(min=0).long()[:, None]
    lp = (y.gather(1, a).double() - m.double() - shift)[:, 0]
    logp = (y - m) - shift.float()
    h = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    keep = tokens >= 0
    zero = torch.zeros_like(h)
    return p, logp, a, torch.where(keep, lp, zero.double()), torch.where(keep, h, zero), keep


def _logit_gradient(p, logp, a, h, keep, g_lp, g_h, temperature, dtype):
    """T^-1 [g_lp (onehot - p) - g_h p (log p + H)], zero in the ignored rows."""
    t = temperature[:, None] if torch.is_tensor(temperature) else temperature
    d = -g_lp[:, None] * p
    if g_h is not None:
        d -= g_h[:, None] * torch.where(p > 0, p * (logp + h[:, None]), torch.zeros_like(p))
    # the token's own p is near 1 in a confident row: 1 - p there by expm1 of log p
    own_p = -torch.expm1(logp.gather(1, a).clamp(max=0.0))
    at = g_lp[:, None] * own_p
    if g_h is not None:
        at -= g_h[:, None] * (p * (logp + h[:, None])).gather(1, a).nan_to_num()
    d.scatter_(1, a, at)
    return torch.where(keep[:, None], d / t, torch.zeros_like(d)).to(dtype)


def _plain_logprobs(s):
    z, temp = s["logits"], s["temperature"]
    p, logp, a, lp, h, keep = _softmax_rows(z, temp, s["tokens"])
    if s["case"]["dir"] == "forward":
        return {"logprobs": lp.float(), "entropies": h}
    return {"d_logits": _logit_gradient(p, logp, a, h, keep, s["d_logprobs"], s["d_entropies"],
                                        temp, z.dtype)}


def _plain_policy(s):
    z, temp, scale = s["logits"], s["temperature"], s["scale"]
    p, logp, a, lp, h, keep = _softmax_rows(z, temp, s["tokens"])
    w = torch.where(keep, s["weights"], torch.zeros_like(s["weights"])).double() * scale
    adv = s["advantages"].double()
    ratio = torch.exp(lp - s["old"].double())
    free = -adv * ratio
    held = -adv * ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    back = torch.exp(s["ref"].double() - lp)
    kl = back - 1.0 - (s["ref"].double() - lp)
    pg = torch.maximum(free, held)
    g_lp = w * (torch.where(free >= held, free, torch.zeros_like(free)) + KL_COEF * (1.0 - back))
    g_h = -w * ENTROPY_COEF
    parts = [(w * pg).sum(), (w * kl).sum(), (w * h.double()).sum(),
             (w * (held > free).double()).sum()]
    terms = torch.stack([parts[0] + KL_COEF * parts[1] - ENTROPY_COEF * parts[2]] + parts).float()
    return {"terms": terms, "logprobs": lp.float(), "entropies": h,
            "d_logits": _logit_gradient(p, logp, a, h, keep, g_lp.float(), g_h.float(), temp,
                                        z.dtype)}


def _plain_preference(s):
    z, temp, scale, off = s["logits"], s["temperature"], s["scale"], s["offsets"].long()
    p, logp, a, lp, h, keep = _softmax_rows(z, temp, s["tokens"])
    n = off.numel() - 1
    seq = torch.bucketize(torch.arange(z.shape[0], device=z.device), off[1:], right=True)
    total = torch.zeros(n, dtype=torch.float64, device=z.device).index_add_(0, seq, lp)
    share = torch.ones_like(total)
    if s["case"]["average"]:
        count = torch.zeros_like(total).index_add_(0, seq, keep.double())
        share = 1.0 / count.clamp(min=1.0)
    total = total * share
    gap = total - s["ref"].double()
    margin = BETA * (gap[: n // 2] - gap[n // 2:]) - MARGIN
    soft = torch.log1p(torch.exp(-margin.abs()))
    losses = (1.0 - SMOOTHING) * (soft + (-margin).clamp(min=0.0)) \
        + SMOOTHING * (soft + margin.clamp(min=0.0))
    d = (SMOOTHING - 1.0) / (1.0 + torch.exp(margin)) + SMOOTHING / (1.0 + torch.exp(-margin))
    g = scale * BETA * torch.cat([d, -d]) * share
    return {"loss": (scale * losses.sum()).float().reshape(1), "losses": losses.float(),
            "sequence_logprobs": total.float(), "logprobs": lp.float(),
            "d_logits": _logit_gradient(p, logp, a, h, keep, g[seq].float(), None, temp, z.dtype)}


def _plain_lmhead(s):
    z = s["hidden"].float() @ s["weight"].float().T
    _, _, _, lp, h, _ = _softmax_rows(z, s["temperature"], s["tokens"])
    return {"logprobs": lp.float(), "entropies": h}


# -- the same as calls of this package ------------------------------------------

_scorers = {}


def _scorer(rows, device):
    """The program's scorer: one handle, made at the first call that needs it."""
    from entropy_bound_canvas_b200 import EBScorer

    held = _scorers.get(device)
    if held is None or held.max_rows < rows:
        held = _scorers[device] = EBScorer(max(rows, 8192), device=device)
    return held


def _own_run(s):
    case, tokens = s["case"], s["tokens"]
    sc = _scorer(tokens.shape[0], tokens.device)
    if case["op"] == "lmhead":
        r = sc.lmhead_logprobs(s["hidden"], s["weight"], tokens, temperature=s["temperature"])
        return {"logprobs": r.logprobs, "entropies": r.entropies}
    if case["op"] == "logprobs":
        if case["dir"] == "forward":
            r = sc.token_logprobs(s["logits"], tokens, temperature=s["temperature"])
            return {"logprobs": r.logprobs, "entropies": r.entropies}
        return {"d_logits": sc.token_logprobs_backward(
            s["logits"], tokens, s["d_logprobs"], s["d_entropies"], temperature=s["temperature"])}
    if case["op"] == "policy":
        r = sc.policy_loss(s["logits"], tokens, s["old"], s["advantages"], ref_logprobs=s["ref"],
                           weights=s["weights"], temperature=s["temperature"], clip_low=CLIP_LOW,
                           clip_high=CLIP_HIGH, kl_coef=KL_COEF, entropy_coef=ENTROPY_COEF,
                           scale=s["scale"])
        return {"terms": r.terms, "logprobs": r.logprobs, "entropies": r.entropies,
                "d_logits": r.d_logits}
    r = sc.preference_loss(s["logits"], tokens, s["offsets"], ref_logprobs=s["ref"], beta=BETA,
                           label_smoothing=SMOOTHING, margin=MARGIN, average=case["average"],
                           temperature=s["temperature"], scale=s["scale"])
    return {"loss": r.loss, "losses": r.losses, "sequence_logprobs": r.sequence_logprobs,
            "logprobs": r.logprobs, "d_logits": r.d_logits}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "policy":
        return _plain_policy(state)
    if op == "preference":
        return _plain_preference(state)
    return _plain_lmhead(state)


def work(case):
    rows, V = _rows(case), case["V"]
    if case["op"] == "lmhead":
        d = case["d"]
        return {"bytes": 2 * d * (rows + V) + 12 * rows, "flops": 2 * rows * V * d + 5 * rows * V}
    elt = 2 if case["dtype"] == "bf16" else 4
    # an ignored row is not read; its gradient is written as zeros
    read = rows - case["ignored"]
    back = case["op"] != "logprobs" or case["dir"] == "back"
    size = (read + (rows if back else 0)) * V * elt + 16 * rows
    return {"bytes": size, "flops": read * V * (10 if back else 5)}


# -- the definitions in 64 bits ---------------------------------------------------


def _log_softmax_64(z, temperature, tokens):
    """(log p of the token, entropy) of each row, through autograd-able 64-bit operations."""
    t = temperature.double()[:, None] if torch.is_tensor(temperature) else temperature
    logp = torch.log_softmax(z / t, dim=1)
    token = tokens.clamp(min=0).long()
    lp = logp[torch.arange(z.shape[0], device=z.device), token]
    finite = torch.where(torch.isneginf(logp), torch.zeros_like(logp), logp)
    h = -(torch.exp(logp) * finite).sum(1)
    return lp, h


def _gradient_64(logits, temperature, tokens, upstream):
    """d/dlogits of sum(upstream * (lp, h)) over blocks of rows, ignored rows zero."""
    out = torch.zeros_like(logits, dtype=torch.float64)
    for lo in range(0, logits.shape[0], 256):
        at = slice(lo, lo + 256)
        z = logits[at].double().requires_grad_()
        temp = temperature[at] if torch.is_tensor(temperature) else temperature
        with torch.enable_grad():
            lp, h = _log_softmax_64(z, temp, tokens[at])
            keep = tokens[at] >= 0
            total = (upstream[0][at] * lp)[keep].sum()
            if upstream[1] is not None:
                total = total + (upstream[1][at] * h)[keep].sum()
            if keep.any():
                out[at] = torch.autograd.grad(total, z)[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    tokens, temp = s["tokens"], s["temperature"]
    keep = tokens >= 0
    lps, hs = [], []
    for lo in range(0, tokens.shape[0], 256):
        at = slice(lo, lo + 256)
        if case["op"] == "lmhead":
            if lo == 0:
                weight = s["weight"].double()
            z = torch.matmul(s["hidden"][at].double(), weight.t())
        else:
            z = s["logits"][at].double()
        lp, h = _log_softmax_64(z, temp[at] if torch.is_tensor(temp) else temp, tokens[at])
        lps.append(lp)
        hs.append(h)
    lp = torch.where(keep, torch.cat(lps), 0.0)
    h = torch.where(keep, torch.cat(hs), 0.0)
    if case["op"] == "lmhead" or (case["op"] == "logprobs" and case["dir"] == "forward"):
        return {"logprobs": lp, "entropies": h}
    if case["op"] == "logprobs":
        return {"d_logits": _gradient_64(s["logits"], temp, tokens,
                                         (s["d_logprobs"].double(), s["d_entropies"].double()))}
    if case["op"] == "policy":
        x, y = (v.clone().requires_grad_() for v in (lp, h))
        with torch.enable_grad():
            w = torch.where(keep, s["weights"].double(), 0.0) * s["scale"]
            ratio = torch.exp(x - s["old"].double())
            adv = s["advantages"].double()
            held = torch.clamp(ratio, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
            pg = -torch.minimum(adv * ratio, adv * held)
            gap = s["ref"].double() - x
            kl = torch.expm1(gap) - gap
            loss = (w * (pg + KL_COEF * kl - ENTROPY_COEF * y)).sum()
            gx, gy = torch.autograd.grad(loss, (x, y))
        cut = (adv * held < adv * ratio).double()
        terms = torch.stack([loss.detach()] + [(w * v).detach().sum() for v in (pg, kl, y, cut)])
        return {"terms": terms, "logprobs": lp, "entropies": h,
                "d_logits": _gradient_64(s["logits"], temp, tokens, (gx, gy))}
    n = 2 * case["pairs"]
    edges = s["offsets"].tolist()
    x = lp.clone().requires_grad_()
    with torch.enable_grad():
        sums = []
        for i in range(n):
            part = x[edges[i]:edges[i + 1]]
            many = int(keep[edges[i]:edges[i + 1]].sum())
            sums.append(part.sum() / (max(1, many) if case["average"] else 1))
        sums = torch.stack(sums)
        gap = sums - s["ref"].double()
        margin = BETA * (gap[: n // 2] - gap[n // 2:]) - MARGIN
        losses = -(1.0 - SMOOTHING) * torch.nn.functional.logsigmoid(margin) \
            - SMOOTHING * torch.nn.functional.logsigmoid(-margin)
        loss = s["scale"] * losses.sum()
        gx = torch.autograd.grad(loss, x)[0]
    return {"loss": loss.detach().reshape(1), "losses": losses.detach(),
            "sequence_logprobs": sums.detach(), "logprobs": lp,
            "d_logits": _gradient_64(s["logits"], temp, tokens, (gx, None))}
