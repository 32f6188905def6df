"""Plain 64-bit forms of the scorer's operators, and the rounding bounds the
tests hold its results to.

The bounds count roundings of u = 2^-24 (fp32, half a unit in the last place):
  - an exponent (z - M) log2(e) / T: the difference, the constant's own two
    roundings (1/T or log2(e)/T), the product: 4 u relative, so an absolute
    error of 4 u |ln p| in nats, and as much again from shifts between parts;
  - ex2.approx: 2^-22 relative = 4 u;
  - a running sum: one u per addition of the longest chain, `chain` (a
    thread's share of the row, the joins of threads, warps and CTAs).  Every
    term is positive, so the sum's relative error is at most chain u.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
TERM = 4 * U  # one ex2


def chain(V: int) -> int:
    """Longest chain of additions of a row's sum: a thread's share (at least 64
    threads to a row, 512 to one over 8192), and the joins."""
    return (-(-V // 64) if V <= 8192 else -(-V // 512)) + 24


def log_softmax64(z, T, tokens):
    t = T.double()[:, None] if torch.is_tensor(T) else T
    y = z.double() / t
    m = y.max(1, keepdim=True).values
    e = torch.exp(y - m)
    logp = (y - m) - torch.log(e.sum(1, keepdim=True))
    p = torch.exp(logp)
    a = tokens.clamp(min=0).long()
    at = torch.arange(z.shape[0], device=z.device)
    # 1 - p_a without cancellation: the other ids' share
    others = e.clone()
    others[at, a] = 0.0
    rest = others.sum(1) / e.sum(1)
    lp = torch.where(rest < 0.5, torch.log1p(-rest), logp[at, a])
    # the token's own ln p from `rest` too: ln p_a = -rest rounds to 0 in logp
    logp[at, a] = lp
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    return p, logp, lp, -plogp.sum(1), rest


def scores(z, T, tokens):
    """(log p_a, H) in 64 bits, 0 for ignored rows."""
    _, _, lp, h, _ = log_softmax64(z, T, tokens)
    keep = tokens >= 0
    return torch.where(keep, lp, 0.0), torch.where(keep, h, 0.0)


def gradient(z, T, tokens, g, h):
    """(1/T) [ g (onehot - p) - h p (ln p + H) ] in 64 bits, and the bound of
    each element before its last rounding."""
    p, logp, lp, H, rest = log_softmax64(z, T, tokens)
    iT = (1.0 / T.double() if torch.is_tensor(T) else torch.full_like(lp, 1.0 / T))[:, None]
    g = g.double()[:, None]
    h = torch.zeros_like(g) if h is None else h.double()[:, None]
    lnp = torch.where(p > 0, logp, torch.zeros_like(logp))
    d = -g * p - h * p * (lnp + H[:, None])
    n = chain(z.shape[1])
    # relative error of p: its exponent, its ex2, the sum's
    eps = U * (8 * lnp.abs() + 16 + 2 * n) + 2 * TERM
    # of ln p + H: absolute
    eps_log = U * (8 * lnp.abs() + 8 * H.abs()[:, None] + 16 + 4 * n) + 4 * TERM
    tol = p * (g.abs() * eps + h.abs() * ((lnp + H[:, None]).abs() * eps + eps_log
                                          * (1 + H.abs()[:, None])))
    a = tokens.clamp(min=0).long()[:, None]
    pa = p.gather(1, a)
    d.scatter_(1, a, g * rest[:, None] - h * pa * (lp + H)[:, None])
    top = U * (8 * lnp.abs().amax() + 16 + 4 * n) + 4 * TERM
    ta = g.abs() * rest[:, None] * top + tol.gather(1, a) - pa * g.abs() * eps.gather(1, a)
    tol.scatter_(1, a, ta.clamp(min=0) + 4 * U * g.abs() * rest[:, None])
    keep = (tokens >= 0)[:, None]
    return torch.where(keep, d * iT, 0.0), torch.where(keep, tol * iT, 0.0)


def logprob_tol(z, T, tokens):
    """Absolute bounds of log p_a and H."""
    p, logp, lp, H, rest = log_softmax64(z, T, tokens)
    n = chain(z.shape[1])
    lnp = torch.where(p > 0, logp, torch.zeros_like(logp)).abs()
    spread = (p * lnp).sum(1)          # the sums' terms' exponents
    rel = U * (8 * spread + 16 + n) + TERM
    # near p_a = 1 the error is relative to 1 - p_a (and to the others' gaps)
    others = torch.minimum(torch.ones_like(rest), 2 * rest)
    t_lp = others * (rel + U * 8 * lnp.amax(1)) + U * 8 * lp.abs()
    # H = ln S - ln 2 W / S: two sums
    t_h = 2 * rel + U * (8 * (p * lnp * lnp).sum(1) + (8 + n) * H) + TERM * (1 + H)
    # terms below 2^-126 of the maximum flush to zero
    dropped = z.shape[1] * 2.0 ** -125 * (1 + lnp.amax(1))
    return t_lp + dropped, t_h + dropped


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check_gradient(d, ref, tol, dtype, name=""):
    """Every element within the bound plus its last rounding (and what flush to
    zero or the type's smallest steps drop)."""
    bound = tol + half_step(dtype) * (ref.abs() + tol) + 2.0 ** -120
    off = (d.double() - ref).abs()
    bad = off > bound
    assert not bool(bad.any()), (name, int(bad.sum()), float((off / bound).max()))


def policy(z, T, tokens, old, adv, ref, weights, lo, hi, kl_coef, ent_coef, scale):
    """Terms, scores and per-row upstream gradients of the policy loss."""
    lp, H = scores(z, T, tokens)
    keep = tokens >= 0
    w = torch.ones_like(lp) if weights is None else weights.double()
    keep = keep & (w != 0)
    w = torch.where(keep, w, 0.0) * scale
    lp, H = torch.where(keep, lp, 0.0), torch.where(keep, H, 0.0)
    A = torch.where(keep, adv.double(), 0.0)
    old = torch.where(keep, old.double(), 0.0)
    r = torch.exp(lp - old)
    free, held = -A * r, -A * r.clamp(1 - lo, 1 + hi)
    cut = held > free
    if ref is None:
        kl = dkl = torch.zeros_like(lp)
    else:
        gap = torch.where(keep, ref.double(), 0.0) - lp
        kl, dkl = torch.expm1(gap) - gap, -torch.expm1(gap)
    pg = torch.maximum(free, held)
    g = w * (torch.where(cut, 0.0, free) + kl_coef * dkl)
    h = -w * ent_coef
    parts = [(w * v).sum() for v in (pg, kl, H, cut.double())]
    terms = torch.stack([parts[0] + kl_coef * parts[1] - ent_coef * parts[2]] + parts)
    size = torch.stack([(w * (pg.abs() + abs(kl_coef) * kl + abs(ent_coef) * H)).abs().sum(),
                        (w * pg).abs().sum(), (w * (kl + 1e-3)).abs().sum(),
                        (w * H).abs().sum(), w.abs().sum()])
    return terms, size, lp, H, g, h, keep


def preference(lp, tokens, offsets, ref, beta, smooth, margin, average, scale):
    """Loss, losses, sequence sums and d loss / d log p per row."""
    off = offsets.tolist()
    n = len(off) - 1
    P = n // 2
    S, share = [], []
    for s in range(n):
        part, keep = lp[off[s]:off[s + 1]], tokens[off[s]:off[s + 1]] >= 0
        many = int(keep.sum())
        share.append(1.0 / max(1, many) if average else 1.0)
        S.append(part[keep].double().sum() * share[-1])
    S = torch.stack(S) if S else lp.new_zeros(0).double()
    r = torch.zeros_like(S) if ref is None else ref.double()
    m = beta * ((S[:P] - r[:P]) - (S[P:] - r[P:])) - margin
    ls = torch.nn.functional.logsigmoid
    losses = -(1 - smooth) * ls(m) - smooth * ls(-m)
    dm = -(1 - smooth) * torch.sigmoid(-m) + smooth * torch.sigmoid(m)
    g = torch.zeros_like(lp, dtype=torch.float64)
    for k in range(P):
        for s, sign in ((k, 1.0), (P + k, -1.0)):
            g[off[s]:off[s + 1]] = sign * dm[k] * beta * scale * share[s]
    return scale * losses.sum(), losses, S, torch.where(tokens >= 0, g, 0.0)


def make_logits(rows, V, dtype, seed, dev, banned=0, ld=None, shift=0):
    """Seeded logits with a boosted id per row, tokens mostly on it; rows at
    stride ld, the first one `shift` elements into its buffer."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((rows, V), generator=g)
    top = torch.randint(0, V, (rows,), generator=g)
    at = torch.arange(rows)
    boost = torch.where(torch.rand(rows, generator=g) < 0.5, 16.0, 2.0)
    z[at, top] += boost
    tokens = torch.where(torch.rand(rows, generator=g) < 0.7, top,
                         torch.randint(0, V, (rows,), generator=g))
    if banned:
        ids = torch.randint(0, V, (banned,), generator=g)
        kept = z[at, tokens].clone(), z[at, top].clone()
        z[:, ids] = -math.inf
        z[at, tokens], z[at, top] = kept
    ld = V if ld is None else ld
    buf = torch.full((shift + rows * ld + 16,), 7.25, dtype=dtype, device=dev)
    view = buf.as_strided((rows, V), (ld, 1), shift)
    view.copy_(z.to(dtype))
    return view, tokens.to(torch.int32).to(dev), buf
