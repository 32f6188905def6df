"""The policy loss far from the policy that drew the tokens: ratios and KL
terms past fp32's range, zero advantages and coefficients, banned tokens.

A finite definition gives a finite result: a zero advantage or coefficient
takes its term out, whatever the ratio or the KL beside it."""
from __future__ import annotations

import math

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
LO, HI, T = 0.2, 0.28, 0.8
# short rows on one warp and on four, long rows on clusters, a row past its ring
SHAPES = [(F32, 50), (F32, 1500), (BF16, 6001), (F32, 32003), (BF16, 262144)]


@pytest.fixture(scope="module")
def scorer():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_bound_canvas_b200 import build as B
    B.build()
    import entropy_bound_canvas_b200 as E
    s = E.EBScorer(64, device=DEV)
    yield s
    s.close()


def inputs(rows, V, dtype, seed=5):
    z, tokens, _ = R.make_logits(rows, V, dtype, seed, DEV)
    z = z.clone()
    z[2, tokens[2].long()] = -math.inf  # a banned token was drawn
    lp, H = R.scores(z, T, tokens)
    tl, th = R.logprob_tol(z, T, tokens)
    return z, tokens, lp, H, torch.nan_to_num(tl, nan=0.0), torch.nan_to_num(th, nan=0.0)


def expected(lp, H, old, adv, ref, w, kl_coef, ent_coef):
    """Rows' terms and the factors of log p_a and H, in 64 bits."""
    x = lp - old.double()
    ratio = torch.exp(x)
    A = adv.double()
    free = torch.where(A == 0, 0.0, -A * ratio)
    held = torch.where(A == 0, 0.0, -A * ratio.clamp(1 - LO, 1 + HI))
    cut = held > free
    pg = torch.where(cut, held, free)
    if ref is None:
        kl = back = torch.zeros_like(lp)
    else:
        gap = ref.double() - lp
        back = torch.expm1(gap)
        kl = torch.where(back == math.inf, back, back - gap)
    zero = torch.zeros_like(pg)
    loss = pg + (kl_coef * kl if kl_coef else zero) - (ent_coef * H if ent_coef else zero)
    g = w * (torch.where(cut, zero, pg) + (-kl_coef * back if kl_coef else zero))
    return w * loss, w * pg, w * kl, w * H, w * cut.double(), g, -w * ent_coef


def check(scorer, z, tokens, lp, H, tl, th, old, adv, ref=None, weights=None, scale=1.0,
          kl_coef=0.0, ent_coef=0.0):
    w = (torch.ones_like(lp) if weights is None else weights.double()) * scale
    *parts, g, h = expected(lp, H, old, adv, ref, w, kl_coef, ent_coef)
    kw = dict(ref_logprobs=ref, weights=weights, temperature=T, clip_low=LO, clip_high=HI,
              kl_coef=kl_coef, entropy_coef=ent_coef, scale=scale)
    r = scorer.policy_loss(z, tokens, old, adv, **kw)
    alone = scorer.policy_loss(z, tokens, old, adv, grad=False, **kw)
    # A ratio's relative error is the absolute one of its exponent: log p_a's
    # own, the roundings of log p_a and of the differences, exp's 2 u, and as
    # many products.  The same for exp(ref - log p_a).
    far = [old] if ref is None else [old, ref]
    size = sum(v.double().abs() + (lp - v.double()).abs() for v in far) + 2 * lp.abs()
    rel = torch.nan_to_num(2 * tl + 4 * R.U * size, nan=0.0, posinf=0.0) + 16 * R.U
    off = torch.stack([(rel * p.abs()).sum() if i != 3 else (th * w.abs()).sum()
                       for i, p in enumerate(parts)])
    off[0] += sum(rel * p.abs() * c for p, c in ((parts[1], 1.0), (parts[2], abs(kl_coef)))
                  if c).nan_to_num().sum() + abs(ent_coef) * off[3]
    terms = torch.stack([p.sum() for p in parts])
    for got in (r.terms.double(), alone.terms.double()):
        for i in range(5):
            if not math.isfinite(float(terms[i].float())):  # past fp32: the sum itself
                assert float(got[i]) == float(terms[i].float()), (i, got, terms)
            else:
                assert abs(float(got[i] - terms[i])) <= float(off[i]) + 2 * R.U * abs(
                    float(terms[i])) + 1e-45, (i, got, terms)
    d, tol = R.gradient(z, T, tokens, g, h)
    # a banned token's own element: g (1 - p_a) / T, no entropy term at p_a = 0
    d = torch.where(torch.isnan(d) & (z == -math.inf), (g / T)[:, None], d)
    p = torch.softmax(z.double() / T, 1)
    one = torch.zeros_like(p).scatter_(1, tokens.long()[:, None], 1.0)
    tol = tol + (g.abs() * rel)[:, None] * (p - one).abs() / T * 1.01
    R.check_gradient(r.d_logits, d, tol, z.dtype)
    assert scorer.status() == 0


@pytest.mark.parametrize("dtype,V", SHAPES)
def test_zero_advantages_far_from_the_policy(scorer, dtype, V):
    """An advantage of 0 gives a loss and a gradient of 0 at any ratio."""
    rows = 8
    v = inputs(rows, V, dtype)
    lp = v[2]
    old = torch.where(torch.isfinite(lp), lp, 0.0).float()
    adv = torch.tensor([0.0, 0.0, 0.0, 0.7, -0.0, 1.5, -0.4, 0.0], device=DEV)
    old[0] -= 100.0          # a ratio of e^100
    old[1] = -3e38           # past 64 bits too
    old[4] -= 89.0
    old[7] += 200.0          # a ratio that underflows
    for scale in (1.0, 0.125):
        check(scorer, *v, old, adv, scale=scale, ent_coef=0.01)


@pytest.mark.parametrize("dtype,V", SHAPES)
def test_advantages_far_from_the_policy(scorer, dtype, V):
    """Ratios past fp32 beside small advantages or weights, and cut ones."""
    rows = 8
    v = inputs(rows, V, dtype)
    lp = v[2]
    old = torch.where(torch.isfinite(lp), lp, 0.0).float()
    adv = torch.tensor([1.0, -1e-30, -1.0, 0.7, -1e-38, 2.0, -0.4, 1.0], device=DEV)
    old[0] -= 100.0          # cut: -(1 + clip_high)
    old[1] -= 100.0          # 1e-30 e^100 = 2.7e13
    old[4] -= 100.0
    old[5] = -math.inf       # cut again
    old[7] += 300.0
    check(scorer, *v, old, adv, ent_coef=0.01)
    # the loss and factor fit fp32 though the ratio does not
    adv[1] = adv[4] = -1.0
    weights = torch.tensor([1e-20, 1e-30, 1.0, 1e-20, 1e-28, 1e-20, 1e-20, 1e-20], device=DEV)
    check(scorer, *v, old, adv, weights=weights)
    # a scale past fp32 beside small weights, and the other way round
    old = torch.where(torch.isfinite(lp), lp + 0.1, 0.0).float()
    weights[2] = 1e-20
    check(scorer, *v, old, adv, weights=weights, scale=1e45, ent_coef=0.01)
    check(scorer, *v, old, adv, weights=torch.full_like(weights, 1e25), scale=1e-48,
          ent_coef=0.01)


@pytest.mark.parametrize("dtype,V", SHAPES)
def test_a_kl_term_switched_off_stays_out(scorer, dtype, V):
    """kl_coef = 0 with reference log-probabilities far above the policy's (and
    a banned token, whose KL is infinite): reported, but no part of the loss."""
    rows = 8
    v = inputs(rows, V, dtype)
    lp = v[2]
    old = torch.where(torch.isfinite(lp), lp + 0.1, 0.0).float()
    ref = torch.where(torch.isfinite(lp), lp + 0.2, -5.0).float()
    adv = torch.tensor([1.0, -1.0, 0.5, 0.0, -0.3, 1.0, -1.0, 2.0], device=DEV)
    ref[0] += 100.0
    ref[3] += 2000.0
    ref[4] -= 300.0
    check(scorer, *v, old, adv, ref=ref, ent_coef=0.01)
    # switched on, the term is what it is
    keep = torch.tensor([True, True, False, False, True, True, True, True], device=DEV)
    weights = torch.where(keep, 1e-20, 0.0).float()
    z, tokens, lp, H, tl, th = (t[keep] for t in v)
    check(scorer, z, tokens, lp, H, tl, th, old[keep], adv[keep], ref=ref[keep],
          weights=weights[keep], kl_coef=0.05, ent_coef=0.01)


def test_a_row_far_out_leaves_the_others(scorer):
    """The other rows' gradients are the same bits with and without it."""
    rows, V = 8, 4099
    z, tokens, lp, *_ = inputs(rows, V, BF16)
    old = torch.where(torch.isfinite(lp), lp + 0.1, 0.0).float()
    adv = torch.linspace(-1, 1, rows, device=DEV)
    near = scorer.policy_loss(z, tokens, old, adv, temperature=T)
    old[0] = -500.0
    far = scorer.policy_loss(z, tokens, old, adv, temperature=T)
    assert torch.equal(near.d_logits[1:], far.d_logits[1:])
