"""The KL term near the reference: e^x - 1 - x keeps its digits where x is
small (a policy that has just left its reference)."""
from __future__ import annotations

import math

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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


def one_row(V):
    """A confident row (1 - p_a = 1e-3): log p_a is known to about 1e-8, so the
    gap to a reference 1e-5 away is known to three digits."""
    z = torch.zeros((1, V), device=DEV)
    z[0, 7] = math.log(999.0 * (V - 1))
    return z, torch.tensor([7], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("V", [64, 1000, 20000])
@pytest.mark.parametrize("far", [1e-5, 3e-5, 1e-4, 1e-3, 1e-2, 0.1, 0.45, 0.55, 1.0, 5.0, 20.0])
def test_kl_of_a_row(scorer, V, far):
    z, tokens = one_row(V)
    lp, _ = R.scores(z, 1.0, tokens)
    tl, _ = R.logprob_tol(z, 1.0, tokens)
    one = torch.ones(1, device=DEV)
    for sign in (1.0, -1.0):
        ref = (lp + sign * far).float()
        gap = float(ref.double() - lp)
        r = scorer.policy_loss(z, tokens, lp.float(), one, ref_logprobs=ref, kl_coef=0.5)
        # e^x - 1 - x in 64 bits: a series where the difference would cancel
        want = math.expm1(gap) - gap if abs(gap) > 0.3 else \
            sum(gap ** k / math.factorial(k) for k in range(2, 16))
        # the gap's error: log p_a's, and the roundings of two differences; the
        # function's: a few roundings, 4.5 times as many where it is a difference
        # (x = 0.5: 0.649 - 0.5)
        off = abs(math.expm1(gap)) * (float(tl) + 2 * R.U * abs(gap)) + 16 * R.U * want
        assert abs(float(r.terms[2]) - want) <= off, (gap, float(r.terms[2]), want, off)
        # the gradient's factor is -(e^x - 1) of the same gap
        rest = 1e-3
        g = -1.0 - 0.5 * math.expm1(gap)
        slack = 1e-3 * abs(g) + 0.5 * math.exp(gap) * float(tl) + 1e-6
        assert abs(float(r.d_logits[0, 7]) - g * rest) <= slack * rest


def test_kl_is_never_negative(scorer):
    """At the reference itself, and a step of fp32 to either side."""
    rows, V = 40, 700
    z, tokens, _ = R.make_logits(rows, V, torch.float32, 3, DEV)
    lp = scorer.token_logprobs(z, tokens).logprobs
    adv = torch.zeros(rows, device=DEV)
    for ref in (lp, torch.nextafter(lp, lp + 1), torch.nextafter(lp, lp - 1)):
        for i in range(0, rows, 8):
            at = slice(i, i + 1)
            r = scorer.policy_loss(z[at], tokens[at], lp[at], adv[at], ref_logprobs=ref[at])
            assert 0.0 <= float(r.terms[2]) <= 1e-9
