"""Scores from hidden states of many rows: past the rows of one round of
CTAs, to one vocabulary range per row tile and several rounds of them."""
from __future__ import annotations

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_bound_canvas_b200 import build as B
    B.build()
    import entropy_bound_canvas_b200 as E
    return E


# 1153: the first pairs of an odd number of tiles; 9472 and 9473: the last rows
# of two ranges and the first of one; 18944 and 18945: one round of tiles and two
@pytest.mark.parametrize("rows,V,d", [(1152, 1500, 72), (1153, 1500, 72), (2049, 1000, 136),
                                      (4096, 2100, 64), (9472, 700, 64), (9473, 700, 64),
                                      (18944, 300, 40), (18945, 300, 40), (40001, 515, 16)])
def test_scores_of_many_rows(E, rows, V, d):
    """Codes over 8: exact logits, so only the softmax rounds.  The scorer is
    made for just these rows."""
    g = torch.Generator().manual_seed(rows + V)
    w = (torch.randint(-2, 3, (V, d), generator=g).float() / 8).to(DEV)
    h = (torch.randint(-2, 3, (rows, d), generator=g).float() / 8).to(DEV)
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32).to(DEV)
    tokens[::7] = -1
    T = 0.3 + torch.rand(rows, generator=g).to(DEV)
    with E.EBScorer(rows, device=DEV) as sc:
        r = sc.lmhead_logprobs(h.to(BF16), w.to(BF16), tokens, temperature=T)
        for lo in range(0, rows, 4096):
            at = slice(lo, lo + 4096)
            z = h[at].double() @ w.double().T
            keep = tokens[at] >= 0
            lp, H = R.scores(z, T[at], tokens[at])
            tl, th = R.logprob_tol(z, T[at], tokens[at])
            zero = torch.zeros_like(tl)
            assert ((r.logprobs[at].double() - lp).abs() <= torch.where(keep, tl, zero)).all()
            assert ((r.entropies[at].double() - H).abs() <= torch.where(keep, th, zero)).all()
        assert sc.status() == 0
