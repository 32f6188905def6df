"""Log-probabilities as far out as fp32 holds them: a token masked with the
type's lowest value, differences near the end of the range."""
from __future__ import annotations

import math

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_bound_canvas_b200 import build as B
    B.build()
    import entropy_bound_canvas_b200 as E
    return E


@pytest.fixture(scope="module")
def scorer(E):
    s = E.EBScorer(64, device=DEV)
    yield s
    s.close()


def close(got, want):
    """The difference, the division and T round once each; ln S is far below a
    rounding."""
    if abs(want) > 3.4028235677973366e38:
        return got == -math.inf
    return abs(got / want - 1) <= 4 * R.U


@pytest.mark.parametrize("T", [0.9, 1.0, 1.4, 2.0, 1000.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [8, 333, 2048, 32003, 262144])
def test_a_token_at_the_lowest_value(scorer, dtype, V, T):
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    z, tokens, _ = R.make_logits(5, V, dtype, V + 5, DEV)
    z, tokens = z.clone(), tokens.clone()
    tokens[:] = 3
    z[:4, 3] = torch.tensor([low, low * 0.75, low * 0.5, low], dtype=dtype)
    z[3, 4] = high * 0.875   # the difference itself is past fp32
    z[4, 3] = -math.inf
    r = scorer.token_logprobs(z, tokens, temperature=T)
    T32 = float(torch.tensor(T, dtype=F32))
    for i in range(4):
        row = z[i].double()
        want = float(row[3] - row.max()) / T32
        assert close(float(r.logprobs[i]), want), (i, float(r.logprobs[i]), want)
    assert float(r.logprobs[4]) == -math.inf
    assert torch.isfinite(r.entropies).all()
    alone = scorer.token_logprobs(z, tokens, temperature=T, entropies=False)
    for i in range(4):
        row = z[i].double()
        assert close(float(alone.logprobs[i]), float(row[3] - row.max()) / T32)
    # a ratio against the same log-probability is 1, whatever its size
    finite = torch.isfinite(r.logprobs)
    p = scorer.policy_loss(z[finite], tokens[finite], r.logprobs[finite],
                           torch.ones(int(finite.sum()), device=DEV), temperature=T)
    assert float(p.terms[0]) == -float(finite.sum())
    assert scorer.status() == 0


def test_two_masked_sequences_have_a_margin(scorer):
    """Finite sums on both sides: the margin is their difference, not inf - inf."""
    z = torch.zeros((2, 16), device=DEV)
    z[:, 3] = torch.finfo(F32).min
    tokens = torch.tensor([3, 3], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    r = scorer.preference_loss(z, tokens, off)
    assert torch.isfinite(r.sequence_logprobs).all()
    assert abs(float(r.loss) - math.log(2.0)) < 4 * R.U


@pytest.mark.parametrize("rows", [3, 70, 140])
def test_lmhead_scores_far_out(scorer, E, rows):
    """z_a = -1.5 x 2^127 exactly: one product of two bf16."""
    V, d = 300, 64
    h = torch.zeros((rows, d), dtype=BF16, device=DEV)
    w = torch.zeros((V, d), dtype=BF16, device=DEV)
    h[:, 5] = 2.0 ** 63
    w[17, 5] = -1.5 * 2.0 ** 64
    tokens = torch.full((rows,), 17, dtype=torch.int32, device=DEV)
    with E.EBScorer(256, device=DEV) as sc:
        for T in (0.9, 1.0, 2.0):
            r = sc.lmhead_logprobs(h, w, tokens, temperature=T)
            want = -1.5 * 2.0 ** 127 / float(torch.tensor(T, dtype=F32))
            assert all(close(float(v), want) for v in r.logprobs), (float(r.logprobs[0]), want)
            assert (r.entropies - math.log(V - 1)).abs().max() < 1e-5
        assert sc.status() == 0


@pytest.mark.parametrize("T", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("V", [40, 20000])
def test_a_banned_token_among_lowest_values(scorer, V, T):
    """-inf for the token where every other logit is the type's lowest: log p is
    -inf, the entropy that of the others."""
    z = torch.full((2, V), torch.finfo(F32).min, device=DEV)
    z[0, 5] = -math.inf
    tokens = torch.tensor([5, 6], dtype=torch.int32, device=DEV)
    r = scorer.token_logprobs(z, tokens, temperature=T)
    assert float(r.logprobs[0]) == -math.inf
    assert abs(float(r.entropies[0]) - math.log(V - 1)) < 1e-5
    assert abs(float(r.logprobs[1]) + math.log(V)) < 1e-5
    assert scorer.status() == 0


@pytest.mark.parametrize("V", [40, 20000])
def test_the_smallest_temperatures(E, scorer, V):
    """fp32's smallest normal number is one; what lies below it (its reciprocal
    is past fp32) is refused, per row reported."""
    tiny = torch.finfo(F32).tiny
    z, tokens, _ = R.make_logits(4, V, F32, 3, DEV)
    tokens = z.argmax(1).to(torch.int32)
    zero = torch.zeros(4, device=DEV)
    r = scorer.token_logprobs(z, tokens, temperature=tiny)
    assert torch.equal(r.logprobs, zero) and torch.equal(r.entropies, zero)
    assert (scorer.token_logprobs_backward(z, tokens, zero + 1, temperature=tiny) == 0).all()
    assert scorer.status() == 0
    h, w = (torch.zeros((n, 8), dtype=BF16, device=DEV) for n in (4, 9))
    for T in (tiny / 2, 1e-40, 1e-45):
        with pytest.raises(E.EBError):
            scorer.token_logprobs(z, tokens, temperature=T)
        with pytest.raises(E.EBError):
            scorer.lmhead_logprobs(h, w, tokens % 9, temperature=T)
        each = torch.tensor([1.0, T, 1.0, tiny], dtype=F32, device=DEV)
        r = scorer.token_logprobs(z, tokens, temperature=each)
        assert torch.equal(torch.isnan(r.logprobs), each < tiny)
        assert scorer.status(clear=True) == E.STATUS_NONFINITE
