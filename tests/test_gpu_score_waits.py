"""The row kernels keep a short wait limit: each call on rows that are copied
into shared memory reports the wait that ran out, and leaves the right result
or NaN."""
from __future__ import annotations

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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,V", [(1, 20001), (300, 20000), (40, 262144), (1003, 131072)])
def test_every_call_reports_a_short_limit(E, dtype, rows, V):
    """One CTA's row and rows on clusters, one round of them and several, shares
    inside the ring and past it."""
    sc = E.EBScorer(rows + 1, device=DEV)
    z, tokens, _ = R.make_logits(rows, V, dtype, 9, DEV)
    lp, _ = sc.token_logprobs(z, tokens)
    adv = torch.ones(rows, device=DEV)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV)
    out = torch.empty_like(z, memory_format=torch.contiguous_format)

    def calls():
        yield "scores", lambda: sc.token_logprobs(z, tokens)
        yield "alone", lambda: sc.token_logprobs(z, tokens, entropies=False)
        yield "back", lambda: [sc.token_logprobs_backward(z, tokens, adv, adv, out=out)]
        yield "back alone", lambda: [sc.token_logprobs_backward(z, tokens, adv, out=out)]
        yield "policy", lambda: sc.policy_loss(z, tokens, lp, adv, entropy_coef=0.1, out=out)
        yield "loss", lambda: sc.policy_loss(z, tokens, lp, adv, grad=False)
        yield "preference", lambda: sc.preference_loss(z, tokens, off, out=out)

    for name, call in calls():
        want = [None if t is None else t.clone() for t in call()]
        assert sc.status() == 0, name
        for limit in (1, 100):
            out.fill_(7.0)
            sc.set_wait_limit(limit)
            got = call()
            assert sc.status(clear=True) & E.STATUS_TIMEOUT, (name, limit)
            assert any(torch.isnan(t).any() for t in got if t is not None), (name, limit)
            if name in ("policy", "loss"):
                assert torch.isnan(got[0]).all()
            if name != "preference":  # there one NaN row is its pair's, so every row's
                for a, b in zip(got, want):
                    if a is not None:
                        assert ((a == b) | torch.isnan(a)).view(a.shape[0], -1).all(1)[
                            ~torch.isnan(a).view(a.shape[0], -1).any(1)].all(), name
            sc.set_wait_limit(0)
            again = call()
            assert sc.status() == 0, (name, limit)
            assert all(a is None or torch.equal(a, b) for a, b in zip(again, want)), name
    sc.close()


@pytest.mark.parametrize("rows,V,d", [(20, 5000, 256), (60, 5000, 2560), (100, 5000, 256),
                                      (256, 5000, 256), (256, 40001, 2560), (300, 9000, 1000),
                                      (1300, 20000, 256), (2048, 9001, 2560), (19100, 300, 64)])
def test_scores_from_hidden_states_report_a_short_limit(E, rows, V, d):
    """Every form of the product, the CTA pairs among them, cut short at its
    first wait and later: a wait that ran out is reported, rows are right or NaN,
    and the next call is right at once."""
    sc = E.EBScorer(rows, device=DEV)
    g = torch.Generator().manual_seed(rows)
    h = torch.randn((rows, d), generator=g).to(BF16).to(DEV)
    w = torch.randn((V, d), generator=g).to(BF16).to(DEV)
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32).to(DEV)
    want = sc.lmhead_logprobs(h, w, tokens)
    assert sc.status() == 0
    for limit in (1, 100, 400, 700, 1000, 2000, 4000, 10000) * 3:
        sc.set_wait_limit(limit)
        got = sc.lmhead_logprobs(h, w, tokens)
        bits = sc.status(clear=True)
        sc.set_wait_limit(0)
        again = sc.lmhead_logprobs(h, w, tokens)
        assert bits & E.STATUS_TIMEOUT or limit > 100, limit
        for a, b, c in zip(got, want, again):
            assert ((a == b) | torch.isnan(a)).all(), limit
            # (a warp of padding rows may give up alone)
            assert bits & E.STATUS_TIMEOUT or not torch.isnan(a).any(), limit
            assert torch.isnan(a).any() or limit > 100, limit
            assert torch.equal(b, c), limit
        assert sc.status() == 0
    sc.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,V", [(600, 9001), (700, 20000), (300, 262144), (2, 1000003)])
def test_rows_cut_short_on_their_way(E, dtype, rows, V):
    """Limits that some rows keep and some do not, again and again: rows are
    right or NaN, a NaN was reported, and the next call is right at once."""
    sc = E.EBScorer(rows, device=DEV)
    z, tokens, _ = R.make_logits(rows, V, dtype, 9, DEV)
    g = torch.ones(rows, device=DEV)
    out = torch.empty_like(z, memory_format=torch.contiguous_format)

    def calls():
        yield lambda: sc.token_logprobs(z, tokens)
        yield lambda: [sc.token_logprobs_backward(z, tokens, g, g, out=out)]
        yield lambda: [sc.token_logprobs_backward(z, tokens, g, out=out)]

    for call in calls():
        want = [t.clone() for t in call()]
        assert sc.status() == 0
        for limit in (500, 1000, 1500, 2500, 4000, 6000, 9000, 14000, 19000) * 2:
            out.fill_(7.0)
            sc.set_wait_limit(limit)
            got = [t.clone() for t in call()]
            bits = sc.status(clear=True)
            sc.set_wait_limit(0)
            again = call()
            assert sc.status() == 0
            for a, b, c in zip(got, want, again):
                a, b = a.view(rows, -1), b.view(rows, -1)
                nan = torch.isnan(a).any(1)
                assert torch.equal(a[~nan], b[~nan]), limit
                assert bits & E.STATUS_TIMEOUT or not nan.any(), limit
                assert torch.equal(b, c.view(rows, -1)), limit
    sc.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("limit", [1, 100])
def test_a_single_row_reports_a_short_limit_every_time(E, dtype, limit):
    """One row has one wait for its sums: it runs out also where its warp comes to
    it late and finds them there."""
    sc = E.EBScorer(4, device=DEV)
    z, tokens, _ = R.make_logits(1, 20001, dtype, 9, DEV)
    want = sc.token_logprobs(z, tokens)
    sc.set_wait_limit(limit)
    for i in range(300):
        r = sc.token_logprobs(z, tokens, entropies=i % 2 == 0)
        assert sc.status(clear=True) & E.STATUS_TIMEOUT, i
        assert torch.isnan(r.logprobs).all(), i
    sc.set_wait_limit(0)
    assert torch.equal(sc.token_logprobs(z, tokens).logprobs, want.logprobs)
    sc.close()
