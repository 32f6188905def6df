"""A handle's workspace is cleared before its first call can begin, whatever
the other streams are doing: made and used inside a side stream while the
default stream is busy, it gives the bits of one made in peace."""
from __future__ import annotations

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BUSY = 400_000_000  # clock cycles of the default stream: about 0.2 s


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_bound_canvas_b200 import build as B
    B.build()
    import entropy_bound_canvas_b200 as E
    return E


def made_and_used(busy, make, use):
    side = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    if busy:
        torch.cuda._sleep(BUSY)
    with torch.cuda.stream(side):
        handle = make()
        got = use(handle)
        first = [t.clone() for t in got]
    # the clear would come here, at the end of the default stream's work
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = [t.clone() for t in use(handle)]
    torch.cuda.synchronize()
    status = handle.status()
    handle.close()
    return first, again, status


def test_a_scorer_made_while_the_default_stream_is_busy(E):
    rows, V, d = 200, 9001, 128
    z, tokens, _ = R.make_logits(rows, V, torch.bfloat16, 3, DEV)
    g = torch.Generator().manual_seed(4)
    old, adv = (torch.randn(rows, generator=g).to(DEV) for _ in range(2))
    off = torch.tensor([0, 40, 90, 150, 200], dtype=torch.int32, device=DEV)
    h = torch.randn((rows, d), generator=g).to(torch.bfloat16).to(DEV)
    w = torch.randn((V, d), generator=g).to(torch.bfloat16).to(DEV)

    def use(sc):
        out = []
        for _ in range(3):
            p = sc.policy_loss(z, tokens, old, adv, entropy_coef=0.1, scale=0.01)
            q = sc.preference_loss(z, tokens, off)
            m = sc.lmhead_logprobs(h, w, tokens)
            out += [p.terms, p.logprobs, p.d_logits, q.loss, q.losses, q.d_logits, *m]
        return out

    def make():
        return E.EBScorer(4096, device=DEV)

    want, _, _ = made_and_used(False, make, use)
    first, again, status = made_and_used(True, make, use)
    assert status == 0
    for got in (first, again):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_sampler_made_while_the_default_stream_is_busy(E):
    B, L, V, steps = 2, 16, 8200, 6
    g = torch.Generator().manual_seed(4)
    logits = (2.0 * torch.randn((steps, B, L, V), generator=g)).to(torch.bfloat16).to(DEV)
    logits[:, :, ::2, 5] += 14.0

    def use(eb):
        canvas, committed, stop = eb.new_canvas()
        H, amax = (t.zero_() for t in eb.outputs())
        out = []
        for s in range(steps):
            eb.step(logits[s], s, canvas, committed, H, amax, stop)
            out += [t.clone() for t in (canvas, committed, H, amax, stop)]
        return out

    def make():
        return E.EBSampler(B, L, V, device=DEV, num_steps=steps, seed=3)

    want, _, _ = made_and_used(False, make, use)
    first, again, status = made_and_used(True, make, use)
    assert status == 0
    for got in (first, again):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
