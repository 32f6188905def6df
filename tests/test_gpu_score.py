"""The scorer (token log-probabilities, policy and preference losses, their
gradients) against plain 64-bit forms, through the Python binding."""
from __future__ import annotations

import math

import pytest

import score_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = [F32, BF16]


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
    s = E.EBScorer(4096, device=DEV)
    yield s
    s.close()


def randn(n, seed):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)).to(DEV)


def check_scores(r, z, T, tokens, keep=None):
    lp, H = R.scores(z, T, tokens)
    tl, th = R.logprob_tol(z, T, tokens)
    if keep is not None:
        lp, H = torch.where(keep, lp, 0.0), torch.where(keep, H, 0.0)
    live = tokens >= 0 if keep is None else keep
    tl, th = torch.where(live, tl, 0.0), torch.where(live, th, 0.0)
    assert ((r.logprobs.double() - lp).abs() <= tl).all(), \
        float(((r.logprobs.double() - lp).abs() - tl).max())
    assert ((r.entropies.double() - H).abs() <= th).all(), \
        float(((r.entropies.double() - H).abs() - th).max())


# V: one id, below a vector, odd, the tiny canvas, ragged, an odd large one, the card's
SIZES = [(1, 1), (3, 2), (17, 7), (5, 64), (16, 1024), (33, 1000), (9, 4099), (300, 515),
         (7, 32003), (3, 50257), (2, 262144), (1, 262143), (4, 131073)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", SIZES)
def test_scores_and_their_gradient(scorer, rows, V, dtype):
    z, tokens, _ = R.make_logits(rows, V, dtype, 100 * rows + V, DEV)
    r = scorer.token_logprobs(z, tokens, temperature=0.7)
    check_scores(r, z, 0.7, tokens)
    g, h = randn(rows, 1), randn(rows, 2)
    for gh in (h, None):
        d = scorer.token_logprobs_backward(z, tokens, g, gh, temperature=0.7)
        R.check_gradient(d, *R.gradient(z, 0.7, tokens, g, gh), dtype)
    assert scorer.status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,ld,shift,dld,dshift", [
    (1000, 1024, 0, 1000, 0),      # padded rows, aligned
    (1001, 1001, 3, 1001, 3),      # every row at its own alignment, both alike
    (1001, 1003, 5, 1002, 2),      # the gradient's rows aligned differently
    (5, 9, 1, 8, 0), (70001, 70004, 7, 70001, 1), (32768, 32769, 0, 32768, 0),
])
def test_strides_alignments_and_what_lies_between_rows(scorer, dtype, V, ld, shift, dld, dshift):
    rows = 11
    z, tokens, zbuf = R.make_logits(rows, V, dtype, V + ld, DEV, ld=ld, shift=shift)
    before = zbuf.clone()
    buf = torch.full((dshift + rows * dld + 16,), 3.5, dtype=dtype, device=DEV)
    out = buf.as_strided((rows, V), (dld, 1), dshift)
    g, h = randn(rows, 3), randn(rows, 4)
    d = scorer.token_logprobs_backward(z, tokens, g, h, temperature=1.3, out=out)
    assert d is out
    R.check_gradient(out, *R.gradient(z, 1.3, tokens, g, h), dtype)
    assert torch.equal(zbuf, before)  # the logits are read only
    touched = torch.zeros_like(buf, dtype=torch.bool)
    touched.as_strided((rows, V), (dld, 1), dshift).fill_(True)
    assert (buf[~touched] == 3.5).all()
    check_scores(scorer.token_logprobs(z, tokens, temperature=1.3), z, 1.3, tokens)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [8, 333, 2048, 32003, 262144])
def test_masked_logits(scorer, dtype, V):
    """-inf and the type's lowest value as masks: all but one id, some, the
    argmax's neighbours; a token that is itself masked; a row of one value."""
    low = torch.finfo(dtype).min
    rows = 9
    z, tokens, _ = R.make_logits(rows, V, dtype, V + 5, DEV)
    z, tokens = z.clone(), tokens.clone()
    every = torch.arange(V, device=DEV)
    z[0, every != tokens[0]] = -math.inf                      # only the token left
    z[1, every != tokens[1]] = low
    z[2, every % 3 == (tokens[2] + 1) % 3] = -math.inf
    z[3, every % 3 == (tokens[3] + 1) % 3] = low
    z[4, :] = low                                             # uniform over the lowest value
    z[5, :] = 0.0
    z[6, : V - 1] = -math.inf                                 # one id, at the end
    tokens[6] = V - 1
    z[7, 0], tokens[7] = low, 0                               # an improbable token
    z[8, :] = torch.finfo(dtype).max                          # uniform at the largest value
    r = scorer.token_logprobs(z, tokens, temperature=0.5)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[7] = False  # ln p of about -1e38: compared by its relative error below
    lp, H = R.scores(z, 0.5, tokens)
    tl, th = R.logprob_tol(z, 0.5, tokens)
    assert ((r.logprobs.double() - lp).abs() <= tl)[keep].all()
    assert ((r.entropies.double() - H).abs() <= th)[keep].all()
    want = (float(z[7, 0]) - float(z[7].float().max())) / 0.5
    if math.isfinite(float(torch.tensor(want, dtype=F32))):
        assert abs(float(r.logprobs[7]) / want - 1) < 4 * R.U
    else:
        assert float(r.logprobs[7]) == -math.inf
    assert float(r.logprobs[0]) == 0.0 and float(r.entropies[0]) == 0.0
    g, h = randn(rows, 6), randn(rows, 7)
    d = scorer.token_logprobs_backward(z, tokens, g, None, temperature=0.5)
    ref, tol = R.gradient(z, 0.5, tokens, g, None)
    R.check_gradient(d[keep], ref[keep], tol[keep], dtype)
    assert float(d[0].float().abs().max()) == 0.0
    assert (d[z == -math.inf] == 0).all()
    d = scorer.token_logprobs_backward(z[:7], tokens[:7], g[:7], h[:7], temperature=0.5)
    R.check_gradient(d, *R.gradient(z[:7], 0.5, tokens[:7], g[:7], h[:7]), dtype)
    assert scorer.status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [50, 32003])
def test_not_finite_rows_stay_in_their_rows(scorer, dtype, V):
    rows = 8
    z, tokens, _ = R.make_logits(rows, V, dtype, V, DEV)
    z, tokens = z.clone(), tokens.clone()
    at = [0, V // 2, V - 1, 3]
    z[0, at[0]] = math.nan
    z[1, at[1]] = math.inf
    z[2, :] = -math.inf
    tokens[3] = V                     # one past the vocabulary
    z[4, tokens[4].long()] = math.nan
    z[5, V - 1] = math.nan
    tokens[6] = -1                    # ignored: NaN logits are not read
    z[6, :] = math.nan
    r = scorer.token_logprobs(z, tokens, temperature=0.9)
    g = torch.ones(rows, device=DEV)
    d = scorer.token_logprobs_backward(z, tokens, g, g, temperature=0.9)
    for i in (0, 1, 2, 3, 4, 5):
        assert torch.isnan(r.logprobs[i]) and torch.isnan(d[i]).any(), i
    for i in (0, 1, 2, 4, 5):
        assert torch.isnan(r.entropies[i]), i
    assert float(r.logprobs[6]) == 0.0 and float(r.entropies[6]) == 0.0
    assert (d[6] == 0).all()
    check_scores(type(r)(r.logprobs[7:], r.entropies[7:]), z[7:], 0.9, tokens[7:])
    R.check_gradient(d[7:], *R.gradient(z[7:], 0.9, tokens[7:], g[7:], g[7:]), dtype)
    assert scorer.status(clear=True) == 1 | 2
    assert scorer.status() == 0


def test_a_banned_token_has_probability_zero(scorer):
    z, tokens, _ = R.make_logits(2, 4099, F32, 8, DEV)
    z = z.clone()
    z[0, tokens[0].long()] = -math.inf
    r = scorer.token_logprobs(z, tokens)
    assert float(r.logprobs[0]) == -math.inf
    _, H = R.scores(z, 1.0, tokens)
    assert abs(float(r.entropies[0]) - float(H[0])) < 1e-5
    d = scorer.token_logprobs_backward(z, tokens, torch.ones(2, device=DEV))
    assert float(d[0, tokens[0].long()]) == 1.0  # 1 - p_a


@pytest.mark.parametrize("gap", [1.0, 8.0, 16.0, 24.0, 40.0])
def test_confident_rows_keep_their_precision(scorer, gap):
    """1 - p_a down to 2^-50: log p_a, H and the token's gradient to a few
    roundings, not to 2^-24 of 1."""
    V = 5000
    z = torch.zeros((1, V), device=DEV)
    z[0, 123] = gap + math.log(V)
    tokens = torch.tensor([123], dtype=torch.int32, device=DEV)
    lp, H = R.scores(z, 1.0, tokens)
    r = scorer.token_logprobs(z, tokens)
    # the exponent's error moves every other term alike
    rel = R.U * (8 * (gap + 9) + R.chain(V) + 32)
    assert abs(float(r.logprobs[0]) / float(lp[0]) - 1) < rel
    assert abs(float(r.entropies[0]) / float(H[0]) - 1) < 2 * rel
    d = scorer.token_logprobs_backward(z, tokens, torch.ones(1, device=DEV))
    _, _, _, _, rest = R.log_softmax64(z, 1.0, tokens)
    assert abs(float(d[0, 123]) / float(rest[0]) - 1) < rel


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [(64, 1000), (700, 2049), (40, 32003), (5, 262144)])
def test_row_temperatures_and_ignored_rows(scorer, dtype, rows, V):
    z, tokens, _ = R.make_logits(rows, V, dtype, rows + V, DEV, banned=V // 20)
    tokens = tokens.clone()
    tokens[::5] = -1
    T = 0.4 + 0.8 * torch.rand(rows, generator=torch.Generator().manual_seed(5)).to(DEV)
    check_scores(scorer.token_logprobs(z, tokens, temperature=T), z, T, tokens)
    g, h = randn(rows, 1), randn(rows, 2)
    d = scorer.token_logprobs_backward(z, tokens, g, h, temperature=T)
    R.check_gradient(d, *R.gradient(z, T, tokens, g, h), dtype)
    assert scorer.status() == 0
    T[1], T[2], T[3] = 0.0, math.nan, -1.0
    r = scorer.token_logprobs(z, tokens, temperature=T)
    assert torch.isnan(r.logprobs[1:4]).all() and not torch.isnan(r.logprobs[4:]).any()
    assert scorer.status(clear=True) == 2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [
    (4096, 300), (2500, 2003), (1900, 4001),   # short rows, several to a block
    (900, 9001), (1000, 20011),                # several rows to a cluster, two shares in the ring
    (650, 70001), (310, 131072)])              # shares longer than the ring, copied twice
def test_many_rows_in_turn(scorer, dtype, rows, V):
    """More rows than are in flight, a fifth of them ignored: every row against
    the 64-bit form, in blocks."""
    z, tokens, _ = R.make_logits(rows, V, dtype, rows + V, DEV, banned=V // 50)
    tokens = tokens.clone()
    tokens[torch.rand(rows, generator=torch.Generator().manual_seed(2)) < 0.2] = -1
    T = 0.4 + 0.8 * torch.rand(rows, generator=torch.Generator().manual_seed(5)).to(DEV)
    g, h = randn(rows, 1), randn(rows, 2)
    r = scorer.token_logprobs(z, tokens, temperature=T)
    both = scorer.token_logprobs_backward(z, tokens, g, h, temperature=T)
    one = scorer.token_logprobs_backward(z, tokens, g, None, temperature=T)
    _, _, old, ref, adv = policy_inputs(scorer, rows, 8, F32, 5)
    lp, H = r
    old = (lp + 0.2 * randn(rows, 3)).contiguous()
    p = scorer.policy_loss(z, tokens, old, adv, temperature=T, scale=0.01,
                           **dict(POLICY, kl_coef=0.0))
    for lo in range(0, rows, 128):
        at = slice(lo, lo + 128)
        zb, tb, Tb = z[at], tokens[at], T[at]
        check_scores(type(r)(lp[at], H[at]), zb, Tb, tb)
        check_scores(type(r)(p.logprobs[at], p.entropies[at]), zb, Tb, tb)
        R.check_gradient(both[at], *R.gradient(zb, Tb, tb, g[at], h[at]), dtype)
        R.check_gradient(one[at], *R.gradient(zb, Tb, tb, g[at], None), dtype)
    # the policy's gradient is that of its own factors
    ratio = torch.exp(lp.double() - old.double())
    free = -adv.double() * ratio
    cut = -adv.double() * ratio.clamp(0.8, 1.28) > free
    gp = torch.where((tokens >= 0) & ~cut, 0.01 * free, 0.0).float()
    hp = torch.full_like(gp, -0.01 * POLICY["entropy_coef"])
    d = scorer.token_logprobs_backward(z, tokens, gp, hp, temperature=T)
    # Apart by the gradients' own roundings, and by the factor's: the ratio here
    # comes from log p_a as written (half a step of its fp32 value, and what
    # two summation orders leave), and the factor is rounded a few times; an
    # element is at most factor / T.
    tl = torch.cat([R.logprob_tol(z[lo:lo + 128], T[lo:lo + 128], tokens[lo:lo + 128])[0]
                    for lo in range(0, rows, 128)])
    rel = torch.where(tokens >= 0, R.U * lp.double().abs() + 2 * tl + 16 * R.U, 0.0)
    bound = (gp.double().abs() * rel / T.double())[:, None] \
        + 4 * R.half_step(dtype) * d.double().abs() + 2.0 ** -120
    assert ((p.d_logits.double() - d.double()).abs() <= bound).all()
    assert scorer.status() == 0


@pytest.mark.parametrize("ignored", ["scattered", "head", "all but one", "all", "none"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_long_calls_share_out_their_live_rows(scorer, dtype, ignored):
    """Enough rows that they are shared out by lists of live and ignored ones:
    each row's results are its own, wherever the ignored ones lie."""
    rows, V = 2050, 131072 if dtype is BF16 else 65601
    z, tokens, _ = R.make_logits(rows, V, dtype, 17, DEV)
    keep = torch.ones(rows, dtype=torch.bool)
    if ignored == "scattered":
        keep = torch.rand(rows, generator=torch.Generator().manual_seed(4)) < 0.7
    elif ignored == "head":
        keep[:611] = False
    elif ignored != "none":
        keep[:] = False
        keep[777] = ignored == "all but one"
    tokens = torch.where(keep.to(DEV), tokens, -1)
    g = randn(rows, 1)
    weights = torch.where(keep.to(DEV), 1.0, 0.0)
    _, _, old, _, adv = policy_inputs(scorer, rows, 8, F32, 5)
    r = scorer.token_logprobs(z, tokens, temperature=0.8)
    d = scorer.token_logprobs_backward(z, tokens, g, temperature=0.8)
    p = scorer.policy_loss(z, tokens.clamp(min=0), old, adv, weights=weights, temperature=0.8,
                           entropy_coef=0.01, scale=0.01)
    for lo in range(0, rows, 128):
        at = slice(lo, lo + 128)
        check_scores(type(r)(r.logprobs[at], r.entropies[at]), z[at], 0.8, tokens[at])
        check_scores(type(r)(p.logprobs[at], p.entropies[at]), z[at], 0.8, tokens[at])
        R.check_gradient(d[at], *R.gradient(z[at], 0.8, tokens[at], g[at], None), dtype)
    gone = (~keep).to(DEV)
    assert (p.d_logits[gone] == 0).all()
    # the same bits again
    q = scorer.policy_loss(z, tokens.clamp(min=0), old, adv, weights=weights, temperature=0.8,
                           entropy_coef=0.01, scale=0.01)
    assert torch.equal(p.terms, q.terms) and torch.equal(p.d_logits, q.d_logits)
    assert scorer.status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_gradient_equals_the_separate_one(scorer, dtype):
    for rows, V in ((5, 1000), (40, 32003), (3, 262144)):
        z, tokens, _ = R.make_logits(rows, V, dtype, V, DEV)
        g, h = randn(rows, 1), randn(rows, 2)
        d = scorer.token_logprobs_backward(z, tokens, g, h, temperature=0.7)
        w = z.contiguous().clone()
        assert scorer.token_logprobs_backward(w, tokens, g, h, temperature=0.7, out=w) is w
        assert torch.equal(w, d)


def test_three_dimensional_logits_are_rows(scorer):
    z, tokens, _ = R.make_logits(32, 1000, BF16, 3, DEV)
    a = scorer.token_logprobs(z, tokens)
    b = scorer.token_logprobs(z.contiguous().view(2, 16, 1000), tokens.view(2, 16))
    assert torch.equal(a.logprobs, b.logprobs) and torch.equal(a.entropies, b.entropies)
    d = scorer.token_logprobs_backward(z.contiguous().view(2, 16, 1000), tokens, randn(32, 1))
    assert d.shape == (2, 16, 1000)


POLICY = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, entropy_coef=0.02)


def policy_inputs(scorer, rows, V, dtype, seed):
    z, tokens, _ = R.make_logits(rows, V, dtype, seed, DEV)
    lp, _ = R.scores(z, 0.8, tokens)
    old = (lp + 0.3 * randn(rows, seed + 1)).float()
    ref = (lp + 0.3 * randn(rows, seed + 2)).float()
    adv = randn(rows, seed + 3)
    return z, tokens, old, ref, adv


def check_policy(r, z, T, tokens, old, adv, ref, weights, scale, kw, dtype, grad=True):
    terms, size, lp, H, g, h, keep = R.policy(
        z, T, tokens, old, adv, ref, weights, kw["clip_low"], kw["clip_high"], kw["kl_coef"],
        kw["entropy_coef"], scale)
    check_scores(r, z, T, tokens, keep)
    tl, _ = R.logprob_tol(z, T, tokens)
    # a ratio's relative error is log p_a's absolute one, and its exp's and rounding
    rel = float(tl[keep].max()) * 2 + 16 * R.U if keep.any() else 0.0
    assert ((r.terms.double() - terms).abs() <= rel * size * 4 + 4 * R.U * size).all(), \
        (r.terms, terms)
    if grad:
        d, tol = R.gradient(z, T, torch.where(keep, tokens, -1), g, h)
        gl = (g.abs() + abs(kw["kl_coef"] * scale))[:, None] * rel
        p = torch.softmax(z.double() / (T.double()[:, None] if torch.is_tensor(T) else T), 1)
        a = tokens.clamp(min=0, max=z.shape[1] - 1).long()[:, None]
        one = torch.zeros_like(p).scatter_(1, a, 1.0)
        iT = 1.0 / (T.double()[:, None] if torch.is_tensor(T) else T)
        tol = tol + torch.where(keep[:, None], gl * (p - one).abs() * iT * 1.01, 0.0)
        R.check_gradient(r.d_logits, d, tol, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [(1, 1), (1, 1000), (16, 1024), (301, 2049), (37, 32003),
                                    (1500, 129), (4, 262144)])
def test_policy_loss_and_gradient(scorer, dtype, rows, V):
    z, tokens, old, ref, adv = policy_inputs(scorer, rows, V, dtype, rows + V)
    scale = 1.0 / rows
    r = scorer.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8, scale=scale,
                           **POLICY)
    check_policy(r, z, 0.8, tokens, old, adv, ref, None, scale, POLICY, dtype)
    alone = scorer.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8,
                               scale=scale, grad=False, **POLICY)
    assert alone.d_logits is None
    check_policy(alone, z, 0.8, tokens, old, adv, ref, None, scale, POLICY, dtype, grad=False)
    again = scorer.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8,
                               scale=scale, **POLICY)
    assert all(torch.equal(x, y) for x, y in zip(r, again))


@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_weights_masks_and_no_reference(scorer, dtype):
    rows, V = 203, 4099
    z, tokens, old, ref, adv = policy_inputs(scorer, rows, V, dtype, 4)
    z, tokens, weights = z.clone(), tokens.clone(), 0.5 + randn(rows, 9).abs()
    tokens[::7] = -1
    weights[1::7] = 0.0
    for t in (old, adv):          # what an ignored row holds is not used
        t[::7] = math.nan
        t[1::7] = math.inf
    z[::7] = math.nan
    z[1::7] = math.inf
    T = 0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(1)).to(DEV)
    lp, _ = R.scores(torch.nan_to_num(z.float(), nan=0.0, posinf=0.0), T, tokens)
    old = torch.where(torch.isfinite(old), (lp + 0.2 * randn(rows, 10)).float(), old)
    kw = dict(POLICY, kl_coef=0.0)
    r = scorer.policy_loss(z, tokens, old, adv, weights=weights, temperature=T, scale=0.25, **kw)
    clean = z.clone()
    clean[::7] = 0
    clean[1::7] = 0
    check_policy(r, clean, T, tokens, old, adv, None, weights, 0.25, kw, dtype)
    assert float(r.terms[2]) == 0.0
    assert scorer.status() == 0
    # nothing counts: all zeros
    r = scorer.policy_loss(z, torch.full_like(tokens, -1), old, adv, temperature=T, **kw)
    assert (r.terms == 0).all() and (r.d_logits == 0).all() and (r.logprobs == 0).all()


def test_policy_of_no_rows(scorer):
    z = torch.zeros((0, 100), device=DEV)
    e = torch.zeros(0, device=DEV)
    t = torch.zeros(0, dtype=torch.int32, device=DEV)
    r = scorer.policy_loss(z, t, e, e)
    assert (r.terms == 0).all() and r.d_logits.shape == (0, 100)
    assert scorer.token_logprobs(z, t).logprobs.shape == (0,)
    assert scorer.token_logprobs_backward(z, t, e).shape == (0, 100)


def test_policy_gradient_against_differences(scorer):
    """Central differences of the 64-bit loss in random directions (fp32
    logits): (L(z + e u) - L(z - e u)) / 2e = <d_logits, u> + O(e^2)."""
    rows, V = 12, 50
    z, tokens, old, ref, adv = policy_inputs(scorer, rows, V, F32, 21)
    r = scorer.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8, scale=0.5,
                           **POLICY)
    step = 1e-5
    for k in range(4):
        u = torch.randn((rows, V), generator=torch.Generator().manual_seed(k),
                        dtype=torch.float64).to(DEV)
        both = [R.policy(z.double() + s * step * u, 0.8, tokens, old, adv, ref, None, 0.2, 0.28,
                         0.05, 0.02, 0.5)[0][0] for s in (1, -1)]
        slope = float((both[0] - both[1]) / (2 * step))
        got = float((r.d_logits.double() * u).sum())
        # third derivatives of the loss along u: below 1e3 |u|^3 here, times e^2
        assert abs(slope - got) < 1e-6 * float(u.abs().sum()), (slope, got)


PREF = dict(beta=0.2, label_smoothing=0.1, margin=0.05)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("lengths,V,tail", [
    ([1, 1], 1000, 0), ([3, 0, 5, 2], 513, 4), ([0, 0], 64, 2), ([40, 33, 1, 17, 29, 40], 2048, 0),
    ([7, 300, 260, 1], 1001, 3), ([2, 3], 262144, 1)])
def test_preference_loss_and_gradient(scorer, dtype, average, lengths, V, tail):
    lead = 2  # rows before the first sequence
    rows = lead + sum(lengths) + tail
    z, tokens, _ = R.make_logits(rows, V, dtype, rows + V, DEV)
    z, tokens = z.clone(), tokens.clone()
    off = [lead]
    for n in lengths:
        off.append(off[-1] + n)
    tokens[lead + 1:off[-1]:4] = -1
    inside = torch.zeros(rows, dtype=torch.bool, device=DEV)
    inside[lead:off[-1]] = True
    clean = z.clone()
    z[~inside] = math.nan        # rows outside the sequences are not read
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    masked = torch.where(inside, tokens, -1)
    lp, _ = R.scores(clean, 0.9, masked)
    P = len(lengths) // 2
    _, _, S, _ = R.preference(lp, masked, offsets, None, average=average, scale=1.0,
                              beta=0.2, smooth=0.1, margin=0.05)
    ref = (S + randn(2 * P, 3)).float()
    for reference in (ref, None):
        r = scorer.preference_loss(z, tokens, offsets, ref_logprobs=reference, average=average,
                                   temperature=0.9, scale=0.5, **PREF)
        loss, losses, S, g = R.preference(lp, masked, offsets, reference, 0.2, 0.1, 0.05,
                                          average, 0.5)
        tl, _ = R.logprob_tol(clean, 0.9, masked)
        tl = torch.where(masked >= 0, tl, 0.0)
        assert ((r.logprobs.double() - lp).abs() <= tl).all()
        # a sequence's sum: its rows' errors, one rounding; a margin: beta times two sums'
        tS = tl.sum() + R.U * S.abs()
        assert ((r.sequence_logprobs.double() - S).abs() <= tS).all()
        tm = 0.2 * 2 * float(tl.sum()) + 1e-12
        assert ((r.losses.double() - losses).abs() <= tm + R.U * losses.abs()).all()
        assert abs(float(r.loss) - float(loss)) <= 0.5 * P * tm + 4 * R.U * abs(float(loss))
        d, tol = R.gradient(clean, 0.9, masked, g, None)
        tol = tol + d.abs() * (tm + 2 * R.U)  # |d sigmoid| <= sigmoid
        tol = tol + 0.5 * 0.2 * 0.1 * tm * (d != 0)  # the smoothed part
        R.check_gradient(r.d_logits, d, tol, dtype)
        assert (r.d_logits[~inside] == 0).all()
        alone = scorer.preference_loss(z, tokens, offsets, ref_logprobs=reference,
                                       average=average, temperature=0.9, scale=0.5, grad=False,
                                       **PREF)
        assert alone.d_logits is None and torch.equal(alone.loss, r.loss)
    w = z.clone()
    again = scorer.preference_loss(w, tokens, offsets, average=average, temperature=0.9,
                                   scale=0.5, out=w, **PREF)
    assert torch.equal(again.d_logits, r.d_logits)  # in place: the same bits
    assert scorer.status() == 0


def test_preference_extremes(scorer):
    """Margins far out on both sides, a banned token, no pairs."""
    z = torch.zeros((4, 10), device=DEV)
    z[:, 0] = 60.0
    tokens = torch.tensor([0, 1, 1, 0], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=DEV)
    r = scorer.preference_loss(z, tokens, off, beta=50.0)
    # margins of +3000 and -3000: losses 0 and 3000, gradient 0 and full
    assert float(r.losses[0]) == 0.0 and abs(float(r.losses[1]) - 3000.0) < 1e-3
    assert (r.d_logits[0] == 0).all() and (r.d_logits[2] == 0).all()
    assert abs(float(r.d_logits[1, 1]) + 50.0) < 1e-4
    z[2, 1] = -math.inf  # the first pair's rejected token cannot be drawn
    r = scorer.preference_loss(z, tokens, off, beta=0.1)
    assert float(r.losses[0]) == 0.0 and float(r.sequence_logprobs[2]) == -math.inf
    none = scorer.preference_loss(z, tokens, off[:1])
    assert float(none.loss) == 0.0 and (none.d_logits == 0).all()
    assert scorer.status() == 0


def test_bad_offsets_are_reported_and_stay_inside(scorer):
    z, tokens, _ = R.make_logits(8, 100, F32, 2, DEV)
    for bad in ([0, 4, 2], [0, 4, 9], [-3, 4, 8], [5, 5, 4]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        r = scorer.preference_loss(z, tokens, off)
        assert torch.isnan(r.loss).all() and torch.isnan(r.losses).all(), bad
        assert scorer.status(clear=True) & 8
    good = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    assert torch.isfinite(scorer.preference_loss(z, tokens, good).loss).all()
    assert scorer.status() == 0


@pytest.mark.parametrize("rows,pairs", [(512, 64), (513, 3), (130, 65), (512, 1)])
def test_few_and_many_pairs(scorer, rows, pairs):
    """One pair to many: the losses, their factors, and a pair out of order among
    good ones."""
    z, tokens, _ = R.make_logits(rows, 700, F32, 5, DEV)
    cuts = torch.linspace(0, rows, 2 * pairs + 1).int()
    lp, _ = R.scores(z, 0.7, tokens)
    off = cuts.to(DEV)
    r = scorer.preference_loss(z, tokens, off, temperature=0.7, **PREF)
    loss, losses, S, g = R.preference(lp, tokens, off, None, 0.2, 0.1, 0.05, False, 1.0)
    tl, _ = R.logprob_tol(z, 0.7, tokens)
    tm = 0.2 * 2 * float(tl.sum()) + 1e-12
    assert ((r.losses.double() - losses).abs() <= tm + R.U * losses.abs()).all()
    assert abs(float(r.loss) - float(loss)) <= pairs * tm + 4 * R.U * abs(float(loss))
    d, tol = R.gradient(z, 0.7, tokens, g, None)
    R.check_gradient(r.d_logits, d, tol + d.abs() * (tm + 2 * R.U) + 0.2 * 0.1 * tm * (d != 0), F32)
    wrong = cuts.clone()
    wrong[1] = rows + 1  # the first sequence's end: out of range, the second's start too
    r2 = scorer.preference_loss(z, tokens, wrong.to(DEV), temperature=0.7, **PREF)
    assert scorer.status(clear=True) & 8
    assert torch.isnan(r2.loss).all() and torch.isnan(r2.losses[0])
    assert torch.equal(r2.losses[2:], r.losses[2:])
    assert torch.equal(scorer.preference_loss(z, tokens, off, temperature=0.7, **PREF).loss, r.loss)
    assert scorer.status() == 0


@pytest.mark.parametrize("rows,V,d", [(1, 1, 8), (1, 256, 64), (3, 255, 72), (24, 1000, 128),
                                      (128, 513, 200), (129, 4096, 64), (300, 5000, 264),
                                      (257, 2047, 2560), (600, 32003, 128), (2, 70001, 64),
                                      (32, 1001, 1032), (33, 128, 64), (50, 3000, 2056),
                                      (64, 40001, 96), (65, 300, 1096), (128, 40001, 2560), (100, 255, 520),
                                      (383, 3001, 600), (1300, 2100, 72), (1500, 700, 136)])
def test_lmhead_scores(scorer, rows, V, d):
    """Codes over 8: the products' fp32 sums are exact, so the logits are the
    64-bit ones and only the softmax rounds."""
    g = torch.Generator().manual_seed(rows + V + d)
    w = torch.randint(-2, 3, (V, d), generator=g).float() / 8
    h = torch.randint(-2, 3, (rows, d), generator=g).float() / 8
    tokens = torch.randint(0, V, (rows,), generator=g)
    h[::2] = w[tokens[::2]]
    w, h = w.to(DEV), h.to(DEV)
    tokens = tokens.to(torch.int32).to(DEV)
    z = h.double() @ w.double().T
    if rows > 4:
        tokens[::6] = -1
    T = 0.3 + torch.rand(rows, generator=g).to(DEV)
    for temp in (0.6, T):
        r = scorer.lmhead_logprobs(h.to(BF16), w.to(BF16), tokens, temperature=temp)
        check_scores(r, z, temp, tokens)
        again = scorer.lmhead_logprobs(h.to(BF16), w.to(BF16), tokens, temperature=temp)
        assert torch.equal(r.logprobs, again.logprobs)
        assert torch.equal(r.entropies, again.entropies)
    alone = scorer.lmhead_logprobs(h.to(BF16), w.to(BF16), tokens, temperature=T,
                                   entropies=False)
    assert alone.entropies is None and torch.equal(alone.logprobs, r.logprobs)
    assert scorer.status() == 0


def test_lmhead_scores_of_random_values(scorer):
    """General bf16 inputs: each logit within gamma_d sum |h w|, so log p_a
    within twice its row's largest."""
    g = torch.Generator().manual_seed(5)
    rows, V, d = 200, 3000 + 7, 520
    h = torch.randn((rows, d), generator=g).to(BF16).to(DEV)
    w = (0.1 * torch.randn((V, d), generator=g)).to(BF16).to(DEV)
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32).to(DEV)
    z = h.double() @ w.double().T
    off = d * R.U * (h.double().abs() @ w.double().abs().T).amax(1) / 0.8
    r = scorer.lmhead_logprobs(h, w, tokens, temperature=0.8)
    lp, H = R.scores(z, 0.8, tokens)
    tl, th = R.logprob_tol(z, 0.8, tokens)
    assert ((r.logprobs.double() - lp).abs() <= tl + 2 * off).all()
    assert ((r.entropies.double() - H).abs() <= th + 2 * off * (1 + H) * 2).all()


def test_lmhead_bad_values_stay_in_their_rows(scorer):
    g = torch.Generator().manual_seed(6)
    h = torch.randn((6, 64), generator=g).to(BF16).to(DEV)
    w = torch.randn((700, 64), generator=g).to(BF16).to(DEV)
    tokens = torch.tensor([3, 700, 5, -1, 699, 0], dtype=torch.int32, device=DEV)
    clean = scorer.lmhead_logprobs(h, w, tokens)
    h[0, 3] = math.nan
    h[3, 0] = math.inf
    r = scorer.lmhead_logprobs(h, w, tokens)
    assert torch.isnan(r.logprobs[:2]).all() and torch.isnan(r.entropies[0])
    assert float(r.logprobs[3]) == 0.0
    for i in (2, 4, 5):
        assert r.logprobs[i] == clean.logprobs[i] and r.entropies[i] == clean.entropies[i]
    assert scorer.status(clear=True) == 1 | 2


def test_captured_calls_replay_on_new_inputs(E):
    sc = E.EBScorer(512, device=DEV)
    rows, V = 64, 4100
    z, tokens, old, ref, adv = policy_inputs(sc, rows, V, BF16, 7)
    z = z.contiguous()
    off = torch.tensor([0, 20, 30, 50, 64], dtype=torch.int32, device=DEV)
    h = torch.randn((rows, 128), device=DEV).to(BF16)
    w = torch.randn((V, 128), device=DEV).to(BF16)

    def calls():
        a = sc.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8, **POLICY)
        b = sc.preference_loss(z, tokens, off, **PREF)
        c = sc.token_logprobs(z, tokens)
        d = sc.token_logprobs_backward(z, tokens, adv, old)
        e = sc.lmhead_logprobs(h, w, tokens)
        return [*a, *b, *c, d, *e]

    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = calls()
    for seed in (1, 2):
        z.copy_(R.make_logits(rows, V, BF16, seed, DEV)[0])
        tokens.copy_(R.make_logits(rows, V, BF16, seed, DEV)[1])
        h.normal_()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, want))
    assert sc.status() == 0
    sc.close()


def test_two_scorers_on_two_streams(E):
    """Handles share nothing: calls in flight together give the bits of calls
    alone."""
    a, b = E.EBScorer(600, device=DEV), E.EBScorer(600, device=DEV)
    rows, V = 500, 8200
    x = policy_inputs(a, rows, V, BF16, 1)
    y = policy_inputs(b, rows, V, F32, 2)

    def call(sc, v):
        z, tokens, old, ref, adv = v
        return sc.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8, **POLICY)

    want = call(a, x), call(b, y)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    got = [None, None]
    for _ in range(4):
        for i, (sc, v) in enumerate(((a, x), (b, y))):
            with torch.cuda.stream(streams[i]):
                got[i] = call(sc, v)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))
    a.close()
    b.close()


@pytest.mark.parametrize("dtype,V", [(F32, 1000003), (BF16, 3000001)])
def test_rows_longer_than_the_rings(scorer, dtype, V):
    """A row of several megabytes: its shares are copied twice on every cluster."""
    rows = 3
    z, tokens, _ = R.make_logits(rows, V, dtype, 9, DEV, shift=1)
    g, h = randn(rows, 1), randn(rows, 2)
    check_scores(scorer.token_logprobs(z, tokens, temperature=0.9), z, 0.9, tokens)
    for gh in (h, None):
        d = scorer.token_logprobs_backward(z, tokens, g, gh, temperature=0.9)
        R.check_gradient(d, *R.gradient(z, 0.9, tokens, g, gh), dtype)
    z[1, 5:V - 3] = -math.inf
    tokens[1] = V - 1
    d = scorer.token_logprobs_backward(z, tokens, g, h, temperature=0.9)
    R.check_gradient(d, *R.gradient(z, 0.9, tokens, g, h), dtype)
    assert scorer.status() == 0


@pytest.mark.parametrize("V", [1000, 40000])
def test_offsets_past_32_bits(scorer, V):
    """Rows 1.2e9 elements apart: the last one starts 2.4e9 elements in."""
    rows, ld = 3, 1200000007
    buf = torch.empty(2 * ld + V + 8, dtype=BF16, device=DEV)
    z = buf.as_strided((rows, V), (ld, 1), 0)
    src, tokens, _ = R.make_logits(rows, V, BF16, 3, DEV)
    for i in range(rows):
        z[i].copy_(src[i])
    near = scorer.token_logprobs(src, tokens, temperature=0.7)
    far = scorer.token_logprobs(z, tokens, temperature=0.7)
    assert (near.logprobs - far.logprobs).abs().max() < 1e-5
    g = randn(rows, 1)
    want = scorer.token_logprobs_backward(src, tokens, g, g, temperature=0.7)
    got = scorer.token_logprobs_backward(z, tokens, g, g, temperature=0.7, out=z)
    assert got is z
    ref, tol = R.gradient(src, 0.7, tokens, g, g)
    R.check_gradient(torch.stack([z[i] for i in range(rows)]), ref, tol, BF16)
    R.check_gradient(want, ref, tol, BF16)
    off = torch.tensor([0, 2, 3], dtype=torch.int32, device=DEV)
    for i in range(rows):
        z[i].copy_(src[i])
    a = scorer.preference_loss(src, tokens, off)
    b = scorer.preference_loss(z, tokens, off, out=z)
    assert abs(float(a.loss) - float(b.loss)) < 1e-5
    assert (a.d_logits.float() - torch.stack([z[i] for i in range(rows)]).float()).abs().max() < 1e-3


def test_a_wait_that_runs_out_is_reported(E):
    """With a limit of 1 ns the first wait for a copy gives up: the status word
    says so, no result passes for a good one, and the next calls are right."""
    sc = E.EBScorer(512, device=DEV)
    z, tokens, old, ref, adv = policy_inputs(sc, 300, 20000, BF16, 3)
    h = torch.randn((300, 256), generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    w = torch.randn((5000, 256), generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    t = tokens % 5000

    def calls():
        p = sc.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8, **POLICY)
        return [p.terms, p.logprobs, p.d_logits, sc.lmhead_logprobs(h, w, t).logprobs,
                sc.lmhead_logprobs(h[:20], w, t[:20]).logprobs]

    want = calls()
    assert sc.status() == 0
    sc.set_wait_limit(1)
    terms = sc.policy_loss(z, tokens, old, adv, ref_logprobs=ref, temperature=0.8,
                           **POLICY).terms
    assert sc.status(clear=True) & E.STATUS_TIMEOUT
    assert torch.isnan(terms).all()
    lp = sc.lmhead_logprobs(h, w, t).logprobs
    assert sc.status(clear=True) & E.STATUS_TIMEOUT
    assert torch.isnan(lp).any()
    lp = sc.lmhead_logprobs(h[:20], w, t[:20]).logprobs
    assert sc.status(clear=True) & E.STATUS_TIMEOUT
    assert torch.isnan(lp).all()
    sc.set_wait_limit(0)
    got = calls()
    assert sc.status() == 0
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    sc.close()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,V", [(300, 20001), (40, 262144), (1003, 131072)])
def test_a_pass_cut_short_leaves_nan(E, dtype, rows, V):
    """Rows that a pass did not reach hold NaN, not what was in the buffers
    before: each row's results are the right ones, or NaN where a wait was
    reported.  (A wait tests its barrier once whatever its limit, and
    that test may last until the copy has come: whether a given wait gives up
    is not promised.)"""
    sc = E.EBScorer(rows, device=DEV)
    z, tokens, _ = R.make_logits(rows, V, dtype, 9, DEV)
    g = randn(rows, 1)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV)
    want = sc.token_logprobs(z, tokens)
    d = sc.token_logprobs_backward(z, tokens, g)
    assert sc.status() == 0

    def right_or_nan(got, ref):
        nan = torch.isnan(got).view(rows, -1).any(1)
        assert torch.equal(nan, ~(got == ref).view(rows, -1).all(1))
        assert sc.status(clear=True) & E.STATUS_TIMEOUT or not nan.any()

    sc.set_wait_limit(1)
    stale = [torch.full((rows,), 7.0, device=DEV) for _ in range(4)]
    del stale  # the results' memory, as the allocator hands it out next
    lp, H = sc.token_logprobs(z, tokens)
    assert torch.equal(torch.isnan(lp), torch.isnan(H))
    assert torch.equal(H[~torch.isnan(H)], want.entropies[~torch.isnan(H)])
    right_or_nan(lp, want.logprobs)
    out = torch.full_like(d, 7.0)
    right_or_nan(sc.token_logprobs_backward(z, tokens, g, out=out), d)
    r = sc.preference_loss(z, tokens, off, out=out.fill_(7.0))
    sc.status(clear=True)
    left = torch.isnan(r.logprobs).any()
    assert torch.isnan(r.loss).all() == left and torch.isnan(r.losses).all() == left
    assert torch.isnan(r.d_logits).any(1).all() == left  # the pair's factor is NaN
    assert (r.d_logits != 7.0).all(1).all()
    sc.set_wait_limit(0)
    again = sc.token_logprobs(z, tokens)
    assert torch.equal(again.logprobs, want.logprobs) and sc.status() == 0
    sc.close()


def test_refusals(E, scorer):
    z = torch.zeros((4, 64), device=DEV)
    t = torch.zeros(4, dtype=torch.int32, device=DEV)
    f = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        scorer.token_logprobs(z.half(), t)
    with pytest.raises(TypeError):
        scorer.token_logprobs(z, t.long())
    with pytest.raises(ValueError):
        scorer.token_logprobs(z, t[:3])
    with pytest.raises(ValueError):
        scorer.token_logprobs(z.T, torch.zeros(64, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        scorer.token_logprobs(z.cpu(), t)
    with pytest.raises(ValueError):
        scorer.token_logprobs(z[:1].expand(4, 64), t)
    with pytest.raises(ValueError):
        scorer.token_logprobs(z[0], t)
    for T in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(E.EBError):
            scorer.token_logprobs(z, t, temperature=T)
    with pytest.raises(E.EBError):
        scorer.token_logprobs(torch.zeros((scorer.max_rows + 1, 2), device=DEV),
                              torch.zeros(scorer.max_rows + 1, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        scorer.token_logprobs_backward(z, t, f, out=torch.zeros((4, 63), device=DEV))
    with pytest.raises(ValueError):
        scorer.token_logprobs_backward(z, t, f, out=torch.zeros((4, 64), dtype=BF16, device=DEV))
    with pytest.raises(E.EBError):
        scorer.policy_loss(z, t, f, f, kl_coef=0.1)      # no reference
    with pytest.raises(E.EBError):
        scorer.policy_loss(z, t, f, f, clip_low=1.5)
    with pytest.raises(E.EBError):
        scorer.policy_loss(z, t, None, f)
    with pytest.raises(ValueError):
        scorer.preference_loss(z, t, torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(E.EBError):
        scorer.preference_loss(z, t, torch.zeros(3, dtype=torch.int32, device=DEV),
                               label_smoothing=1.0)
    h, w = torch.zeros((4, 12), dtype=BF16, device=DEV), torch.zeros((9, 12), dtype=BF16,
                                                                     device=DEV)
    with pytest.raises(E.EBError):
        scorer.lmhead_logprobs(h, w, t)                  # d not a multiple of 8
    with pytest.raises(ValueError):
        scorer.lmhead_logprobs(h.float(), w, t)
    with pytest.raises(ValueError):
        scorer.lmhead_logprobs(h[:, :8], w, t)
    assert scorer.status() == 0


@pytest.mark.parametrize("kw", [dict(temperature=1e-60), dict(temperature=1e60),
                                dict(entropy_coef=1e60), dict(clip_high=1e60),
                                dict(kl_coef=-1e60)])
def test_values_past_fp32_are_refused(E, scorer, kw):
    """Finite in 64 bits, but 0 or infinite as the fp32 the kernels use."""
    z = torch.zeros((4, 64), device=DEV)
    t = torch.zeros(4, dtype=torch.int32, device=DEV)
    f = torch.zeros(4, device=DEV)
    with pytest.raises(E.EBError):
        scorer.policy_loss(z, t, f, f, ref_logprobs=f, **kw)
    if "temperature" in kw:
        h = torch.zeros((4, 8), dtype=BF16, device=DEV)
        with pytest.raises(E.EBError):
            scorer.lmhead_logprobs(h, torch.zeros((9, 8), dtype=BF16, device=DEV), t, **kw)
    assert scorer.status() == 0


def test_a_trajectory_is_sampled_scored_and_learned_from(E):
    """As the pieces are used together: a canvas is sampled, its committed
    tokens scored at their step's temperature (from logits and from hidden
    states), then a policy step and a preference step take their gradients."""
    B, L, V, d = 2, 16, 1024, 64
    eb = E.EBSampler(B, L, V, device=DEV, num_steps=4, seed=3)
    sc = E.EBScorer(256, device=DEV)
    canvas, committed, stop = eb.new_canvas()
    H, amax = eb.outputs()
    g = torch.Generator().manual_seed(4)
    weight = (torch.randint(-2, 3, (V, d), generator=g).float() / 8).to(BF16).to(DEV)
    hidden = (torch.randint(-2, 3, (B * L, d), generator=g).float() / 8).to(BF16).to(DEV)
    logits = E.lmhead_logits(hidden, weight).view(B, L, V)
    eb.step(logits, 0, canvas, committed, H, amax, stop)
    T0 = eb.cfg.t_max
    tokens = torch.where(committed.bool(), canvas, -1).reshape(-1)
    assert (tokens >= 0).any()
    r = sc.token_logprobs(logits, tokens, temperature=T0)
    live = tokens >= 0
    # the step's entropies are those of the committed rows
    assert (r.entropies - H.reshape(-1)).abs()[live].max() < 1e-4
    lm = sc.lmhead_logprobs(hidden, weight, tokens, temperature=T0)
    check_scores(lm, logits.view(-1, V), T0, tokens)
    check_scores(r, logits.view(-1, V), T0, tokens)

    # one gradient step on the logits with a positive advantage raises the tokens' probability
    adv = torch.ones(B * L, device=DEV)
    p = sc.policy_loss(logits, tokens, r.logprobs, adv, temperature=T0, clip_high=10.0)
    assert torch.equal(p.logprobs, r.logprobs)
    z = (logits - 0.1 * p.d_logits).contiguous()
    assert (sc.token_logprobs(z, tokens, temperature=T0).logprobs > r.logprobs)[live].all()

    # through autograd: the head's weight gets the gradient of the formula
    wf = weight.double().requires_grad_()
    zf = hidden.double() @ wf.T
    zf.backward(p.d_logits.view(-1, V).double())
    logp = torch.log_softmax(hidden.double() @ (w2 := weight.double().requires_grad_()).T / T0, 1)
    pick = logp[torch.arange(B * L, device=DEV), tokens.clamp(min=0).long()]
    (-(torch.exp(pick - r.logprobs.double()) * live)).sum().backward()
    err = (wf.grad - w2.grad).norm() / w2.grad.norm()
    assert err < 1e-5

    off = torch.tensor([0, L, 2 * L], dtype=torch.int32, device=DEV)
    q = sc.preference_loss(logits, tokens, off, temperature=T0)
    chosen = r.logprobs[:L].double().sum()
    rejected = r.logprobs[L:].double().sum()
    want = torch.nn.functional.softplus(-0.1 * (chosen - rejected))
    assert abs(float(q.loss) - float(want)) < 1e-5
    assert sc.status() == 0 and eb.status() == 0
    sc.close()
    eb.close()
