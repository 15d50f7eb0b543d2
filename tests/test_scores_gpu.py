"""Scores of logits on the GPU against 64 bits.

Tolerances: S is a sum of V positive fp32 terms, each within 2^-22 (the exponential) + 2^-24 |x - m|
log2(e) (its argument, two roundings) of exact; terms of |x - m| < 32 matter, so a term's relative
error is below 2^-22 + 2^-18.4 at the far end but those weigh e^-20; over what weighs, |x - m| < 8,
below 2^-20.  Sums of 32 terms per thread, then trees and at most 64 chunks: fewer than 110 roundings
of 2^-24, below 2^-17.2 if all pointed one way; they are independent, their root is 10 2^-24.
    logprob: |err| <= 2^-19 + 2^-23 |value|  (log S's error, then two subtractions)
    entropy: |err| <= 2^-18 (1 + value)      (D / S has the errors of two sums, weighted by |x - m|)
Ids are exact."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import xv as m
    return m


def score(xv, x, tokens, top, n_rows=None, fill=5.0):
    M, V = x.shape
    lp, en = (torch.full((M,), fill, device="cuda") for _ in range(2))
    ids = torch.full((M, top), -7, dtype=torch.int32, device="cuda") if top else None
    tl = torch.full((M, top), fill, device="cuda") if top else None
    ws = xv.workspace(xv.xv_logprobs_workspace_size(M, V, top))
    xv.xv_logprobs(x, tokens, lp, ws, entropy=en, top_ids=ids, top_logprobs=tl, n_rows=n_rows)
    assert not ws[:4096].any()      # the counters are zero between calls
    return lp, en, ids, tl


def order(x, top):
    """The top largest of each row, the lowest index first among equals, NaN last."""
    y = torch.where(x.isnan(), torch.full_like(x, -INF), x).double()
    y = torch.where(x.isnan(), torch.full_like(y, -1e308), torch.where(y == -INF, torch.full_like(y, -1e307), y))
    return torch.sort(y + 0.0, dim=-1, descending=True, stable=True).indices[:, :top].int()


def check(xv, x, tokens, top):
    lp, en, ids, tl = score(xv, x, tokens, top)
    d = x.double()
    full = torch.log_softmax(d, -1)
    ok = (x.float().amax(-1) < INF) & (x.float().amax(-1) > -INF) & ~x.isnan().any(-1)
    near = lambda a, b: ((a.double() - b).abs() <= 2.0 ** -19 + 2.0 ** -23 * b.abs()) | (a.double() == b)   # noqa: E731
    want = full.gather(1, tokens.clamp_min(0).long()[:, None])[:, 0]
    want = torch.where(tokens < 0, torch.zeros_like(want), want)
    assert near(lp, want)[ok].all()
    entropy = -torch.where(full == -INF, torch.zeros_like(full), full.exp() * full).sum(-1)
    assert ((en.double() - entropy).abs() <= 2.0 ** -18 * (1 + entropy))[ok].all()
    if top:
        assert torch.equal(ids, order(x.float(), top))
        assert near(tl, full.gather(1, ids.long()))[ok].all()
    return lp, en, ids, tl


def logits(M, V, dtype, seed=0, sigma=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((M, V), generator=g, device="cuda") * sigma).to(dtype)


def toks(M, V, seed=1):
    return torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 33, 1000, 8191, 8192, 8193, 50257, 151936, 524288])
def test_vocabularies(xv, V, dtype):
    for top in sorted({0, 1, min(V, 2), min(V, 7), min(V, 32)}):
        x, t = logits(3, V, dtype, V + top), toks(3, V)
        t[1] = -1
        check(xv, x, t, top)
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["constant", "masked", "all_but_few", "few_values", "rising", "falling", "large", "tied_top", "clustered"])
def test_rows_of_hard_values(xv, kind, dtype):
    V, top = 20001, 32
    x = logits(4, V, torch.float32, 3)
    if kind == "constant":
        x.fill_(1.25)
    if kind == "masked":                       # all of a chunk and more
        x[:, 3000:] = -INF
    if kind == "all_but_few":
        keep = x[:, [5, 9000, 20000]].clone()
        x.fill_(-INF)
        x[:, [5, 9000, 20000]] = keep
    if kind == "few_values":
        x = torch.round(x)
    if kind == "rising":
        x = torch.arange(V, device="cuda").float().expand(4, V).contiguous() / 1000
    if kind == "falling":
        x = -torch.arange(V, device="cuda").float().expand(4, V).contiguous() / 1000
    if kind == "large":
        x = x + 20000
    if kind == "tied_top":
        x[:, 19000:19100] = 40.0
        x[:, 777] = 40.0
    if kind == "clustered":                    # the largest 4000 are a group of neighbours and its strides
        i = torch.arange(V, device="cuda")
        x[:, ((i // 16) % 64) < 31] += 100
    check(xv, x.to(dtype), toks(4, V), top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", ["finfo.min", -1e36, -1e30, -65504.0])
@pytest.mark.parametrize("M,V", [(4, 20001), (3, 1000), (307, 33333), (2, 524288)])
def test_masks_of_a_finite_low_value(xv, M, V, low, dtype):
    """Masked logits that are finite: whole shares of a warp, parts of one, the row's end, all but a few logits of
    the row, all of it, -inf among them, and rows that lie in several CTAs.  A masked term is 0 in 64 bits, too, so the
    tolerances stay those of the terms that weigh."""
    low = torch.finfo(dtype).min if low == "finfo.min" else torch.tensor(low).to(dtype).item()
    x = logits(M, V, torch.float32, V + 11)
    at = torch.arange(V, device="cuda")
    off = torch.zeros((M, V), dtype=torch.bool, device="cuda")
    for r in range(M):
        kind = r % 7 if M > 4 else (r + V) % 7
        off[r] = ((at >= V // 7), (at // 32) % 8 == 3, at >= V - 50, (at % 997 != 5), at >= 0, at < V // 2, at % 3 == 0)[kind]
    x = x.to(dtype).masked_fill(off, low)
    x[0, V // 3: V // 2] = -INF
    t = toks(M, V)
    check(xv, x, t, 0)
    lp, en, ids, tl = check(xv, x, t, 9)
    assert en.isfinite().all()
    if M > 4 or V == 20001:      # few allowed tokens, more alternatives asked for
        few = torch.full_like(x, low)
        few[:, [3, V // 2, V - 1]] = x[:, [3, V // 2, V - 1]]
        assert check(xv, few, t, 20)[1].isfinite().all()
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("V", [40, 9000])
def test_rows_that_are_empty_or_not_finite(xv, V):
    x = logits(6, V, torch.float32, 4)
    x[0] = -INF
    x[1, 7] = NAN
    x[2, 8] = INF
    x[3] = NAN
    x[4, ::2] = -0.0
    x[4, 1::2] = 0.0
    x[5, : V // 2] = NAN
    t = toks(6, V)
    lp, en, ids, tl = check(xv, x, t, 5)
    assert lp[0] == -INF and en[0] == 0 and (tl[0] == -INF).all()
    for r in (1, 2, 3, 5):
        assert lp[r].isnan() and en[r].isnan() and tl[r].isnan().all(), r
    assert xv.xv_device_check() == 0


def test_all_nan_but_few_candidates(xv):
    """Fewer numbers than alternatives: NaNs follow by index, a number each at chunk ends."""
    x = torch.full((2, 17000), NAN, device="cuda")
    x[0, [3, 8191, 16999]] = torch.tensor([1.0, 5.0, -2.0], device="cuda")
    x[1, 16385:] = -INF
    assert torch.equal(score(xv, x, toks(2, 17000), 32)[2], order(x, 32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_has_the_same_bits_in_any_call(xv, dtype):
    """Rows of an odd vocabulary (every alignment), alone, among others, strided."""
    M, V, top = 9, 30011, 20
    x, t = logits(M, V, dtype, 5), toks(M, V)
    whole = score(xv, x, t, top)
    wide = torch.zeros((M, V + 5), dtype=dtype, device="cuda")[:, 2:V + 2]
    wide.copy_(x)
    for i, part in enumerate(zip(*[score(xv, wide, t, top), whole])):
        assert torch.equal(part[0], part[1]), i
    for r in range(M):
        for a, b in zip(score(xv, x[r:r + 1].clone(), t[r:r + 1], top), whole):
            assert torch.equal(a, b[r:r + 1])


def test_rows_behind_the_count_are_left(xv):
    x, t = logits(6, 20000, torch.float32, 6), toks(6, 20000)
    want = score(xv, x, t, 4)
    for n in (0, 4, 6, 9, -2):
        got = score(xv, x, t, 4, n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        k = min(max(n, 0), 6)
        for a, b in zip(got, want):
            assert torch.equal(a[:k], b[:k])
            assert (a[k:] == (-7 if a.dtype == torch.int32 else 5.0)).all()


def test_tokens_outside_the_vocabulary_are_recorded(xv):
    x = logits(3, 100, torch.float32, 7)
    lp, *_ = score(xv, x, torch.tensor([100, 4, -2], dtype=torch.int32, device="cuda"), 0)
    with pytest.raises(xv.XVError):
        xv.xv_device_check()
    assert lp.isnan().tolist() == [True, False, True]


def test_no_entropy_no_top_and_one_buffer_for_many_sizes(xv):
    ws = xv.workspace(xv.xv_logprobs_workspace_size(64, 200000, 32))
    for M, V, top in ((64, 200000, 32), (3, 151936, 5), (64, 1000, 0), (17, 60000, 1)):
        x, t = logits(M, V, torch.float32, V), toks(M, V)
        lp = torch.zeros(M, device="cuda")
        xv.xv_logprobs(x, t, lp, ws)
        assert torch.equal(lp, score(xv, x, t, 0)[0])


def test_small_calls_before_large_ones_in_one_buffer(xv):
    """What a call leaves in the workspace is nothing that another one counts on."""
    ws = xv.workspace(xv.xv_logprobs_workspace_size(1000, 151936, 32))
    for M, V, top in ((1, 151936, 20), (1000, 20000, 32), (3, 524288, 7), (700, 151936, 1), (2, 16385, 32), (1000, 20000, 5)):
        x, t = logits(M, V, torch.float32, M + V), toks(M, V)
        lp, en = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda")
        ids, tl = torch.zeros((M, top), dtype=torch.int32, device="cuda"), torch.zeros((M, top), device="cuda")
        xv.xv_logprobs(x, t, lp, ws, entropy=en, top_ids=ids, top_logprobs=tl)
        for a, b in zip((lp, en, ids, tl), score(xv, x, t, top)):
            assert torch.equal(a, b), (M, V)
        assert torch.equal(ids, order(x, top))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [150, 151, 303, 305, 457, 613])
def test_rows_over_the_borders_of_ctas(xv, M, dtype):
    """Numbers of rows about the number of CTAs, chunks that do not divide among them."""
    V, top = 33333, 9
    x, t = logits(M, V, dtype, M), toks(M, V)
    check(xv, x, t, top)


def test_captured_and_replayed_on_another_stream(xv):
    M, V, top = 8, 151936, 20
    x, t = logits(M, V, torch.float32, 8), toks(M, V)
    lp, en, tl = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros((M, top), device="cuda")
    ids = torch.zeros((M, top), dtype=torch.int32, device="cuda")
    ws = xv.workspace(xv.xv_logprobs_workspace_size(M, V, top))
    go = lambda: xv.xv_logprobs(x, t, lp, ws, entropy=en, top_ids=ids, top_logprobs=tl)   # noqa: E731
    go()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        go()
    for seed in range(3):
        x.copy_(logits(M, V, torch.float32, 100 + seed))
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            g.replay()
        torch.cuda.default_stream().wait_stream(s)
        for a, b in zip((lp, en, ids, tl), score(xv, x, t, top)):
            assert torch.equal(a, b)


def test_more_than_65535_rows(xv):
    M, V = 70001, 50
    x, t = logits(M, V, torch.bfloat16, 9), toks(M, V)
    check(xv, x, t, 3)
