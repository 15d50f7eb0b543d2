"""The 8-bit KV cache on the GPU: appended codes and scales against the rule in 64 bits, and decode
rows over it against a plain attention in 64 bits, bit for bit against each other where one row is
computed in calls of different shapes.

Tolerance of an attention output (vs the 64-bit value over the same codes), per element:
    |err| <= 2^-8 |ref| + (2^-10 + 2^-12) A,   A = sum_j w_j |V_j|  (w the row's weights)
The output's rounding to bf16 is half a step, 2^-8 of the value at most.  A weight before its product
with V is rounded to fp16 (2^-11; what is cut off below 2^-29 of the largest weight is at most
8192 2^-29 = 2^-16 of A in these lengths).  Its exponent t_j carries the score's errors: q's second e4m3 term
is off by at most 2^-18 of the row's largest value or 2^-9 of the value, whichever is larger, so the
score by 2^-9 sum |q_d k_d| scale at worst and a random walk of hd such terms in fact; for q, k ~
N(0, 1) at hd 64..256 that is 2^-9 0.6 rms(score) sqrt(2) ~ 2^-10 in the weight, and as the errors of
different positions are independent they average out in the sum; 2^-12 is left for the exponentials,
the fp32 sums and the order of both.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HEADS = [(2, 1, 64), (32, 8, 128), (24, 4, 256)]
NAN = float("nan")


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import xv as m
    return m


def dequant(codes, scale):
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


class Cache:
    """Codes and scales of n_pages pages of `page` positions, values of differing sizes per token."""

    def __init__(self, xv, n_pages, Hkv, page, hd, seed=0, outlier=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.ks = self.side(g, n_pages, Hkv, page, hd, False)
        self.v, self.vs = self.side(g, n_pages, Hkv, page, hd, outlier)
        self.q8 = xv.kv_q8(self.k, self.v, self.ks, self.vs)

    @staticmethod
    def side(g, n_pages, Hkv, page, hd, outlier):
        x = torch.randn((n_pages, Hkv, page, hd), generator=g, device="cuda")
        codes = (x * 130).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        spread = torch.randn((n_pages, Hkv, page), generator=g, device="cuda") * (3.0 if outlier else 0.3)
        return codes, torch.exp(spread) / 130


def reference(c, table, q, ctx, counts, R, Hq, Hkv, hd, page, window, sinks, scale, gate=None):
    """[B*R, Hq*hd] in 64 bits, and A of the tolerance; rows behind a sequence's count are 0."""
    B, G = len(ctx), Hq // Hkv
    out = torch.zeros((B, R, Hq, hd), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    rows = q[:, : Hq * hd].reshape(B, R, Hq, hd).double()
    for b in range(B):
        n = counts[b]
        if not n:
            continue
        far = ctx[b] + n - 1
        at = torch.arange(far, device="cuda")
        pg = table[b].long()[at // page]
        for h in range(Hkv):
            k = dequant(c.k[pg, h, at % page], c.ks[pg, h, at % page])
            v = dequant(c.v[pg, h, at % page], c.vs[pg, h, at % page])
            for r in range(n):
                L = ctx[b] + r
                see = at < L
                if window:
                    see &= (at >= L - window) | (at < sinks)
                s = rows[b, r, h * G:(h + 1) * G] @ k[see].T * scale
                p = torch.softmax(s, -1)
                out[b, r, h * G:(h + 1) * G] = p @ v[see]
                mag[b, r, h * G:(h + 1) * G] = p @ v[see].abs()
    if gate is not None:
        s = torch.sigmoid(gate[:, : Hq * hd].double()).reshape(B, R, Hq, hd)
        out, mag = out * s, mag * s
    return out.reshape(B * R, -1), mag.reshape(B * R, -1)


def close(got, ref, mag):
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -12) * mag
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} past the bound, worst " \
        f"{float(((got.double() - ref).abs() / bound.clamp_min(1e-300)).nan_to_num(9e9).max()):.2f} of it"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, max_ctx, window=0, sinks=0, gate=None, counts=None, paged=True,
        fill=0.0, scale=None):
    B = len(ctx)
    out = torch.full((B * R, Hq * hd), fill, dtype=torch.bfloat16, device="cuda")
    ws = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window, sinks))
    kw = dict(window=window, sinks=sinks, gate=gate, n_rows=None if counts is None else i32(counts))
    scale = hd ** -0.5 if scale is None else scale
    if paged:
        xv.xv_attn_decode_rows_q8_paged(q, c.q8, xv.kv_pages(table, page, n_pages), i32(ctx), R, B, Hq, Hkv, hd, max_ctx, scale,
                                        out, ws, **kw)
    else:
        xv.xv_attn_decode_rows_q8(q, c.q8, i32(ctx), R, B, Hq, Hkv, hd, page, max_ctx, scale, out, ws, **kw)
    return out


def normal(shape, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def shuffled(B, per, n_pages, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n_pages, generator=g)[: B * per].to(torch.int32).reshape(B, per).cuda()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("Hkv,hd", [(1, 64), (3, 128), (4, 256)])
@pytest.mark.parametrize("paged", [False, True])
def test_append_codes_and_scales(xv, Hkv, hd, paged):
    B, R, page = 3, 5, 64
    ctx, counts = [1, 62, 130], [5, 4, 0]
    per = 4
    n_pages = B * per + 2 if paged else B
    if not paged:
        page = 203
    table = shuffled(B, per, n_pages, 1) if paged else torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    c = Cache(xv, n_pages, Hkv, page, hd)
    before = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    g = torch.Generator(device="cuda").manual_seed(3)
    src = torch.randn((B * R, 2 * Hkv * hd + 16), generator=g, device="cuda") * torch.exp(torch.randn((B * R, 1), generator=g, device="cuda") * 4)
    src = src.to(torch.bfloat16)
    # a head of zeros, one of the smallest and one of the largest values, exact borders of codes
    src[0, :hd] = 0
    src[1, :hd] = 0
    src[1, 0] = 2.0 ** -133
    src[2, :hd] = 3e38
    src[3, :hd] = 0.75 * 1.140625
    src[3, 1] = 1.140625
    rows = src[:, : 2 * Hkv * hd]
    args = (i32(ctx), R, B, Hkv, hd)
    if paged:
        xv.xv_kv_append_q8_paged(src, *args, xv.kv_pages(table, page, n_pages), c.q8, n_rows=i32(counts))
    else:
        xv.xv_kv_append_q8(src, *args, page, c.q8, n_rows=i32(counts))
    assert xv.xv_device_check() == 0
    x = rows.reshape(B, R, 2, Hkv, hd).double()
    den = x.abs().amax(-1, keepdim=True).clamp(448 * 2.0 ** -40, 448 * 2.0 ** 60)
    # the quotient is exact or rounded once to fp32 before the code's rounding; fp32 of it is that value
    codes = (x * 448 / den).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
    scale = (den / 448)[..., 0]
    want = [x.clone() for x in before]
    for b in range(B):
        for r in range(counts[b]):
            p = ctx[b] - 1 + r
            pg, at = int(table[b, p // page]), p % page
            want[0][pg, :, at], want[1][pg, :, at] = codes[b, r, 0], codes[b, r, 1]
            want[2][pg, :, at], want[3][pg, :, at] = scale[b, r, 0].float(), scale[b, r, 1].float()
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        # -0 and +0 are one value
        if got.dtype == torch.uint8:
            got, w = (torch.where(t == 128, torch.zeros_like(t), t) for t in (got, w))
        assert torch.equal(got, w)


def test_every_quotient_of_two_significands(xv):
    """Codes of all values of 8 bits of significand down to 2^-18 of the largest, for every largest: borders of
    two codes are hit exactly, and missed by 2^-13 at least."""
    hd, Hkv = 256, 1
    m = 1 + torch.arange(128, device="cuda", dtype=torch.float64) / 128
    e = torch.tensor([2.0 ** -i for i in range(19)], dtype=torch.float64, device="cuda")
    values = (m[None] * e[:, None]).reshape(-1)                       # all in [2^-18, 2)
    rows = []
    for big in m.tolist():
        v = values[values <= big]
        v = torch.nn.functional.pad(v, (0, -v.numel() % (hd - 1))).reshape(-1, hd - 1)
        rows.append(torch.cat([torch.full((v.shape[0], 1), big, device="cuda", dtype=torch.float64), v], 1))
    x = torch.cat(rows)
    x[:, 2::2] *= -1
    N = x.shape[0]
    c = Cache(xv, 1, Hkv, N, hd)
    src = torch.cat([x, x.flip(1)], 1).to(torch.bfloat16)
    assert torch.equal(src[:, :hd].double(), x)
    xv.xv_kv_append_q8(src, i32([1]), N, 1, Hkv, hd, N, c.q8)
    codes = (x * 448 / x.abs().amax(-1, keepdim=True)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    for got, want in ((c.k[0, 0], codes), (c.v[0, 0], codes.flip(1))):
        assert torch.equal(torch.where(got == 128, 0, got), torch.where(want == 128, 0, want))


def test_append_of_values_that_are_not_finite(xv):
    B, R, Hkv, hd, page = 1, 4, 2, 64, 64
    c = Cache(xv, 1, Hkv, page, hd)
    src = normal((R, 2 * Hkv * hd), 5)
    src[1, 3], src[2, Hkv * hd + 70] = NAN, -math.inf
    xv.xv_kv_append_q8(src, i32([1]), R, B, Hkv, hd, page, c.q8)
    ks, vs = c.ks[0, :, :R].isnan(), c.vs[0, :, :R].isnan()
    assert ks.nonzero().tolist() == [[0, 1]] and vs.nonzero().tolist() == [[1, 2]]
    assert not c.k[0, 0, 1].any() and not c.v[0, 1, 2].any()


def test_append_outside_the_cache_is_recorded_and_skipped(xv):
    B, R, Hkv, hd, page, n_pages = 2, 3, 2, 64, 64, 3
    c = Cache(xv, n_pages, Hkv, page, hd)
    before = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    src = normal((B * R, 2 * Hkv * hd), 5)
    for table, ctx, counts, bit in (([[7], [-1]], [1, 2], None, 16), ([[0], [1]], [66, -5], None, 4), ([[0], [1]], [66, 66], [9, -1], 12)):
        xv.xv_kv_append_q8_paged(src, i32(ctx), R, B, Hkv, hd, xv.kv_pages(i32(table), page, n_pages), c.q8,
                                 n_rows=None if counts is None else i32(counts))
        with pytest.raises(xv.XVError):
            xv.xv_device_check()
        assert xv.xv_device_check() == 0
        assert all(torch.equal(a, b) for a, b in zip(before, (c.k, c.v, c.ks, c.vs))), bit


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("ctx", [[1], [63, 64], [65, 1, 200], [255, 256, 257], [700, 4095, 4100], [5200]])
def test_lengths(xv, Hq, Hkv, hd, ctx):
    B, R, page = len(ctx), 3, 128
    per = -(-(max(ctx) + R) // page)
    n_pages = B * per + 1
    c, table = Cache(xv, n_pages, Hkv, page, hd), shuffled(B, per, n_pages, 2)
    q = normal((B * R, Hq * hd), 7)
    out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, max(ctx) + R - 1)
    assert xv.xv_device_check() == 0
    close(out, *reference(c, table, q, ctx, [R] * B, R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))


WINDOWS = [(1, 0), (5, 3), (64, 1), (100, 4), (256, 300), (1000, 64), (1000, 70), (3000, 5)]


@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows_and_sinks(xv, Hq, Hkv, hd, window, sinks):
    """Windows that begin inside tiles and splits, sinks that meet them, sequences shorter than both."""
    ctx, counts, R, page = [5300, 3, window, window + sinks + 1, 1290], [7, 7, 3, 1, 0], 7, 64
    B, per = len(ctx), 84
    n_pages = B * per
    c, table = Cache(xv, n_pages, Hkv, page, hd), shuffled(B, per, n_pages, 3)
    q = normal((B * R, 2 * Hq * hd), 8)
    gate = q[:, Hq * hd:]
    out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, 5340, window, sinks, gate, counts, fill=7.0)
    assert xv.xv_device_check() == 0
    ref, mag = reference(c, table, q, ctx, counts, R, Hq, Hkv, hd, page, window, sinks, hd ** -0.5, gate)
    live = (torch.arange(R)[None] < torch.tensor(counts)[:, None]).reshape(-1).cuda()
    close(out[live], ref[live], mag[live])
    assert (out[~live] == 7.0).all()          # rows behind a sequence's count: left as they were


@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("sinks", [10 ** 6, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
def test_sinks_past_every_length_are_the_whole_context(xv, Hq, Hkv, hd, sinks):
    """Any number of sinks may be asked for: past the context they leave nothing out, so a window changes no bit.
    The workspace holds NaN, so a split that is not computed shows."""
    ctx, R, page = [5300, 700, 40, 1], 3, 64
    B, per = len(ctx), 84
    n_pages = B * per
    c, table = Cache(xv, n_pages, Hkv, page, hd), shuffled(B, per, n_pages, 4)
    q = normal((B * R, Hq * hd), 23)
    pages = xv.kv_pages(table, page, n_pages)
    max_ctx = per * page
    def go(window, sinks):
        out = torch.zeros((B * R, Hq * hd), dtype=torch.bfloat16, device="cuda")
        ws = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, max_ctx, window, sinks))
        ws.fill_(0xff)
        xv.xv_attn_decode_rows_q8_paged(q, c.q8, pages, i32(ctx), R, B, Hq, Hkv, hd, max_ctx, hd ** -0.5, out, ws, window=window,
                                        sinks=sinks)
        return out
    want = go(0, 0)
    close(want, *reference(c, table, q, ctx, [R] * B, R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))
    for window in (1, 100, 2000, max_ctx - 1):
        assert torch.equal(go(window, sinks).view(torch.int16), want.view(torch.int16)), window
    assert xv.xv_device_check() == 0


def test_traced_bytes_of_a_window(xv):
    """What the trace says of a windowed call: the window's and the sinks' positions, at most the context's."""
    Hq, Hkv, hd, R, page = 8, 2, 64, 2, 2048
    c = Cache(xv, 1, Hkv, page, hd)
    q = normal((R, Hq * hd), 24)
    traced = {}
    for window, sinks in ((0, 0), (100, 0), (100, 28), (100, 5000), (100, 2 ** 31 - 1), (2000, 2 ** 31 - 1)):
        xv.xv_trace_enable(16)
        try:
            run(xv, c, None, q, [1500], R, Hq, Hkv, hd, page, 1, page, window, sinks, paged=False)
            torch.cuda.synchronize()
            traced[window, sinks] = next(b for kind, _, b in xv.xv_trace_read() if kind == "attn_q8")
        finally:
            xv.xv_trace_disable()
    per = Hkv * (2 * hd + 8)      # bytes a position
    slots = lambda w, s: xv.xv_attn_q8_workspace_size(1, R, Hq, hd, page, w, s) // (R * Hq * (hd + 2) * 4)   # noqa: E731
    fixed = lambda w, s: 2 * R * Hq * hd + 4 * R * Hq * slots(w, s) * (hd + 2)   # noqa: E731
    for (window, sinks), got in traced.items():
        seen = min(window + sinks, page) if window else page
        assert got == per * seen + fixed(window, sinks), (window, sinks)


@pytest.mark.parametrize("Hq,Hkv,hd", [(6, 2, 64), (8, 8, 128), (24, 4, 256), (5, 1, 64), (128, 1, 128)])
@pytest.mark.parametrize("R", [1, 17, 64])
def test_rows_and_heads(xv, Hq, Hkv, hd, R):
    """From one row of one head per kv head to 64 rows of 128."""
    ctx, page = [700, 333], 320
    c = Cache(xv, 2, Hkv, 1280, hd)
    q = normal((2 * R, Hq * hd), 9)
    table = torch.arange(2, dtype=torch.int32, device="cuda")[:, None]
    out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, 1280, 2, 1280, paged=False)
    assert xv.xv_device_check() == 0
    close(out, *reference(c, table, q, ctx, [R, R], R, Hq, Hkv, hd, 1280, 0, 0, hd ** -0.5))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 7, 9])
def test_row_tiles_of_every_size(xv, hd, R):
    """8 to 72 rows of a kv head in a call, with and without a window, and each row's bits when it is alone."""
    Hq, Hkv, page = 8, 1, 192
    ctx, per = [3000, 129, 40], 17
    c = Cache(xv, 3 * per, Hkv, page, hd)
    table = shuffled(3, per, 3 * per, 10)
    q = normal((3 * R, Hq * hd), R)
    for window, sinks in ((0, 0), (200, 5)):
        out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, 3 * per, per * page, window, sinks)
        close(out, *reference(c, table, q, ctx, [R] * 3, R, Hq, Hkv, hd, page, window, sinks, hd ** -0.5))
        for b in range(3):
            one = run(xv, c, table[b:b + 1].contiguous(), q[b * R + R - 1:b * R + R].contiguous(), [ctx[b] + R - 1], 1, Hq, Hkv, hd, page,
                      3 * per, ctx[b] + R - 1, window, sinks)
            assert torch.equal(one.view(torch.int16), out[b * R + R - 1:b * R + R].view(torch.int16)), b
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("Lmax", [1, 2, 63, 65, 97, 1001])
@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
def test_contiguous_caches_of_any_length(xv, Lmax, Hq, Hkv, hd):
    c = Cache(xv, 2, Hkv, Lmax, hd)
    R = min(3, Lmax)
    q = normal((2 * R, Hq * hd), 4)
    ctx = [Lmax - R + 1, 1]
    table = torch.arange(2, dtype=torch.int32, device="cuda")[:, None]
    out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, Lmax, 2, Lmax, paged=False)
    assert xv.xv_device_check() == 0
    close(out, *reference(c, table, q, ctx, [R, R], R, Hq, Hkv, hd, Lmax, 0, 0, hd ** -0.5))


@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 2), (70, 500)])
def test_a_verify_row_has_the_bits_of_its_decode_row(xv, Hq, Hkv, hd, window, sinks):
    """Rows across a tile's and a split's border and across 4096; then other batches and pages."""
    page, per, R = 64, 72, 64
    n_pages = 4 * per
    c = Cache(xv, n_pages, Hkv, page, hd)
    table = shuffled(4, per, n_pages, 5)
    for L in (1, 230, 4060):
        q = normal((R, Hq * hd), L)
        wide = run(xv, c, table[:1], q, [L], R, Hq, Hkv, hd, page, n_pages, per * page, window, sinks)
        for r in (0, 1, 25, 26, 27, 36, 37, 63):
            one = run(xv, c, table[:1], q[r:r + 1], [L + r], 1, Hq, Hkv, hd, page, n_pages, L + r, window, sinks)
            assert torch.equal(one.view(torch.int16), wide[r:r + 1].view(torch.int16)), (L, r)
        # as the third of four sequences, whose others have other lengths
        qs = torch.cat([normal((2 * R, Hq * hd), 1), q, normal((R, Hq * hd), 2)])
        many = run(xv, c, table[[1, 2, 0, 3]].contiguous(), qs, [4500, 7, L, 2000], R, Hq, Hkv, hd, page, n_pages, 4563, window,
                   sinks)
        assert torch.equal(many[2 * R:3 * R].view(torch.int16), wide.view(torch.int16)), L
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_v_scales_of_any_size_and_a_strong_sink(xv, hd):
    """V scales that differ by e^10 and more, a first token that takes half of the weight, the rest
    spread thin over a long context; the smallest and largest scales an append gives."""
    Hq, Hkv, R, page, ctx = 4, 2, 2, 8192, 8000
    c = Cache(xv, 1, Hkv, page, hd, outlier=True)
    q = normal((R, Hq * hd), 11, 0.05)
    q32 = q.float().reshape(R, Hkv, 2, hd).mean((0, 2))
    k0 = q32 / q32.abs().amax(-1, keepdim=True) * 400
    c.k[0, :, 0] = k0.to(torch.float8_e4m3fn).view(torch.uint8)
    s = (q32 * dequant(c.k[0, :, 0], torch.ones(Hkv, device="cuda")).float()).sum(-1) * hd ** -0.5
    c.ks[0, :, 0] = math.log(8000) / s
    c.vs[0, :, 0] = 2.0 ** -40
    c.vs[0, 0, 77] = 2.0 ** -40
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    out = run(xv, c, table, q, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False)
    close(out, *reference(c, table, q, [ctx], [R], R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))
    c.vs[0, :, 100] = 2.0 ** 60
    out = run(xv, c, table, q, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False)
    close(out, *reference(c, table, q, [ctx], [R], R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_q_of_any_size(xv, size):
    """q far from 1, the scale making up for it: the bits of the plain q where the factor, a power of two,
    loses none of q's (2^-120 does: q's values below 2^-6 get past bf16's smallest normal number, 2^-126)."""
    Hq, Hkv, hd, R, page, ctx = 4, 2, 128, 3, 1024, 600
    c = Cache(xv, 1, Hkv, page, hd)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q = normal((R, Hq * hd), 12)
    q[1, :hd] = 0
    want = run(xv, c, table, q, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False, scale=2.0 ** -3)
    big = (q.float() * size).to(torch.bfloat16)
    got = run(xv, c, table, big, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False, scale=2.0 ** -3 / size)
    close(got, *reference(c, table, big, [ctx], [R], R, Hq, Hkv, hd, page, 0, 0, 2.0 ** -3 / size))
    exact = torch.equal(big.double() / size, q.double())
    assert exact or size < 2.0 ** -100
    if exact:
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
def test_what_is_not_finite_stays_where_it_is_seen(xv, Hq, Hkv, hd):
    """NaN scales of a later draft, of tokens before the window, NaN bytes behind the length and q that is not
    finite: rows that do not see them keep their bits, those that do are NaN."""
    R, page, ctx = 4, 1024, 500
    c = Cache(xv, 1, Hkv, page, hd)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q = normal((R, Hq * hd), 13)
    go = lambda **kw: run(xv, c, table, q, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False, **kw)   # noqa: E731
    clean, windowed = go(), go(window=200, sinks=2)
    c.k[0, :, ctx + R - 1:] = 0x7f            # behind every row
    c.v[0, :, ctx + R - 1:] = 0xff
    c.ks[0, :, ctx + R - 1:] = NAN
    c.vs[0, :, ctx + R - 1:] = NAN
    assert torch.equal(go().view(torch.int16), clean.view(torch.int16))
    c.ks[0, 0, ctx + 1] = NAN                 # row 2's own token
    G = Hq // Hkv
    hit = torch.zeros((R, Hq), dtype=torch.bool, device="cuda")
    hit[2:, :G] = True
    def check(out, want, hit):
        o, w = out.reshape(R, Hq, hd), want.reshape(R, Hq, hd)
        assert o[hit].isnan().all()
        assert torch.equal(o[~hit].view(torch.int16), w[~hit].view(torch.int16))
    check(go(), clean, hit)
    c.vs[0, -1, ctx - 200] = NAN              # the first position of row 0's window (500 - 200), before those of the rows behind it
    seen = torch.zeros_like(hit)
    seen[2:, :G] = True
    seen[0, -G:] = True
    check(go(window=200, sinks=2), windowed, seen)
    q[0, hd + 5] = math.inf
    q[1, 3] = NAN
    seen[0, 1] = seen[1, 0] = True
    check(go(window=200, sinks=2), windowed, seen)
    assert xv.xv_device_check() == 0


def test_codes_of_every_value(xv):
    """All 254 finite codes in K and in V."""
    Hq, Hkv, hd, R, page, ctx = 4, 2, 128, 2, 256, 250
    c = Cache(xv, 1, Hkv, page, hd)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (c.k, c.v):
        x = torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.int32)
        t.copy_(torch.where((x & 127) == 127, x - 1, x).to(torch.uint8))
    c.ks.div_(8)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    q = normal((R, Hq * hd), 14)
    out = run(xv, c, table, q, [ctx], R, Hq, Hkv, hd, page, 1, ctx + R - 1, paged=False)
    close(out, *reference(c, table, q, [ctx], [R], R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))


def test_strided_rows_and_gate(xv):
    Hq, Hkv, hd, R, page = 4, 2, 128, 3, 512
    B, ctx = 2, [300, 411]
    c = Cache(xv, B, Hkv, page, hd)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    proj = normal((B * R, 3 * Hq * hd + 8), 15)
    wide = torch.zeros((B * R, 2 * Hq * hd), dtype=torch.bfloat16, device="cuda")
    ws = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, page))
    q, gate, out = proj[:, 8:], proj[:, Hq * hd + 8:], wide[:, Hq * hd:]
    xv.xv_attn_decode_rows_q8(q, c.q8, i32(ctx), R, B, Hq, Hkv, hd, page, page, hd ** -0.5, out, ws, gate=gate)
    close(out, *reference(c, table, q, ctx, [R] * B, R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5, gate))
    assert not wide[:, : Hq * hd].any()


def test_a_pool_past_two_to_the_32_bytes(xv):
    """Pages at the end of a pool of more than 2^32 codes; the rest of the pool is never written."""
    Hkv, hd, page, R, Hq = 8, 256, 64, 2, 8
    n_pages = (1 << 32) // (Hkv * hd * page) + 40
    k = torch.empty((n_pages, Hkv, page, hd), dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty((n_pages, Hkv, page), device="cuda")
    vs = torch.empty_like(ks)
    cache = xv.kv_q8(k, v, ks, vs)
    ctx, B = [130], 1
    table = i32([[n_pages - 1, n_pages - 7, n_pages - 3]])
    pages = xv.kv_pages(table, page, n_pages)
    src = normal((131, 2 * Hkv * hd), 16)
    xv.xv_kv_append_q8_paged(src, i32([1]), 131, B, Hkv, hd, pages, cache)
    q = normal((R, Hq * hd), 17)
    out = torch.zeros((R, Hq * hd), dtype=torch.bfloat16, device="cuda")
    ws = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, 192))
    xv.xv_attn_decode_rows_q8_paged(q, cache, pages, i32(ctx), R, B, Hq, Hkv, hd, 192, hd ** -0.5, out, ws)
    assert xv.xv_device_check() == 0
    small = Cache(xv, 3, Hkv, page, hd)
    for a, b in zip((small.k, small.v, small.ks, small.vs), (k, v, ks, vs)):
        a.copy_(b[table[0].long()])
    t = i32([[0, 1, 2]])
    close(out, *reference(small, t, q, ctx, [R], R, Hq, Hkv, hd, page, 0, 0, hd ** -0.5))


def test_bad_lengths_counts_and_pages_are_recorded(xv):
    Hq, Hkv, hd, R, page, n_pages = 4, 2, 64, 3, 64, 9
    c = Cache(xv, n_pages, Hkv, page, hd)
    q = normal((3 * R, Hq * hd), 18)
    table = i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    good = run(xv, c, table, q, [100, 150, 60], R, Hq, Hkv, hd, page, n_pages, 152)
    for ctx in ([100, 151, 60], [100, 0, 60], [100, -2 ** 31, 60], [100, 2 ** 31 - 1, 60]):
        out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, 152, fill=3.0)
        with pytest.raises(xv.XVError, match="error"):
            xv.xv_device_check()
        assert torch.equal(out[:R], good[:R]) and torch.equal(out[2 * R:], good[2 * R:]) and (out[R: 2 * R] == 3).all()
    run(xv, c, table, q, [100, 150, 60], R, Hq, Hkv, hd, page, n_pages, 152, counts=[3, 4, -1])
    with pytest.raises(xv.XVError):
        xv.xv_device_check()
    bad = table.clone()
    bad[1, 1] = n_pages
    out = run(xv, c, bad, q, [100, 150, 60], R, Hq, Hkv, hd, page, n_pages, 152)
    with pytest.raises(xv.XVError):
        xv.xv_device_check()
    assert torch.equal(out[:R], good[:R]) and torch.equal(out[2 * R:], good[2 * R:])
    # pages before the window and past the sinks are not read
    bad = table.clone()
    bad[1, 1] = -1
    run(xv, c, bad, q, [100, 150, 60], R, Hq, Hkv, hd, page, n_pages, 152, window=20, sinks=3)
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("hd,Hq,Hkv", [(64, 8, 2), (128, 32, 8), (256, 24, 4)])
def test_many_items_per_cta(xv, hd, Hq, Hkv):
    """Batches past two waves of items: persistent CTAs, ragged lengths, counts of 0 between others."""
    B, R, page, per = 40, 2, 128, 40
    ctx = [5000 - 120 * b for b in range(B)]
    counts = [(b * 7) % 3 for b in range(B)]
    n_pages = 300
    c = Cache(xv, n_pages, Hkv, page, hd)
    table = torch.randint(0, n_pages, (B, per), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    q = normal((B * R, Hq * hd), 19)
    for window, sinks in ((0, 0), (700, 130)):
        out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, 5001, window, sinks, counts=counts)
        assert xv.xv_device_check() == 0
        close(out, *reference(c, table, q, ctx, counts, R, Hq, Hkv, hd, page, window, sinks, hd ** -0.5))


@pytest.mark.parametrize("Hq,Hkv,hd,R", [(2, 1, 64, 5), (8, 2, 128, 1), (24, 4, 256, 8)])
def test_contexts_past_the_last_change_of_splits(xv, Hq, Hkv, hd, R):
    """Contexts around and far past 32768, where splits are the longest, short ones between them, and a row's
    bits alone."""
    ctx, page = [90000, 32768 - R, 200, 32769, 41000], 128
    B, per = len(ctx), 704
    n_pages = 1500
    c = Cache(xv, n_pages, Hkv, page, hd)
    table = torch.randint(0, n_pages, (B, per), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    q = normal((B * R, Hq * hd), 22)
    for window, sinks in ((0, 0), (40000, 300)):
        out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, per * page, window, sinks)
        close(out, *reference(c, table, q, ctx, [R] * B, R, Hq, Hkv, hd, page, window, sinks, hd ** -0.5))
        for b in (0, 3):
            r = R - 1
            one = run(xv, c, table[b:b + 1].contiguous(), q[b * R + r:b * R + r + 1].contiguous(), [ctx[b] + r], 1, Hq, Hkv, hd, page, n_pages,
                      ctx[b] + r, window, sinks)
            assert torch.equal(one.view(torch.int16), out[b * R + r:b * R + r + 1].view(torch.int16)), b
    assert xv.xv_device_check() == 0


def test_many_sequences_with_bad_ones_among_them(xv):
    """More sequences than one pass of the shares takes, in persistent CTAs: bad lengths, counts of 0 and bad
    counts between good ones, which keep the bits they have alone."""
    Hq, Hkv, hd, R, page, per, B = 16, 8, 128, 3, 64, 40, 70
    n_pages = 500
    c = Cache(xv, n_pages, Hkv, page, hd)
    table = torch.randint(0, n_pages, (B, per), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    ctx = [2500 - 35 * b for b in range(B)]
    counts = [3 - b % 4 for b in range(B)]
    q = normal((B * R, Hq * hd), 21)
    bad = {5: -7, 33: 0, 34: 2 ** 31 - 1, 69: 3000}
    for b, v in bad.items():
        ctx[b] = v
    out = run(xv, c, table, q, ctx, R, Hq, Hkv, hd, page, n_pages, 2560, counts=counts, fill=5.0)
    with pytest.raises(xv.XVError):
        xv.xv_device_check()
    for b in (0, 1, 4, 6, 32, 35, 66, 68):
        n = counts[b]
        if n:
            one = run(xv, c, table[b:b + 1].contiguous(), q[b * R:b * R + n].contiguous(), [ctx[b]], n, Hq, Hkv, hd, page, n_pages, 2560)
            assert torch.equal(one.view(torch.int16), out[b * R:b * R + n].view(torch.int16)), b
        assert (out[b * R + n:(b + 1) * R] == 5).all()
    for b in bad:
        assert counts[b] == 0 or (out[b * R:(b + 1) * R] == 5).all()
    assert xv.xv_device_check() == 0


def test_a_captured_step_replayed_with_new_lengths_on_another_stream(xv):
    """Append and attention in one graph, replayed as the context grows; two graphs of one workspace, one
    after the other."""
    Hq, Hkv, hd, R, page, B, per = 8, 2, 128, 2, 64, 2, 8
    c = Cache(xv, B * per, Hkv, page, hd)
    table = shuffled(B, per, B * per, 6)
    pages = xv.kv_pages(table, page, B * per)
    ctx = i32([100, 61])
    proj = normal((B * R, (Hq + 2 * Hkv) * hd), 20)
    out = torch.zeros((B * R, Hq * hd), dtype=torch.bfloat16, device="cuda")
    ws = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, per * page, 100, 4))
    def step(window):
        xv.xv_kv_append_q8_paged(proj[:, Hq * hd:], ctx, R, B, Hkv, hd, pages, c.q8)
        xv.xv_attn_decode_rows_q8_paged(proj, c.q8, pages, ctx, R, B, Hq, Hkv, hd, per * page, hd ** -0.5, out, ws, window=window,
                                        sinks=4)
    step(0)
    step(100)
    s = torch.cuda.Stream()
    graphs = []
    for window in (0, 100):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step(window)
        graphs.append((gr, window))
    for i in range(6):
        ctx.add_(i * 3)
        proj.copy_(normal(proj.shape, 30 + i))
        gr, window = graphs[i % 2]
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            gr.replay()
        torch.cuda.default_stream().wait_stream(s)
        close(out, *reference(c, table, proj, ctx.tolist(), [R] * B, R, Hq, Hkv, hd, page, window, 4 if window else 0, hd ** -0.5))
    assert xv.xv_device_check() == 0


def test_two_streams_at_once(xv):
    """Calls with workspaces of their own at the same time."""
    Hq, Hkv, hd, R, page = 24, 4, 256, 8, 4096
    c = Cache(xv, 1, Hkv, page, hd)
    qs = [normal((R, Hq * hd), 40 + i) for i in range(4)]
    ctx, table = i32([4000]), None
    alone = [run(xv, c, table, q, [4000], R, Hq, Hkv, hd, page, 1, page, paged=False) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.zeros_like(a) for a in alone]
    wss = [xv.workspace(xv.xv_attn_q8_workspace_size(1, R, Hq, hd, page)) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, s, o, ws in zip(qs, streams, outs, wss):
            xv.xv_attn_decode_rows_q8(q, c.q8, ctx, R, 1, Hq, Hkv, hd, page, page, hd ** -0.5, o, ws, stream=s)
    torch.cuda.synchronize()
    assert xv.xv_device_check() == 0
    for a, o in zip(alone, outs):
        assert torch.equal(a.view(torch.int16), o.view(torch.int16))


def test_repeated_runs_have_the_same_bits(xv):
    Hq, Hkv, hd, R, page, ctx = 32, 8, 128, 4, 8192, [8000, 5001]
    c = Cache(xv, 2, Hkv, page, hd)
    q = normal((2 * R, Hq * hd), 50)
    one = run(xv, c, None, q, ctx, R, Hq, Hkv, hd, page, 2, page, paged=False)
    for _ in range(20):
        assert torch.equal(run(xv, c, None, q, ctx, R, Hq, Hkv, hd, page, 2, page, paged=False).view(torch.int16), one.view(torch.int16))


def test_appended_verify_equals_sequential_decode(xv):
    """The step as it is used: a verify's rows appended and attended together, against one append and one
    attention per token; then the accepted tokens are kept and the next verify overwrites the rest."""
    Hq, Hkv, hd, page, per = 24, 4, 256, 64, 6
    a, b = Cache(xv, per, Hkv, page, hd), Cache(xv, per, Hkv, page, hd)
    table = shuffled(1, per, per, 7)
    pages = xv.kv_pages(table, page, per)
    L = 120
    for step, keep in enumerate((3, 8, 1)):
        R = 8
        proj = normal((R, (Hq + 2 * Hkv) * hd), 60 + step)
        out = torch.zeros((R, Hq * hd), dtype=torch.bfloat16, device="cuda")
        ws = xv.workspace(xv.xv_attn_q8_workspace_size(1, R, Hq, hd, per * page, 50, 2))
        xv.xv_kv_append_q8_paged(proj[:, Hq * hd:], i32([L]), R, 1, Hkv, hd, pages, a.q8)
        xv.xv_attn_decode_rows_q8_paged(proj, a.q8, pages, i32([L]), R, 1, Hq, Hkv, hd, per * page, hd ** -0.5, out, ws, window=50, sinks=2)
        for r in range(keep):
            one = torch.zeros((1, Hq * hd), dtype=torch.bfloat16, device="cuda")
            xv.xv_kv_append_q8_paged(proj[r:r + 1, Hq * hd:], i32([L + r]), 1, 1, Hkv, hd, pages, b.q8)
            xv.xv_attn_decode_rows_q8_paged(proj[r:r + 1], b.q8, pages, i32([L + r]), 1, 1, Hq, Hkv, hd, per * page, hd ** -0.5, one, ws,
                                            window=50, sinks=2)
            assert torch.equal(one.view(torch.int16), out[r:r + 1].view(torch.int16)), (step, r)
        L += keep
    assert xv.xv_device_check() == 0


def test_a_stream_of_kernels_that_take_tensor_memory(xv):
    """bf16 attention, 8-bit attention of row tiles with 512 columns, GEMM and back, at sizes of which two fit an SM's
    memory together (hd 64), launched while the first still waits: each has the bits of a call by itself."""
    B, R, Hq, Hkv, hd, L = 8, 8, 12, 2, 64, 1500
    c = Cache(xv, B, Hkv, L, hd)
    q = normal((B * R, Hq * hd), 70)
    kc, vc = normal((B, Hkv, L, hd), 71), normal((B, Hkv, L, hd), 72)
    X, W = normal((8, 1024), 73), normal((4096, 1024), 74, 0.05)
    ctx = i32([1400 - 100 * b for b in range(B)])
    scale = hd ** -0.5
    new = lambda: [torch.zeros_like(q), torch.zeros_like(q),   # noqa: E731
                   torch.zeros((8, 4096), dtype=torch.bfloat16, device="cuda")]
    ws = [xv.workspace(xv.xv_attn_workspace_size(B, R, Hq, hd, L)), xv.workspace(xv.xv_attn_q8_workspace_size(B, R, Hq, hd, L)),
          xv.workspace(xv.xv_gemm_workspace_size(8, 4096, 1024))]
    def bf16(o):
        xv.xv_attn_decode_rows(q, Hq * hd, kc, vc, ctx, R, B, Hq, Hkv, hd, L, L, scale, o[0], Hq * hd, ws[0])
    def q8(o):
        xv.xv_attn_decode_rows_q8(q, c.q8, ctx, R, B, Hq, Hkv, hd, L, L, scale, o[1], ws[1])
    def gemm(o):
        xv.xv_gemm_small_m(X, W, o[2], ws[2])
    want = new()
    for f in (bf16, q8, gemm):
        f(want)
        torch.cuda.synchronize()
    for order in ((bf16, q8), (q8, gemm), (bf16, q8, gemm), (gemm, q8, bf16), (q8, bf16), (q8, q8, gemm, gemm)):
        outs = []
        torch.cuda._sleep(2_000_000)      # about a millisecond, while the launches queue up
        for _ in range(6):
            outs.append(new())
            for f in order:
                f(outs[-1])
        torch.cuda.synchronize()
        for o in outs:
            for f, a, b in zip((bf16, q8, gemm), o, want):
                if f in order:
                    assert torch.equal(a.view(torch.int16), b.view(torch.int16)), [g.__name__ for g in order]
    assert xv.xv_device_check() == 0
