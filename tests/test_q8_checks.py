"""Refusals of the 8-bit cache's entry points and of the scores: by the Python functions before the
library is called (host tensors stand in for the device's), and by the C entry points before anything
is launched (addresses that are never followed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


B, R, Hq, Hkv, hd, page, n_pages, Lmax, M, V = 3, 5, 4, 2, 64, 64, 7, 192, 6, 50


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def rows(m, width):
    return torch.zeros((m, width), dtype=torch.bfloat16)


def cache(xv, *lead):
    codes = lambda: torch.zeros((*lead, hd), dtype=torch.uint8)   # noqa: E731
    return xv.kv_q8(codes(), codes(), f32(*lead), f32(*lead))


def calls(xv):
    """Each entry point with arguments of the right types and the least sizes."""
    pages = xv.kv_pages(i32(B, 3), page, n_pages)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    append = dict(kv_src=rows(B * R, 2 * Hkv * hd), ctx_len=i32(B), R=R, B=B, Hkv=Hkv, hd=hd, n_rows=i32(B))
    attn = dict(q=rows(B * R, Hq * hd), ctx_len=i32(B), R=R, B=B, Hq=Hq, Hkv=Hkv, hd=hd, max_ctx=100, scale=0.125,
                out=rows(B * R, Hq * hd), ws=ws, gate=rows(B * R, Hq * hd), n_rows=i32(B))
    flat = dict(Lmax=Lmax, cache=cache(xv, B, Hkv, Lmax))
    paged = dict(pages=pages, cache=cache(xv, n_pages, Hkv, page))
    return {
        "xv_kv_append_q8": dict(append, **flat),
        "xv_kv_append_q8_paged": dict(append, **paged),
        "xv_attn_decode_rows_q8": dict(attn, **flat),
        "xv_attn_decode_rows_q8_paged": dict(attn, **paged),
        "xv_logprobs": dict(logits=f32(M, V), tokens=i32(M), logprob=f32(M), ws=ws, entropy=f32(M), top_ids=i32(M, 4),
                            top_logprobs=f32(M, 4), n_rows=i32(1)),
    }


NAMES = ["xv_kv_append_q8", "xv_kv_append_q8_paged", "xv_attn_decode_rows_q8", "xv_attn_decode_rows_q8_paged", "xv_logprobs"]


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(xv, name):
    with pytest.raises(ValueError, match="current device"):
        getattr(xv, name)(**calls(xv)[name])


@pytest.mark.parametrize("name", NAMES)
def test_other_types_are_refused(xv, name):
    args = calls(xv)[name]
    for k, t in args.items():
        if not torch.is_tensor(t) or k == "ws":
            continue
        for dtype in (torch.int32, torch.int64, torch.float32, torch.int8):
            if dtype == t.dtype:
                continue
            with pytest.raises(ValueError, match=f"^{k}:"):
                getattr(xv, name)(**dict(args, **{k: torch.zeros(t.shape, dtype=dtype)}))


@pytest.mark.parametrize("name", NAMES)
def test_16_bit_floats_of_the_other_kind_are_refused(xv, name):
    """float16 would be read as bf16; bf16 may be given as its bits."""
    args = calls(xv)[name]
    for k, t in args.items():
        if not torch.is_tensor(t) or t.itemsize != 2:
            continue
        with pytest.raises(ValueError, match=f"^{k}:.*bfloat16"):
            getattr(xv, name)(**dict(args, **{k: torch.zeros(t.shape, dtype=torch.float16)}))
        for bits in (torch.bfloat16, torch.int16, torch.uint16):
            with pytest.raises(ValueError, match="current device"):
                getattr(xv, name)(**dict(args, **{k: torch.zeros(t.shape, dtype=bits)}))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_with_too_few_entries_are_refused(xv, name):
    args = calls(xv)[name]
    for k, t in args.items():
        if not torch.is_tensor(t) or k in ("ws", "logits"):      # logits fix a call's sizes
            continue
        with pytest.raises(ValueError, match=f"^{k}:"):
            getattr(xv, name)(**dict(args, **{k: t[:-1]}))
        if t.dtype == torch.bfloat16:      # rows too narrow
            with pytest.raises(ValueError, match=f"^{k}:"):
                getattr(xv, name)(**dict(args, **{k: t[:, :-1]}))


@pytest.mark.parametrize("name", NAMES)
def test_strided_tensors_are_refused(xv, name):
    """Every other entry of a tensor twice as long (rows may be strided, their values not)."""
    args = calls(xv)[name]
    for k, t in args.items():
        if not torch.is_tensor(t) or t.numel() < 2:
            continue
        wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
        with pytest.raises(ValueError, match=f"^{k}:"):
            getattr(xv, name)(**dict(args, **{k: wide}))


def test_sizes_beside_the_tensors(xv):
    """B, R, heads and pages are given beside the tensors: more of them than the tensors hold."""
    for name in NAMES[:4]:
        for more in (dict(B=B + 1), dict(R=R + 1), dict(Hkv=4), dict(hd=128)):
            with pytest.raises(ValueError):
                getattr(xv, name)(**dict(calls(xv)[name], **more))
    for name in (NAMES[0], NAMES[2]):
        with pytest.raises(ValueError, match="^cache:"):
            getattr(xv, name)(**dict(calls(xv)[name], Lmax=Lmax + 1))
    for name in (NAMES[1], NAMES[3]):
        with pytest.raises(ValueError, match="^cache:"):
            getattr(xv, name)(**dict(calls(xv)[name], pages=xv.kv_pages(i32(B, 3), page, n_pages + 1)))
        with pytest.raises(ValueError, match="page_table"):
            getattr(xv, name)(**dict(calls(xv)[name], pages=xv.kv_pages(i32(B - 1, 3), page, n_pages)))


def test_caches_of_other_types_and_layouts_are_refused(xv):
    codes, scales = torch.zeros((2, 2, 8, 64), dtype=torch.uint8), f32(2, 2, 8)
    xv.kv_q8(codes.view(torch.float8_e4m3fn), codes, scales, scales)
    for k, bad in (("k", codes.view(torch.int8)), ("k", codes.view(torch.float8_e5m2)), ("k", codes[..., ::2]), ("v", codes.transpose(1, 2)),
                   ("k_scale", scales.double()), ("v_scale", scales.transpose(1, 2)), ("v_scale", scales[..., ::2])):
        with pytest.raises(ValueError, match=f"^{k}:"):
            xv.kv_q8(**dict(dict(k=codes, v=codes, k_scale=scales, v_scale=scales), **{k: bad}))


def test_alternatives_without_their_scores_are_refused(xv):
    args = calls(xv)["xv_logprobs"]
    for k in ("top_ids", "top_logprobs"):
        with pytest.raises(ValueError, match="both or neither"):
            xv.xv_logprobs(**dict(args, **{k: None}))


def test_alternatives_of_another_width_than_their_scores_are_refused(xv):
    """Both are written as [M, top]: a wider one has its rows elsewhere."""
    args = calls(xv)["xv_logprobs"]
    for scores in (f32(M, 8), f32(M, 3), f32(2 * M, 2), f32(4 * M), f32(1, M, 4)):
        with pytest.raises(ValueError, match="^top_logprobs:"):
            xv.xv_logprobs(**dict(args, top_logprobs=scores))
    for ids in (i32(M, 8), i32(2 * M, 2), i32(M, 5)):
        with pytest.raises(ValueError, match="^top_"):
            xv.xv_logprobs(**dict(args, top_ids=ids))
    with pytest.raises(ValueError, match="current device"):      # more rows than the call's: as everywhere
        xv.xv_logprobs(**dict(args, top_ids=i32(M + 2, 4), top_logprobs=f32(M + 1, 4)))


P, ODD = 0x10000, 0x10008


def c_cache(xv, **kw):
    return ctypes.byref(xv.KvQ8(*[kw.get(k, P) for k in ("k", "v", "k_scale", "v_scale")]))


def c_pages(xv, **kw):
    return ctypes.byref(xv.KvPages(*[kw.get(k, v) for k, v in (("page_table", P), ("page_size", 64), ("max_pages", 8), ("n_pages", 100))]))


def test_c_append_refusals(xv):
    L = xv.lib()

    def call(paged=False, **kw):
        a = dict(src=P, stride=512, ctx=P, rows=None, R=3, B=2, Hkv=2, hd=128, Lmax=500, cache=c_cache(xv), pages=c_pages(xv))
        a.update(kw)
        if paged:
            return L.xv_kv_append_q8_paged(a["src"], a["stride"], a["ctx"], a["rows"], a["R"], a["B"], a["Hkv"], a["hd"], a["pages"], a["cache"], None)
        return L.xv_kv_append_q8(a["src"], a["stride"], a["ctx"], a["rows"], a["R"], a["B"], a["Hkv"], a["hd"], a["Lmax"], a["cache"], None)

    for paged in (False, True):
        for kw in (dict(src=None), dict(ctx=None), dict(R=0), dict(B=0), dict(Hkv=0), dict(stride=511), dict(cache=None),
                   dict(cache=c_cache(xv, k=None)), dict(cache=c_cache(xv, v_scale=None))):
            assert call(paged, **kw) == xv.XV_ERR_ARG, kw
        for kw in (dict(hd=96), dict(hd=512, stride=4096), dict(src=ODD), dict(stride=516), dict(cache=c_cache(xv, v=ODD)),
                   dict(cache=c_cache(xv, k_scale=ODD)), dict(R=1 << 20, B=1 << 10)):
            assert call(paged, **kw) == xv.XV_ERR_UNSUPPORTED, kw
    assert call(Lmax=0) == xv.XV_ERR_ARG and call(Lmax=(1 << 30) + 1) == xv.XV_ERR_UNSUPPORTED
    for kw in (dict(page_table=None), dict(page_size=0), dict(max_pages=0), dict(n_pages=0)):
        assert call(True, pages=c_pages(xv, **kw)) in (xv.XV_ERR_ARG, xv.XV_ERR_UNSUPPORTED), kw
    assert call(True, pages=c_pages(xv, page_size=100)) == xv.XV_ERR_UNSUPPORTED      # not a multiple of 64


@pytest.mark.parametrize("R,B,Hkv", [(1 << 30, 1 << 30, 16), ((1 << 31) - 1, (1 << 31) - 1, 2), (1 << 20, 1 << 22, 1 << 21),
                                     (1 << 29, 1, 2), (1, 1, (1 << 29) + 1), ((1 << 29) + 1, 1, 1)])
def test_more_rows_times_heads_than_an_append_takes(xv, R, B, Hkv):
    """Products past 2^63, which come out as any number in 64 bits, and the least ones past 2^29."""
    code = xv.lib().xv_kv_append_q8_paged(P, 2 * Hkv * 64, P, None, R, B, Hkv, 64, c_pages(xv, n_pages=1), c_cache(xv), None)
    assert code == xv.XV_ERR_UNSUPPORTED


def test_c_attention_refusals(xv):
    L = xv.lib()

    def call(paged=False, **kw):
        a = dict(q=P, qs=1024, ctx=P, rows=None, R=3, B=2, Hq=8, Hkv=2, hd=128, Lmax=500, max_ctx=400, window=0, sinks=0, gate=None, gs=0,
                 out=P, os=1024, ws=P, bytes=1 << 40, cache=c_cache(xv), pages=c_pages(xv))
        a.update(kw)
        tail = (a["max_ctx"], a["window"], a["sinks"], 0.1, a["gate"], a["gs"], a["out"], a["os"], a["ws"], a["bytes"], None)
        sizes = (a["ctx"], a["rows"], a["R"], a["B"], a["Hq"], a["Hkv"], a["hd"])
        if paged:
            return L.xv_attn_decode_rows_q8_paged(a["q"], a["qs"], a["cache"], a["pages"], *sizes, *tail)
        return L.xv_attn_decode_rows_q8(a["q"], a["qs"], a["cache"], *sizes, a["Lmax"], *tail)

    for paged in (False, True):
        for kw in (dict(q=None), dict(ctx=None), dict(out=None), dict(R=0), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(max_ctx=0),
                   dict(max_ctx=513), dict(window=-1), dict(sinks=-1), dict(qs=1023), dict(os=1023), dict(gate=P, gs=1023), dict(cache=None),
                   dict(cache=c_cache(xv, v=None))):
            assert call(paged, **kw) == xv.XV_ERR_ARG, kw
        for kw in (dict(hd=96), dict(R=xv.XV_KMAX + 1), dict(q=ODD), dict(out=ODD), dict(gate=ODD, gs=1024), dict(qs=1028), dict(os=1028),
                   dict(gate=P, gs=1028), dict(ws=ODD), dict(cache=c_cache(xv, v_scale=ODD))):
            assert call(paged, **kw) == xv.XV_ERR_UNSUPPORTED, kw
        need = xv.xv_attn_q8_workspace_size(2, 3, 8, 128, 400)
        for kw in (dict(ws=None), dict(bytes=need - 1), dict(bytes=0)):
            assert call(paged, **kw) == xv.XV_ERR_WORKSPACE, kw
    assert call(B=65536, Lmax=400) == xv.XV_ERR_UNSUPPORTED
    size = xv.xv_attn_q8_workspace_size
    for bad in ((0, 3, 8, 128, 400), (2, 0, 8, 128, 400), (2, 65, 8, 128, 400), (2, 3, 0, 128, 400), (2, 3, 8, 96, 400), (2, 3, 8, 128, 0),
                (2, 3, 8, 128, (1 << 30) + 1), (2, 3, 8, 128, 400, -1), (2, 3, 8, 128, 400, 0, -1), (65536, 3, 8, 128, 400),
                (65535, 64, 512, 128, 400)):
        assert size(*bad) == 0, bad
    # a window needs less, one that holds every row what none needs
    assert 0 < size(2, 3, 8, 128, 100000, 1000, 4) < size(2, 3, 8, 128, 100000) == size(2, 3, 8, 128, 100000, 100000, 4)


def test_c_score_refusals(xv):
    L = xv.lib()

    def call(bf16=False, **kw):
        a = dict(x=P, ld=1000, tok=P, rows=None, M=4, V=1000, lp=P, en=None, top=0, ids=None, lps=None, ws=P, bytes=1 << 40)
        a.update(kw)
        f = L.xv_logprobs_bf16 if bf16 else L.xv_logprobs
        return f(a["x"], a["ld"], a["tok"], a["rows"], a["M"], a["V"], a["lp"], a["en"], a["top"], a["ids"], a["lps"], a["ws"], a["bytes"], None)

    for bf16 in (False, True):
        for kw in (dict(x=None), dict(tok=None), dict(lp=None), dict(M=0), dict(V=0), dict(ld=999), dict(top=-1), dict(top=4), dict(top=4, ids=P),
                   dict(top=4, lps=P), dict(V=3, top=4, ids=P, lps=P)):
            assert call(bf16, **kw) == xv.XV_ERR_ARG, kw
        for kw in (dict(top=33, ids=P, lps=P), dict(V=(1 << 19) + 1, ld=1 << 20), dict(x=P + 1), dict(ws=ODD), dict(M=1 << 30, V=20000, ld=20000)):
            assert call(bf16, **kw) == xv.XV_ERR_UNSUPPORTED, kw
        for kw in (dict(ws=None), dict(bytes=xv.xv_logprobs_workspace_size(4, 1000, 0) - 1)):
            assert call(bf16, **kw) == xv.XV_ERR_WORKSPACE, kw
    assert call(x=P + 2) == xv.XV_ERR_UNSUPPORTED      # fp32 at an odd half
    for bad in ((0, 5, 0), (5, 0, 0), (5, (1 << 19) + 1, 0), (5, 5, -1), (5, 5, 6), (5, 100, 33)):
        assert xv.xv_logprobs_workspace_size(*bad) == 0, bad


def test_split_boundaries(xv):
    """Rising, on tiles' borders, at most 1024 positions, and as the row's slots are counted."""
    at = [xv.xv_attn_q8_split_begin(s) for s in range(3000)]
    assert at[0] == 0 and xv.xv_attn_q8_split_begin(-1) == -1
    steps = [b - a for a, b in zip(at, at[1:])]
    assert all(s % 128 == 0 and 0 < s <= 1024 for s in steps) and steps == sorted(steps)
    for ctx in (1, 256, 257, 2048, 2049, 32768, 32769, 131072):
        slots = sum(a < ctx for a in at)
        rows = 2 * 8
        up = lambda n: -(-n // 256) * 256   # noqa: E731
        assert xv.xv_attn_q8_workspace_size(1, 2, 8, 64, ctx) == up(rows * slots * 64 * 4) + up(rows * slots * 8)


def test_tensor_memory_is_taken_between_the_wait_and_the_launch():
    """The wait for tensor memory has no limit.  Columns taken before the kernels ahead are done may be columns that one
    of them still needs; kernels behind that are let go before the columns are there may take them (the GEMM does,
    while it waits)."""
    import os
    from bit_exact_speculative_gb300 import build
    text = open(os.path.join(build.CSRC, "attn_q8.cu")).read()
    body = text[text.index("attn_q8_kernel(const __grid_constant__"):]
    body = body[:body.index("constexpr int CB_SLOTS")]
    at = [body.index(name + "(") for name in ("griddep_wait", "tmem_alloc", "griddep_launch")]
    assert at == sorted(at)
    assert body.count("griddep_launch(") == body.count("tmem_alloc(") == 1


def test_split_boundaries_past_every_position(xv):
    """Rising to the last split that an int can say, and 2^31 - 1 from there on."""
    at = xv.xv_attn_q8_split_begin
    last = next(s for s in range(2_090_000, 2_110_000) if at(s + 1) == 2 ** 31 - 1)
    assert at(last) % 1024 == 0 and 2 ** 31 - 1024 <= at(last) < 2 ** 31 - 1 and at(last) - at(last - 1) == 1024
    for s in (last + 2, 2 ** 22, 2 ** 30, 2 ** 31 - 1):
        assert at(s) == 2 ** 31 - 1, s


def test_what_two_terms_hold_of_q():
    """The two e4m3 terms of a q whose row's largest value lies in [128, 256), as the attention scales it: exact for
    values from 2^-9 of the largest on, and off by at most 2^-17 of it for smaller ones (2^-10, half of e4m3's smallest
    step, against 128).  Every significand of bf16 at every size that matters, and the bound is reached."""
    m = 1 + torch.arange(128, dtype=torch.float32) / 128
    x = torch.cat([m * 2.0 ** e for e in range(-20, 8)])        # up to 255, all of them bf16
    e4m3 = lambda v: v.to(torch.float8_e4m3fn).float()   # noqa: E731
    first = e4m3(x)
    off = (x - first - e4m3(x - first)).abs()
    assert not off[x >= 0.25].any() and 0.25 == 128 * 2.0 ** -9
    assert off.max() == 2.0 ** -10 == 128 * 2.0 ** -17
