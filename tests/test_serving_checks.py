"""The Python entry points of the serving operators refuse a tensor that the library would read or
write past its end: of another type, strided, too small, or in other memory.  Every refusal comes
before the library is called, so host tensors stand in here for the device's."""
import pytest
import torch


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


B, N, Hq, Hkv, hd, page, n_pages, Lmax, M = 3, 5, 4, 2, 64, 64, 7, 192, 15


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def i64(*shape):
    return torch.zeros(shape, dtype=torch.int64)


def rows(m, width):
    return torch.zeros((m, width), dtype=torch.bfloat16)


def calls(xv):
    """Each entry point with arguments of the right types and the least sizes (as on the device)."""
    pages = xv.kv_pages(i32(B, 3), page, n_pages)
    pool = lambda: torch.zeros((n_pages, Hkv, page, hd), dtype=torch.int16)   # noqa: E731
    cache = lambda: torch.zeros((B, Hkv, Lmax, hd), dtype=torch.int16)   # noqa: E731
    ws = lambda: torch.zeros(1 << 20, dtype=torch.uint8)   # noqa: E731
    norms = dict(q_norm=rows(1, hd)[0], k_norm=rows(1, hd)[0], freqs=i64(16), n_rows=i32(1))
    attn = dict(ctx_len=i32(B), kv_src=rows(B * N, 2 * Hkv * hd), parent=i32(B, N), n_nodes=i32(B), N=N, B=B, Hq=Hq, Hkv=Hkv, hd=hd,
                max_ctx=100, scale=0.125, out=rows(B * N, Hq * hd), ws=ws(), gate=rows(B * N, Hq * hd), q=rows(B * N, Hq * hd))
    path = dict(kv_src=rows(B * N, 2 * Hkv * hd), path=i32(B, N), n_keep=i32(B), ctx_len=i32(B), N=N, B=B, Hkv=Hkv, hd=hd)
    return {
        "xv_kv_pages_update": dict(pages=pages, free_pages=i32(n_pages), n_free=i32(1), held=i32(B), ctx_len=i32(B), n_new=i32(B),
                                   row_start=i32(B + 1), pos=i32(M), slots=i64(M), ws=ws(), n_free_out=i32(1), held_out=i32(B)),
        "xv_qk_norm_rope": dict(q=rows(M, Hq * hd), k=rows(M, Hkv * hd), pos=i32(M), Hq=Hq, Hkv=Hkv, hd=hd, q_out=rows(M, Hq * hd),
                                k_out=rows(M, Hkv * hd), **norms),
        "xv_qk_norm_rope_append": dict(q=rows(M, Hq * hd), kv=rows(M, 2 * Hkv * hd), pos=i32(M), slots=i64(M), Hq=Hq, Hkv=Hkv, hd=hd,
                                       q_out=rows(M, Hq * hd), kpool=pool(), vpool=pool(), page_size=page, n_pages=n_pages, **norms),
        "xv_tree_positions": dict(parent=i32(B, N), n_nodes=i32(B), ctx_len=i32(B), pos=i32(B, N)),
        "xv_attn_tree": dict(attn, kc=cache(), vc=cache(), Lmax=Lmax),
        "xv_attn_tree_paged": dict(attn, kpool=pool(), vpool=pool(), pages=pages),
        "xv_tree_accept": dict(tokens=i32(B, N), parent=i32(B, N), n_nodes=i32(B), argmax=i32(B, N), path=i32(B, N), n_keep=i32(B),
                               next_token=i32(B)),
        "xv_kv_append_path": dict(path, Lmax=Lmax, kc=cache(), vc=cache()),
        "xv_kv_append_path_paged": dict(path, pages=pages, kpool=pool(), vpool=pool()),
    }


NAMES = ["xv_kv_pages_update", "xv_qk_norm_rope", "xv_qk_norm_rope_append", "xv_tree_positions", "xv_attn_tree", "xv_attn_tree_paged",
         "xv_tree_accept", "xv_kv_append_path", "xv_kv_append_path_paged"]
# the tensor that fixes a call's sizes: with fewer of it the others are refused, or it is a smaller call
SIZES = {"xv_kv_pages_update": ("ctx_len", "slots"), "xv_qk_norm_rope": ("q", "freqs"), "xv_qk_norm_rope_append": ("q", "freqs"),
         "xv_tree_positions": ("parent",), "xv_tree_accept": ("parent",)}


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(xv, name):
    """All arguments right but for the memory they are in."""
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
        if not torch.is_tensor(t) or k == "ws" or k in SIZES.get(name, ()):
            continue
        with pytest.raises(ValueError, match=f"^{k}:"):
            getattr(xv, name)(**dict(args, **{k: t[:-1]}))
        if t.dtype == torch.bfloat16 and t.dim() == 2:      # rows too narrow
            with pytest.raises(ValueError, match=f"^{k}:"):
                getattr(xv, name)(**dict(args, **{k: t[:, :-1]}))


@pytest.mark.parametrize("name", NAMES)
def test_strided_tensors_are_refused(xv, name):
    """Every other entry of a tensor twice as long; of rows, every other column (rows may be strided)."""
    args = calls(xv)[name]
    for k, t in args.items():
        if not torch.is_tensor(t) or t.numel() < 2:
            continue
        wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
        with pytest.raises(ValueError, match=f"^{k}:"):
            getattr(xv, name)(**dict(args, **{k: wide}))


@pytest.mark.parametrize("name", ["xv_tree_positions", "xv_attn_tree", "xv_tree_accept"])
def test_a_transposed_parent_is_refused(xv, name):
    with pytest.raises(ValueError, match="^parent:"):
        getattr(xv, name)(**dict(calls(xv)[name], parent=i32(N, B).t()))


def test_rows_of_sizes_beside_the_tensors(xv):
    """N, B and a pool's pages are given beside the tensors: more of them than the tensors hold."""
    for name, more in (("xv_attn_tree", dict(N=N + 1)), ("xv_attn_tree", dict(B=B + 1)), ("xv_attn_tree", dict(Lmax=Lmax + 1)),
                       ("xv_attn_tree", dict(Hkv=4)), ("xv_kv_append_path", dict(N=N + 1)), ("xv_kv_append_path", dict(Lmax=Lmax + 1)),
                       ("xv_qk_norm_rope_append", dict(n_pages=n_pages + 1)), ("xv_qk_norm_rope", dict(Hq=Hq + 1)),
                       ("xv_qk_norm_rope", dict(hd=128))):
        with pytest.raises(ValueError):
            getattr(xv, name)(**dict(calls(xv)[name], **more))
    for name in ("xv_kv_pages_update", "xv_attn_tree_paged", "xv_kv_append_path_paged"):
        with pytest.raises(ValueError, match="page_table"):
            getattr(xv, name)(**dict(calls(xv)[name], pages=xv.kv_pages(i32(B - 1, 3), page, n_pages)))
    for name in ("xv_attn_tree_paged", "xv_kv_append_path_paged"):
        with pytest.raises(ValueError, match="kpool"):
            getattr(xv, name)(**dict(calls(xv)[name], pages=xv.kv_pages(i32(B, 3), page, n_pages + 1)))


def test_page_tables_of_other_types_and_layouts_are_refused(xv):
    for bad in (i64(B, 3), i32(B, 6)[:, :3], i32(3, B).t(), i32(3)):
        with pytest.raises(ValueError, match="page_table"):
            xv.kv_pages(bad, page, n_pages)


def test_rows_may_be_strided_and_have_more_dimensions(xv):
    """Columns of a wider projection, heads as a dimension of their own: refused for their memory alone."""
    proj = rows(M, (2 * Hq + 2 * Hkv) * hd)
    args = calls(xv)["xv_qk_norm_rope"]
    for q in (proj[:, : Hq * hd], proj, proj[:, : Hq * hd].unflatten(1, (Hq, hd))):
        with pytest.raises(ValueError, match="current device"):
            xv.xv_qk_norm_rope(**dict(args, q=q, q_out=q))
    with pytest.raises(ValueError, match="^q:"):      # heads apart
        xv.xv_qk_norm_rope(**dict(args, q=torch.zeros((M, Hq, 2 * hd), dtype=torch.bfloat16)[..., :hd]))


def test_attn_tree_sizes_past_what_the_kernels_index(xv):
    """Positions are 32-bit ints in the kernels, and max_ctx + N is one on the way: past 2^30 positions the
    call is refused, whatever the workspace is said to hold, and no workspace is sized."""
    import ctypes
    P, L = ctypes.c_void_p(0x10000), xv.lib()

    def call(Lmax, max_ctx):
        return L.xv_attn_tree(P, 1024, P, P, P, P, 1024, P, None, 16, 2, 4, 2, 256, Lmax, max_ctx, 0.0625, None, 0, P, 1024, P,
                              1 << 50, None)

    top = 2 ** 31 - 1
    for Lmax, max_ctx in ((top, top), (top, top - 16), (top, top - 15), (top, (1 << 30) + 1), ((1 << 30) + 1, (1 << 30) + 1)):
        assert call(Lmax, max_ctx) == xv.XV_ERR_UNSUPPORTED, (Lmax, max_ctx)
        assert b"2^30" in L.xv_last_error()
        assert xv.xv_attn_tree_workspace_size(2, 16, 4, 256, max_ctx) == 0
    size = xv.xv_attn_tree_workspace_size
    assert size(2, 16, 4, 256, 1 << 30) > 0 and size(65535, 64, 4, 64, 0) > 0 and size(1, 1, 1, 128, 0) > 0
    for bad in ((2, 16, 4, 96, 500), (2, 16, 4, 512, 500), (65536, 16, 4, 256, 500), (2, 16, 0, 256, 500), (2, 16, 4, 256, -1),
                (65535, 64, 512, 256, 500)):      # the last: more than 2^30 rows
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("rot,base,scale", [(64, 1e4, 1.0), (128, 1e7, 1.0), (16, 500000.0, 8.0), (256, 1e6, 0.3), (64, 10000, 4), (2, 1e4, 1.0)])
def test_rope_freqs_are_the_nearest_fractions(xv, rot, base, scale):
    """Every entry is the binary fraction of 64 bits nearest to its turns, so the angle at position 2^31 is
    within 2^-33 of a turn; a double's 53 bits leave 2^-24, which an fp32 sine shows."""
    from decimal import Context, Decimal, localcontext
    from fractions import Fraction

    with localcontext(Context(prec=60)):
        def arctan_inverse(n):      # sum of (-1)^k / ((2 k + 1) n^(2 k + 1))
            return sum((-1) ** k / (Decimal(2 * k + 1) * Decimal(n) ** (2 * k + 1)) for k in range(60))
        pi = 16 * arctan_inverse(5) - 4 * arctan_inverse(239)
        want = [(Decimal(-2 * i) / rot * Decimal(base).ln()).exp() / (2 * pi * Decimal(scale)) for i in range(rot // 2)]
    got = xv.rope_freqs(rot, base, scale, device="cpu")
    assert got.dtype == torch.int64 and got.shape == (rot // 2,)
    for x, w in zip(got.tolist(), want):
        assert abs(Fraction(x % 2 ** 64, 2 ** 64) - Fraction(w)) <= Fraction(500001, 1000000) / 2 ** 64


def test_the_current_stream_is_found_without_torchs_private_name(xv, monkeypatch):
    """The raw handle and the device come from private functions of torch where there are such, else from
    the public ones: the same."""
    import importlib.util
    import types

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=700 + dev))
    spec = importlib.util.spec_from_file_location("xv_without_private_names", xv.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m._stream() == 703 and m._on(3) == 703
