"""Calls at the edges of what the serving operators take: tensors in host memory among the device's, counters in
place, batches of mostly idle requests, the roundings of a gated output."""
import pytest
import torch

from test_serving_checks import NAMES, calls

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


def on_device(xv, name):
    args = {k: t.cuda() if torch.is_tensor(t) else t for k, t in calls(xv)[name].items()}
    if "pages" in args:
        args["pages"] = xv.kv_pages(args["pages"]._table.cuda(), args["pages"].page_size, args["pages"].n_pages)
    return args


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_in_host_memory_is_refused(xv, name):
    """Each tensor in turn, the first one among them (it says which device the others must be on)."""
    args = on_device(xv, name)
    for k, t in args.items():
        if torch.is_tensor(t):
            with pytest.raises(ValueError, match="device"):
                getattr(xv, name)(**dict(args, **{k: t.cpu()}))
    if "pages" in args:
        with pytest.raises(ValueError, match="page_table"):
            getattr(xv, name)(**dict(args, pages=xv.kv_pages(args["pages"]._table.cpu(), args["pages"].page_size, args["pages"].n_pages)))
    getattr(xv, name)(**args)      # the least sizes are enough
    getattr(xv, name)(**args, stream=torch.cuda.current_stream())
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("B", [1, 40, 1024])
def test_page_updates_in_place_equal_those_apart(xv, B):
    """The counters in the place of the old ones are written only after every CTA has read those: call
    after call over rows for many CTAs, against the same calls with outputs of their own."""
    page, most, steps = 64, 40, 60
    g = torch.Generator().manual_seed(B)
    new = [torch.randint(-1, most + 1, (B,), generator=g, dtype=torch.int32).cuda() for _ in range(steps)]
    states = []
    for apart in (False, True):
        table = torch.full((B, 60), -1, dtype=torch.int32, device="cuda")
        pages = xv.kv_pages(table, page, 60 * B + 1)
        free = torch.arange(60 * B + 1, dtype=torch.int32, device="cuda")
        n_free, held, ctx = torch.tensor([60 * B + 1], dtype=torch.int32).cuda(), *(torch.zeros(B, dtype=torch.int32).cuda() for _ in range(2))
        start, pos = torch.zeros(B + 1, dtype=torch.int32).cuda(), torch.zeros(B * most, dtype=torch.int32).cuda()
        slots, ws = torch.zeros(B * most, dtype=torch.int64).cuda(), xv.workspace(xv.xv_kv_pages_workspace_size(B))
        seen = []
        for n in new:
            if apart:
                nf, h = torch.zeros_like(n_free), torch.zeros_like(held)
                xv.xv_kv_pages_update(pages, free, n_free, held, ctx, n, start, pos, slots, ws, n_free_out=nf, held_out=h)
                n_free, held = nf, h
            else:
                xv.xv_kv_pages_update(pages, free, n_free, held, ctx, n, start, pos, slots, ws)
            ctx = torch.where(n < 0, 0, ctx + n)
            seen += [x.clone() for x in (table, free, n_free, held, start, pos, slots)]
        states.append(seen)
    assert all(torch.equal(a, b) for a, b in zip(*states))
    assert xv.xv_device_check() == 0


def gpu_us(run, reps=20):
    """Least time of a call among its like in a graph, in us."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for _ in range(reps):
            run()
    best = float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000 / reps)
    return best


@pytest.mark.parametrize("B", [1, 2, 31, 33, 1024, 1025, 65535])
@pytest.mark.parametrize("where", ["ends", "every 97th", "last"])
def test_rows_find_their_request_past_idle_ones(xv, B, where):
    """Few requests with new rows among many without: positions and slots, and no more time than a row
    for every request takes (a walk from request to request took 6 times that for 1024 requests)."""
    page, counts = 64, torch.zeros(B, dtype=torch.int32)
    if where == "ends":
        counts[0], counts[-1] = 21, 43
    elif where == "last":
        counts[-1] = 5
    else:
        counts[::97] = 1 + torch.arange(len(counts[::97]), dtype=torch.int32) % 3
    idle = torch.arange(B) % 2 == 1      # idle, or finished without a page
    ctx = (torch.arange(B, dtype=torch.int32) * 37) % 120
    table = torch.full((B, 4), -1, dtype=torch.int32)
    held = (ctx + page - 1) // page
    first = torch.cumsum(held, 0) - held
    for j in range(2):
        table[held > j, j] = (first + j)[held > j].int()
    done = idle & (counts == 0) & (held == 0)
    n_pages = int(held.sum()) + 2 * B + 8
    used, total = int(held.sum()), int(counts.sum())

    def state(new, rows):
        d = dict(pages=xv.kv_pages(table.cuda(), page, n_pages), held=held.int().cuda(), ctx_len=ctx.cuda(), n_new=new.cuda(),
                 n_free=torch.tensor([n_pages - used], dtype=torch.int32).cuda(), row_start=torch.zeros(B + 1, dtype=torch.int32).cuda(),
                 free_pages=torch.arange(used, used + n_pages, dtype=torch.int32).clamp_max(n_pages - 1).cuda(),
                 pos=torch.full((rows,), -7, dtype=torch.int32).cuda(), slots=torch.full((rows,), -7, dtype=torch.int64).cuda(),
                 ws=xv.workspace(xv.xv_kv_pages_workspace_size(B)))
        return dict(d, n_free_out=torch.zeros_like(d["n_free"]), held_out=torch.zeros_like(d["held"]))

    s = state(torch.where(done, torch.tensor(-1, dtype=torch.int32), counts), total + 3)
    xv.xv_kv_pages_update(**s)
    seq = torch.repeat_interleave(torch.arange(B), counts.long())
    start = torch.cumsum(counts, 0) - counts
    want = ctx[seq].long() + torch.arange(total) - start[seq]
    after = s["pages"]._table.cpu().long()
    assert s["pos"].tolist() == want.tolist() + [-7] * 3
    assert s["slots"].tolist() == (after[seq, want // page] * page + want % page).tolist() + [-7] * 3
    assert xv.xv_device_check() == 0
    dense = state(torch.ones(B, dtype=torch.int32), B)
    few, all_of_them = (gpu_us(lambda x=x: xv.xv_kv_pages_update(**x)) for x in (s, dense))
    assert few <= 1.5 * all_of_them + 2, f"{few:.1f} us for {total} rows, {all_of_them:.1f} us for {B}"


@pytest.mark.parametrize("ctx", [3, 700])      # one split, finished in place; two and the combine
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_a_gated_output_is_rounded_once_where_no_decode_row_rounds_twice(xv, hd, ctx):
    """Queries of zero and values of whole numbers make everything up to the quotient exact but for one
    fp32 rounding, so a gated output o z is off by half a bf16 step and 2^-20 of it (the quotient's, the
    product's and the logistic's fp32 roundings, 16 of them at most). At hd 64 and 256 a gated output has
    the bits of the decode rows, which round o before the product: another 2^-8 of it."""
    Hq, Hkv, N = 4, 2, 6
    g = torch.Generator().manual_seed(hd + ctx)
    proj = torch.randn((N, (2 * Hq + 2 * Hkv) * hd), generator=g).bfloat16()
    proj[:, : Hq * hd] = 0
    proj[:, (2 * Hq + Hkv) * hd:] = torch.randint(1, 200, (N, Hkv * hd), generator=g).bfloat16()
    kc, vc = torch.randn((1, Hkv, ctx, hd), generator=g).bfloat16(), torch.randint(1, 200, (1, Hkv, ctx, hd), generator=g).bfloat16()
    par = [-1, 0, 1, 1, 0, 3]
    X, out = proj.cuda(), torch.zeros((N, Hq * hd), dtype=torch.bfloat16, device="cuda")
    xv.xv_attn_tree(X, kc.cuda(), vc.cuda(), torch.tensor([ctx], dtype=torch.int32).cuda(), X[:, 2 * Hq * hd:],
                    torch.tensor([par], dtype=torch.int32).cuda(), None, N, 1, Hq, Hkv, hd, ctx, ctx, 0.125, out,
                    xv.workspace(xv.xv_attn_tree_workspace_size(1, N, Hq, hd, ctx)), gate=X[:, Hq * hd: 2 * Hq * hd])
    v = proj[:, (2 * Hq + Hkv) * hd:].double().reshape(N, Hkv, hd)
    z = torch.sigmoid(proj[:, Hq * hd: 2 * Hq * hd].double()).reshape(N, Hq, hd)
    for i in range(N):
        path, a = [], i
        while a >= 0:
            path.append(a)
            a = par[a]
        o = (vc[0].double().sum(1) + v[path].sum(0)) / (ctx + len(path))
        want = o.repeat_interleave(Hq // Hkv, 0) * z[i]
        half = 2.0 ** (torch.floor(torch.log2(want)) - 8)
        tol = half + 2.0 ** -20 * want + (0 if hd == 128 else 2.0 ** -8 * want)
        err = (out[i].double().cpu().reshape(Hq, hd) - want).abs()
        assert (err <= tol).all(), f"node {i}: {int((err > tol).sum())} of {err.numel()} off, worst {float((err / tol).max()):.2f} of the bound"
    assert xv.xv_device_check() == 0
