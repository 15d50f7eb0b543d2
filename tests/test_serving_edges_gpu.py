"""Calls at the edges of what the serving operators take: tensors in host memory among the device's."""
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
