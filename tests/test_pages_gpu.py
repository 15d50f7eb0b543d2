"""Page tables, positions and slots on the device against the host's page pool: the same pages in
the same order, step after step, for requests that grow, wait and finish."""
import numpy as np
import pytest
import torch

from bit_exact_speculative_gb300.model import KvPagePool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


class Device:
    """The device state of B requests over n_pages pages, and one step on it."""

    def __init__(self, xv, B, page, max_pages, n_pages, order, max_rows):
        self.xv, self.B = xv, B
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.pages = xv.kv_pages(self.table, page, n_pages)
        self.free = i32(order[::-1])
        self.n_free, self.held = i32([len(order)]), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.start = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
        self.pos = torch.full((max_rows,), -7, dtype=torch.int32, device="cuda")
        self.slots = torch.full((max_rows,), -7, dtype=torch.int64, device="cuda")
        self.ws = xv.workspace(xv.xv_kv_pages_workspace_size(B))

    def step(self, ctx, new, **kw):
        self.pos.fill_(-7)
        self.slots.fill_(-7)
        self.xv.xv_kv_pages_update(self.pages, self.free, self.n_free, self.held, i32(ctx), i32(new), self.start, self.pos,
                                   self.slots, self.ws, **kw)


def check(d, pool, ctx, new, page):
    """The device state against the host pool after the same releases and requests."""
    held = d.held.cpu().numpy()
    assert held.tolist() == pool.held
    table = d.table.cpu().numpy()
    for b in range(d.B):
        assert np.array_equal(table[b, :held[b]], pool.host[b, :held[b]]), b
    nf = int(d.n_free.item())
    assert nf == len(pool.free)
    assert d.free[:nf].tolist() == pool.free
    rows = [max(n, 0) for n in new]
    assert d.start.tolist() == [0] + np.cumsum(rows).tolist()
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, rows)]) if sum(rows) else np.zeros(0, int)
    seq = np.repeat(np.arange(d.B), rows)
    slots = [int(pool.host[b, p // page]) * page + p % page for b, p in zip(seq, pos)]
    t = sum(rows)
    assert d.pos[:t].tolist() == pos.tolist()
    assert d.slots[:t].tolist() == slots
    assert (d.pos[t:] == -7).all() and (d.slots[t:] == -7).all(), "rows behind the last request were written"


@pytest.mark.parametrize("B,page,steps,big", [(1, 64, 12, 300), (8, 64, 20, 200), (37, 128, 12, 700), (1500, 64, 5, 90),
                                              (5, 192, 8, 5000)])
def test_steps_equal_the_host_pool(xv, B, page, steps, big):
    """Requests grow by nothing, one row, a page's end and many rows; some finish and start again."""
    rng = np.random.default_rng(B * 1000 + page)
    max_pages = big * 3 // page + 3
    n_pages = B * max_pages + 3
    order = rng.permutation(n_pages).tolist()
    d = Device(xv, B, page, max_pages, n_pages, order, B * big + 9)
    pool = KvPagePool(n_pages, page, B, max_pages, device="cpu", order=order)
    ctx = [0] * B
    for _ in range(steps):
        new = []
        for b in range(B):
            kind = rng.integers(0, 6)
            n = [0, 1, int(rng.integers(1, big + 1)), page - ctx[b] % page, int(rng.integers(1, 9)), -1][kind]
            if n >= 0 and ctx[b] + n > max_pages * page:
                n = -1
            new.append(min(n, big))
        d.step(ctx, new)
        for b in range(B):
            if new[b] < 0:
                pool.release(b)
        for b in range(B):
            if new[b] >= 0:
                pool.ensure(b, ctx[b] + new[b])
        check(d, pool, ctx, new, page)
        ctx = [0 if n < 0 else c + n for c, n in zip(ctx, new)]
    assert xv.xv_device_check() == 0


def test_outputs_apart_leave_the_inputs(xv):
    """With n_free_out and held_out given, a call repeated on the same inputs gives the same pages."""
    d = Device(xv, 3, 64, 6, 20, list(range(20)), 200)
    d.step([0, 0, 0], [100, 64, 1])
    nf, held = torch.zeros_like(d.n_free), torch.zeros_like(d.held)
    got = []
    for _ in range(2):
        d.step([100, 64, 1], [64, -1, 70], n_free_out=nf, held_out=held)
        got.append([x.tolist() for x in (d.table, d.free, nf, held, d.start, d.pos, d.slots)])
    assert got[0] == got[1] and d.held.tolist() == [2, 1, 1] and held.tolist() == [3, 0, 2]
    assert nf.tolist() == [d.n_free.item() + 1 - 2]


def device_bits(xv):
    import ctypes
    code = ctypes.c_uint(0)
    xv.lib().xv_device_check(None, ctypes.byref(code))
    return code.value


def test_too_few_pages_gives_nobody_a_page(xv):
    """All or nothing: the finished request's pages come back, no one gets any, and a row has a slot
    only on a page its request already holds."""
    d = Device(xv, 3, 64, 16, 6, list(range(6)), 600)
    d.step([0, 0, 0], [64, 65, 128])            # 1 + 2 + 2 of 6 pages
    d.step([64, 65, 128], [10, -1, 400])        # back to 3 free, 1 + 7 wanted
    assert device_bits(xv) == 64
    assert d.held.tolist() == [1, 0, 2] and d.n_free.item() == 3
    assert (d.slots[:10] == -1).all() and (d.slots[10:410] == -1).all() and d.pos[:10].tolist() == list(range(64, 74))
    d.step([64, 0, 100], [10, 0, 40])           # 1 + 0 + 1 of 3: fits; positions 100..127 sit on a held page
    assert device_bits(xv) == 0
    assert d.held.tolist() == [2, 0, 3] and d.n_free.item() == 1
    t2 = d.table[2].tolist()
    assert d.slots[10:50].tolist() == [t2[p // 64] * 64 + p % 64 for p in range(100, 140)]


def test_bad_requests_are_recorded_and_get_no_rows(xv):
    d = Device(xv, 5, 64, 2, 40, list(range(40)), 64)
    d.step([0, 100, -5, 0, 0], [8, 40, 3, -2, 8])     # past 128 positions; negative length; bad count
    assert device_bits(xv) == 4 | 8
    assert d.start.tolist() == [0, 8, 8, 8, 8, 16] and d.held.tolist() == [1, 0, 0, 0, 1]
    d.step([8, 0, 0, 0, 8], [40, 0, 0, 0, 40])        # 80 rows into room for 64: the last 16 are dropped
    assert device_bits(xv) == 8
    assert d.start.tolist() == [0, 40, 40, 40, 40, 64] and d.held.tolist() == [1, 0, 0, 0, 1]
    assert d.pos.tolist() == list(range(8, 48)) + list(range(8, 32))
    d.n_free.fill_(41)                                # more free pages than the pool has
    d.step([8, 0, 0, 0, 8], [100, -1, 0, 0, 1])
    assert device_bits(xv) == 8
    assert d.n_free.item() == 41 and d.held.tolist() == [1, 0, 0, 0, 1]
    d.n_free.fill_(38)
    d.table[0, 0] = 40                                # a held page outside the pool
    d.step([8, 0, 0, 0, 8], [2, 0, 0, 0, 1])
    assert device_bits(xv) == 16
    assert d.slots[:2].tolist() == [-1, -1] and d.slots[2].item() == d.table[4, 0].item() * 64 + 8


def test_captured_and_replayed(xv):
    """A captured step replays on the lengths it finds, each replay advancing the state."""
    d = Device(xv, 4, 64, 16, 64, list(range(64)), 256)
    ctx, new = i32([0, 0, 0, 0]), i32([33, 64, 0, 7])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d.xv.xv_kv_pages_update(d.pages, d.free, d.n_free, d.held, ctx, i32([0, 0, 0, 0]), d.start, d.pos, d.slots, d.ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.xv.xv_kv_pages_update(d.pages, d.free, d.n_free, d.held, ctx, new, d.start, d.pos, d.slots, d.ws)
        ctx.add_(new)
    pool = KvPagePool(64, 64, 4, 16, device="cpu")
    lens = [0, 0, 0, 0]
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        for b, n in enumerate([33, 64, 0, 7]):
            pool.ensure(b, lens[b] + n)
        assert d.held.tolist() == pool.held
        assert np.array_equal(d.table.cpu().numpy(), pool.host)
        t = 0
        for b, n in enumerate([33, 64, 0, 7]):
            assert d.slots[t:t + n].tolist() == [int(pool.host[b, p // 64]) * 64 + p % 64 for p in range(lens[b], lens[b] + n)]
            t += n
        lens = [x + n for x, n in zip(lens, [33, 64, 0, 7])]
    assert xv.xv_device_check() == 0
