"""The serving operators as a server uses them: whole steps one after another, eager and from a
captured graph, ragged batches whose items persistent CTAs take in runs, calls on several streams,
and pools past 2^32 elements.  Comparisons are of bits unless a test says otherwise."""
import numpy as np
import pytest
import torch

import synth
from _gpu import dev, f64, host_u16, same_bits
from test_tree_gpu import bits, cache, check, decode_bits, i32, parents, rows, run, tree, walk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


def batch(seed, B, N, Hq, Hkv, hd, low, high, kinds=("mixed", "wide", "pairs", "chain", "star")):
    """Lengths low..high (both present) and trees of 0..N nodes (both present), with their inputs."""
    rng = np.random.default_rng(seed)
    ctx = [high, low] + [int(x) for x in rng.integers(low, high + 1, B - 2)]
    counts = [N, N, 0] + [int(x) for x in rng.integers(0, N + 1, B - 3)]
    trees = [tree(kinds[b % len(kinds)], n, rng) if n else [] for b, n in enumerate(counts)]
    name = f"serving{seed}.{hd}.{N}"
    return ctx, counts, trees, rows(seed, B, N, Hq, Hkv, hd, name), cache(seed, B, Hkv, max(high, 1), hd, name)


@pytest.mark.parametrize("hd,Hq,Hkv,N,B,low,high,gate", [
    (64, 4, 2, 64, 180, 0, 200, False),      # every item a tail, many in a row
    (128, 8, 2, 13, 64, 0, 1500, True),      # splits without and with a tail
    (128, 32, 8, 40, 12, 440, 520, False),   # trees that reach into the split after, two row tiles
    (256, 6, 1, 30, 60, 0, 1100, True),
    (64, 16, 1, 33, 24, 4000, 4200, False)])  # around the change of the splits' length, five row tiles
def test_ragged_batches_equal_their_sequences_alone(xv, hd, Hq, Hkv, N, B, low, high, gate):
    ctx, counts, trees, proj, (kc, vc) = batch(11, B, N, Hq, Hkv, hd, low, high)
    X, K, V, par, n = dev(proj), dev(kc), dev(vc), parents(trees, N), i32(counts)
    out = run(xv, X, K, V, ctx, par, n, N, Hq, Hkv, hd, gate=gate, fill=3)
    for b in range(B):
        one = run(xv, X[b * N:(b + 1) * N], K[b:b + 1], V[b:b + 1], [ctx[b]], par[b:b + 1], n[b:b + 1], N, Hq, Hkv, hd,
                  gate=gate, fill=3)
        assert same_bits(out[b * N:(b + 1) * N].contiguous(), one), f"sequence {b}: ctx {ctx[b]}, {counts[b]} nodes"
    S = min(B, 16)
    check(out[: S * N], proj[: S * N], kc[:S], vc[:S], ctx[:S], trees[:S], N, Hq, Hkv, hd, gate, "batch", nodes=(0, N // 2, N - 1))
    for _ in range(10):
        assert same_bits(out, run(xv, X, K, V, ctx, par, n, N, Hq, Hkv, hd, gate=gate, fill=3))
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,N,B,low,high", [
    (128, 32, 8, 40, 12, 100, 1500),    # two row tiles
    (64, 16, 1, 56, 24, 400, 1200),     # seven
    (256, 24, 4, 60, 4, 2000, 9000),    # three
    (64, 64, 1, 63, 8, 0, 700),         # 32, the last one short; too many for whole bundles of CTAs
    (64, 3, 1, 64, 200, 0, 200)])       # two, every item a tail
def test_row_tiles_of_full_trees(xv, hd, Hq, Hkv, N, B, low, high):
    """All trees have all their row tiles, which then go side by side to CTAs; some sequences have
    none or a bad length."""
    ctx, counts, trees, proj, (kc, vc) = batch(17, B, N, Hq, Hkv, hd, low, high)
    rng = np.random.default_rng(1)
    trees = [tree("mixed", N, rng) if b != 2 else [] for b in range(B)]
    counts = [len(t) for t in trees]
    X, K, V, par, n = dev(proj), dev(kc), dev(vc), parents(trees, N), i32(counts)
    given = list(ctx)
    given[3] = high + 1
    out = run(xv, X, K, V, given, par, n, N, Hq, Hkv, hd, max_ctx=high, fill=3).reshape(B, N, -1)
    assert bits(xv) == 4
    for b in range(B):
        one = run(xv, X[b * N:(b + 1) * N], K[b:b + 1], V[b:b + 1], [ctx[b]], par[b:b + 1], n[b:b + 1], N, Hq, Hkv, hd, fill=3)
        assert (out[b] == 3).all() if b in (2, 3) else same_bits(out[b], one), f"sequence {b}: ctx {ctx[b]}"
    check(out.reshape(B * N, -1)[: 2 * N], proj[: 2 * N], kc[:2], vc[:2], ctx[:2], trees[:2], N, Hq, Hkv, hd, False, "full", nodes=(0, 20, N - 1))
    assert xv.xv_device_check() == 0


def test_bad_sequences_of_a_large_batch_leave_the_others(xv):
    """Lengths out of range are reported and their rows left; all sequences bad is an empty call."""
    hd, Hq, Hkv, N, B = 128, 8, 2, 13, 80
    ctx, counts, trees, proj, (kc, vc) = batch(12, B, N, Hq, Hkv, hd, 0, 1200)
    X, K, V, par, n = dev(proj), dev(kc), dev(vc), parents(trees, N), i32(counts)
    want = run(xv, X, K, V, ctx, par, n, N, Hq, Hkv, hd, fill=3).reshape(B, N, -1)
    wrong = list(ctx)
    spoiled = {0: -5, 17: 1201, 40: 2 ** 31 - 1, 79: -2 ** 31}
    for b, c in spoiled.items():
        wrong[b] = c
    got = run(xv, X, K, V, wrong, par, n, N, Hq, Hkv, hd, max_ctx=1200, fill=3).reshape(B, N, -1)
    assert bits(xv) == 4
    for b in range(B):
        assert (got[b] == 3).all() if b in spoiled else same_bits(got[b], want[b]), b
    got = run(xv, X, K, V, [-1] * B, par, n, N, Hq, Hkv, hd, max_ctx=1200, fill=3)
    assert bits(xv) == 4 and (got == 3).all()
    got = run(xv, X, K, V, ctx, par, i32([0] * B), N, Hq, Hkv, hd, fill=3)
    assert bits(xv) == 0 and (got == 3).all()


@pytest.mark.parametrize("ctx", [[100, 31], [700, 100]])   # one split; two and a combine
def test_outputs_of_any_stride_and_alignment(xv, ctx):
    """out and gate rows need no alignment: odd strides, a first element off 16 bytes."""
    hd, Hq, Hkv, N, L = 64, 4, 2, 9, ctx[0]
    trees = [tree("mixed", N, np.random.default_rng(1))] * 2
    proj, (kc, vc) = rows(13, 2, N, Hq, Hkv, hd, "odd"), cache(13, 2, Hkv, L, hd, "odd")
    X, K, V, par = dev(proj), dev(kc), dev(vc), parents(trees, N)
    want = run(xv, X, K, V, ctx, par, None, N, Hq, Hkv, hd, gate=True)
    wide = torch.full((2 * N, Hq * hd + 7), 5, dtype=torch.int16, device="cuda")
    gates = torch.zeros((2 * N, Hq * hd + 3), dtype=torch.int16, device="cuda")
    gates[:, 1: 1 + Hq * hd] = X[:, Hq * hd: 2 * Hq * hd]
    xv.xv_attn_tree(X, K, V, i32(ctx), X[:, 2 * Hq * hd:], par, None, N, 2, Hq, Hkv, hd, L, L, hd ** -0.5, wide[:, 3: 3 + Hq * hd],
                    xv.workspace(xv.xv_attn_tree_workspace_size(2, N, Hq, hd, L)), gate=gates[:, 1: 1 + Hq * hd])
    assert same_bits(wide[:, 3: 3 + Hq * hd].contiguous(), want)
    assert (wide[:, :3] == 5).all() and (wide[:, 3 + Hq * hd:] == 5).all() and xv.xv_device_check() == 0


class Server:
    """B sequences over a page pool: one prompt, then verify steps of drafted trees, all on the device."""

    def __init__(self, xv, B, N, Hq, Hkv, hd, page, n_pages, max_ctx, max_rows):
        self.xv, self.dims, self.max_ctx = xv, (B, N, Hq, Hkv, hd, page, n_pages), max_ctx
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")
        self.table = torch.full((B, -(-max_ctx // page)), -1, dtype=torch.int32, device="cuda")
        self.pages = xv.kv_pages(self.table, page, n_pages)
        self.free = i32(np.random.default_rng(0).permutation(n_pages))
        self.n_free, self.held, self.ctx, self.new = i32([n_pages]), z(B), z(B), z(B)
        self.start, self.pos, self.slots = z(B + 1), z(max_rows), z(max_rows, t=torch.int64)
        self.kp, self.vp = z(n_pages, Hkv, page, hd, t=torch.int16), z(n_pages, Hkv, page, hd, t=torch.int16)
        self.tpos, self.path, self.keep, self.next = z(B, N), z(B, N), z(B), z(B)
        self.out = z(B * N, Hq * hd, t=torch.int16)
        self.ws_pages = xv.workspace(xv.xv_kv_pages_workspace_size(B))
        self.ws = xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, max_ctx))
        self.rope = dict(q_norm=dev(synth.normal_bf16(1, 1, (hd,), 0.3)), k_norm=dev(synth.normal_bf16(1, 2, (hd,), 0.3)),
                         freqs=xv.rope_freqs(hd // 2, 1e6))

    def grow(self):
        self.xv.xv_kv_pages_update(self.pages, self.free, self.n_free, self.held, self.ctx, self.new, self.start, self.pos,
                                   self.slots, self.ws_pages)

    def prompt(self, X, lengths):
        """X: projection rows of all prompts, one after another."""
        B, N, Hq, Hkv, hd, page, n_pages = self.dims
        self.new.copy_(lengths)
        self.grow()
        q = torch.empty((X.shape[0], Hq * hd), dtype=torch.int16, device="cuda")
        self.xv.xv_qk_norm_rope_append(X, X[:, 2 * Hq * hd:], self.pos[: X.shape[0]], self.slots[: X.shape[0]], Hq, Hkv, hd, q, self.kp,
                                       self.vp, page, n_pages, **self.rope)
        self.ctx.add_(self.new)

    def verify(self, X, par, n_nodes, tokens, argmax):
        """One step over the trees; X's q and k columns are normed and rotated in place."""
        B, N, Hq, Hkv, hd, page, n_pages = self.dims
        q, kv = X[:, : Hq * hd], X[:, 2 * Hq * hd:]
        self.xv.xv_tree_positions(par, n_nodes, self.ctx, self.tpos)
        self.xv.xv_qk_norm_rope(q, kv, self.tpos.view(-1), Hq, Hkv, hd, q, kv, **self.rope)
        self.xv.xv_attn_tree_paged(q, self.kp, self.vp, self.pages, self.ctx, kv, par, n_nodes, N, B, Hq, Hkv, hd, self.max_ctx,
                                   hd ** -0.5, self.out, self.ws, gate=X[:, Hq * hd: 2 * Hq * hd])
        self.xv.xv_tree_accept(tokens, par, n_nodes, argmax, self.path, self.keep, self.next)
        self.new.copy_(self.keep)
        self.grow()
        self.xv.xv_kv_append_path_paged(kv, self.path, self.keep, self.ctx, N, B, Hkv, hd, self.pages, self.kp, self.vp)
        self.ctx.add_(self.keep)

    def state(self):
        return [x.clone() for x in (self.table, self.free, self.n_free, self.held, self.ctx, self.kp, self.vp, self.out, self.path,
                                    self.keep, self.next)]

    def contiguous(self, b, length):
        """The pool's first `length` positions of sequence b, K and V [1, Hkv, length, hd]."""
        page = self.dims[5]
        t = self.table[b].cpu().numpy()
        return [np.concatenate([p[t[j]][:, : min(page, length - j * page)] for j in range(-(-length // page))], 1)[None]
                for p in (host_u16(self.kp), host_u16(self.vp))]


def drafts(seed, steps, B, N, Hq, Hkv, hd):
    """Trees, tokens, argmaxes (a vocabulary of 3, so that paths are kept) and rows of some steps."""
    rng = np.random.default_rng(seed)
    out = []
    for s in range(steps):
        counts = [N, 1, 0, N - 1][: B] if s % 2 else [N, N // 2, N, 1][: B]
        trees = [tree(["mixed", "pairs", "chain", "wide"][(s + b) % 4], n, rng) if n else [] for b, n in enumerate(counts)]
        tokens, argmax = rng.integers(0, 3, (B, N)).astype(np.int32), rng.integers(0, 3, (B, N)).astype(np.int32)
        out.append((counts, trees, tokens, argmax, rows(seed + s, B, N, Hq, Hkv, hd, f"step{s}")))
    return out


@pytest.mark.parametrize("hd,Hq,Hkv", [(64, 4, 2), (256, 6, 1)])
def test_steps_of_a_server(xv, hd, Hq, Hkv):
    """A prompt and verify steps: outputs within the formula's bound, the kept paths the host's, and
    every kept row the bits of a decode row over the cache that the step left."""
    B, N, page, n_pages, prompts = 3, 24, 64, 40, [70, 250, 1]
    s = Server(xv, B, N, Hq, Hkv, hd, page, n_pages, 500, 400)
    s.prompt(dev(rows(50, 1, sum(prompts), Hq, Hkv, hd, "prompt")), i32(prompts))
    ctx, kept = list(prompts), 0
    for counts, trees, tokens, argmax, proj in drafts(60, 4, B, N, Hq, Hkv, hd):
        before = [s.contiguous(b, ctx[b]) for b in range(B)]
        X = dev(proj)
        s.verify(X, parents(trees, N), i32(counts), i32(tokens), i32(argmax))
        rotated = host_u16(X)
        L = max(ctx)
        kc, vc = (np.concatenate([np.pad(c[j], ((0, 0), (0, 0), (0, L - c[j].shape[2]), (0, 0))) for c in before]) for j in (0, 1))
        check(s.out, rotated, kc, vc, ctx, trees, N, Hq, Hkv, hd, True, "step")
        for b in range(B):
            want = walk(trees[b], tokens[b], argmax[b]) if trees[b] else []
            assert s.path[b, : len(want)].tolist() == want and s.keep[b].item() == len(want)
            after = s.contiguous(b, ctx[b] + len(want))
            heads = rotated.reshape(B, N, 2 * Hq + 2 * Hkv, hd)[b]
            for c, old, o in zip(after, before[b], (2 * Hq, 2 * Hq + Hkv)):
                assert np.array_equal(c[:, :, : ctx[b]], old)
                assert np.array_equal(c[0, :, ctx[b]:], heads[want, o: o + Hkv].transpose(1, 0, 2))
            for t, i in enumerate(want):
                one = decode_bits(xv, rotated, kc, vc, ctx[b], trees[b], b, N, i, Hq, Hkv, hd, True)
                assert same_bits(s.out[b * N + i], one)
            ctx[b] += len(want)
            kept += len(want)
        assert s.ctx.tolist() == ctx
    assert kept > 8 and xv.xv_device_check() == 0


def test_a_captured_step_replays_like_the_eager_one(xv):
    """The whole step in a graph, replayed over changing drafts, beside a second graph of another
    server that shares the workspaces."""
    hd, Hq, Hkv, B, N = 128, 8, 2, 4, 24
    prompts = [70, 250, 1, 129]
    P = dev(rows(70, 1, sum(prompts), Hq, Hkv, hd, "prompt"))
    steps = drafts(80, 4, B, N, Hq, Hkv, hd)
    servers = [Server(xv, B, N, Hq, Hkv, hd, 64, 40, 500, 500) for _ in range(3)]
    for s in servers:
        s.prompt(P, i32(prompts))
    eager, *captured = servers
    buf = [torch.zeros_like(dev(steps[0][4])), *(torch.zeros((B, N), dtype=torch.int32, device="cuda") for _ in range(3)), i32([0] * B)]
    fresh = captured[0].state()
    captured[1].ws, captured[1].ws_pages = captured[0].ws, captured[0].ws_pages
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                s.verify(buf[0], buf[1], buf[4], buf[2], buf[3])
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(fresh, captured[0].state()):
        assert torch.equal(a, b), "capturing ran something"
    for counts, trees, tokens, argmax, proj in steps:
        eager.verify(dev(proj), parents(trees, N), i32(counts), i32(tokens), i32(argmax))
        for g, s in zip(graphs, captured):
            for x, y in zip(buf, (dev(proj), parents(trees, N), i32(tokens), i32(argmax), i32(counts))):
                x.copy_(y)
            g.replay()
        for s in captured:
            for a, b in zip(eager.state(), s.state()):
                assert torch.equal(a, b)
    assert xv.xv_device_check() == 0


def test_calls_at_once_on_two_streams(xv):
    """Two batches on two streams with a workspace each, over and over: the bits of each alone."""
    cases = [(128, 8, 2, 13, 20, 0, 1500), (256, 6, 1, 30, 6, 0, 3000)]
    made = []
    for hd, Hq, Hkv, N, B, low, high in cases:
        ctx, counts, trees, proj, (kc, vc) = batch(14, B, N, Hq, Hkv, hd, low, high)
        X, K, V, par, n = dev(proj), dev(kc), dev(vc), parents(trees, N), i32(counts)
        want = run(xv, X, K, V, ctx, par, n, N, Hq, Hkv, hd)
        made.append((X, K, V, i32(ctx), par, n, N, B, Hq, Hkv, hd, max(high, 1), max(ctx), want, torch.zeros_like(want),
                     xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, max(ctx))), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for X, K, V, c, par, n, N, B, Hq, Hkv, hd, Lmax, m, want, out, ws, stream in made:
            with torch.cuda.stream(stream):
                out.zero_()
                xv.xv_attn_tree(X, K, V, c, X[:, 2 * Hq * hd:], par, n, N, B, Hq, Hkv, hd, Lmax, m, hd ** -0.5, out, ws)
    torch.cuda.synchronize()
    for *_, want, out, ws, stream in made:
        assert same_bits(out, want)
    assert xv.xv_device_check() == 0


def test_pools_past_2_to_the_32_elements(xv):
    """Pages whose offsets pass 2^32 elements are read and written like any others."""
    hd, Hq, Hkv, N, page, ctx = 128, 8, 8, 20, 256, 600
    n_pages = 2 ** 32 // (Hkv * page * hd) + 8
    pools = [torch.empty((n_pages, Hkv, page, hd), dtype=torch.int16, device="cuda") for _ in range(2)]
    small = [torch.zeros((3, Hkv, page, hd), dtype=torch.int16, device="cuda") for _ in range(2)]
    table = [n_pages - 1, 2, n_pages - 2]
    big, ref = xv.kv_pages(t0 := i32([table]), page, n_pages), xv.kv_pages(t1 := i32([[0, 1, 2]]), page, 3)
    M = ctx
    X = dev(rows(15, 1, M, Hq, Hkv, hd, "big"))
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    q = torch.empty((M, Hq * hd), dtype=torch.int16, device="cuda")
    for (kp, vp), t in ((pools, table), (small, [0, 1, 2])):
        slots = torch.tensor([t[p // page] * page + p % page for p in range(M)], dtype=torch.int64, device="cuda")
        xv.xv_qk_norm_rope_append(X, X[:, 2 * Hq * hd:], pos, slots, Hq, Hkv, hd, q, kp, vp, page, kp.shape[0], freqs=xv.rope_freqs(hd))
    par = parents([tree("mixed", N, np.random.default_rng(3))], N)
    T = dev(rows(16, 1, N, Hq, Hkv, hd, "bigtree"))
    outs = []
    for (kp, vp), pg in ((pools, big), (small, ref)):
        out = torch.zeros((N, Hq * hd), dtype=torch.int16, device="cuda")
        xv.xv_attn_tree_paged(T, kp, vp, pg, i32([ctx]), T[:, 2 * Hq * hd:], par, None, N, 1, Hq, Hkv, hd, ctx, hd ** -0.5, out,
                              xv.workspace(xv.xv_attn_tree_workspace_size(1, N, Hq, hd, ctx)))
        xv.xv_kv_append_path_paged(T[:, 2 * Hq * hd:], i32([list(range(N))]), i32([N]), i32([ctx]), N, 1, Hkv, hd, pg, kp, vp)
        outs.append(out)
    assert same_bits(outs[0], outs[1])
    for p, s in zip(pools, small):
        for j, t in enumerate(table):
            filled = min(page, ctx + N - j * page)
            assert same_bits(p[t, :, :filled].contiguous(), s[j, :, :filled].contiguous())
    assert xv.xv_device_check() == 0
