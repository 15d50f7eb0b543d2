"""A tree of drafted tokens: positions, attention over a cache and the tree's own rows, the greedy
walk and the kept path's append, against plain implementations in 64 bits.

Attention tolerance, before any run: with p = softmax and A = sum p |v|, the kernel rounds each
p (unnormalised) to bf16 for its product (at most 2^-8 of it: 2^-8 A on the output) and the output
once (2^-8 |out|).  Scores are fp32 sums of hd products of bf16 values, at most hd roundings of
2^-24 sum |q k| each; exponentials add 2^-22, the sums of L terms in tiles and splits less than
2^-18 here: together e = 2 hd 2^-24 max_p(sum |q k|) scale + 2^-17, taken on A.  An output gate
adds the product's own rounding, 2^-8 |out|, and the logistic's 2^-21."""
import numpy as np
import pytest
import torch

import synth
from _gpu import dev, f64, host_u16, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def tree(kind, n, rng):
    par = [-1]
    for i in range(1, n):
        par.append({"chain": i - 1, "star": 0, "mixed": int(rng.integers(max(0, i - 6), i)),
                    "wide": int(rng.integers(0, max(1, i // 3))), "forest": int(rng.integers(-1, i)),
                    "pairs": (i - 1) // 2}[kind])
    return par


def chain_of(par, i):
    """The nodes from the root to node i."""
    out = []
    while i >= 0:
        out.append(i)
        i = par[i]
    return out[::-1]


def parents(trees, N):
    return i32([t + [-1] * (N - len(t)) for t in trees])


def rows(seed, B, N, Hq, Hkv, hd, name):
    """Projection rows [q | gate | k | v]."""
    return synth.normal_bf16(seed, synth.tid(f"tree.{name}"), (B * N, (2 * Hq + 2 * Hkv) * hd))


def cache(seed, B, Hkv, Lmax, hd, name):
    return tuple(synth.normal_bf16(seed, synth.tid(f"tree.{name}.{x}"), (B, Hkv, Lmax, hd)) for x in "kv")


def run(xv, proj, kc, vc, ctx, par, nodes, N, Hq, Hkv, hd, max_ctx=None, gate=False, fill=0):
    B, Lmax = kc.shape[0], kc.shape[2]
    max_ctx = max(ctx) if max_ctx is None else max_ctx
    out = torch.full((B * N, Hq * hd), fill, dtype=torch.int16, device="cuda")
    ws = xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, max_ctx))
    xv.xv_attn_tree(proj, kc, vc, i32(ctx), proj[:, 2 * Hq * hd:], par, nodes, N, B, Hq, Hkv, hd, Lmax, max_ctx, hd ** -0.5,
                    out, ws, gate=proj[:, Hq * hd:] if gate else None)
    return out


def reference(proj, kc, vc, ctx, par, b, N, i, Hq, Hkv, hd, gate):
    """Node i of sequence b: (out, tolerance), both [Hq, hd]."""
    r = f64(proj).reshape(-1, N, 2 * Hq + 2 * Hkv, hd)[b]
    path = chain_of(par, i)
    G = Hq // Hkv
    K = np.concatenate([f64(kc[b, :, : ctx]), r[path, 2 * Hq: 2 * Hq + Hkv].transpose(1, 0, 2)], 1)
    V = np.concatenate([f64(vc[b, :, : ctx]), r[path, 2 * Hq + Hkv:].transpose(1, 0, 2)], 1)
    out, tol = np.empty((Hq, hd)), np.empty((Hq, hd))
    for h in range(Hq):
        s = K[h // G] @ r[i, h] * hd ** -0.5
        p = np.exp(s - s.max())
        p /= p.sum()
        o, A = p @ V[h // G], p @ np.abs(V[h // G])
        e = 2 * hd * 2.0 ** -24 * float((np.abs(K[h // G]) @ np.abs(r[i, h])).max()) * hd ** -0.5 + 2.0 ** -17
        t = 2.0 ** -8 * (A + np.abs(o)) + e * A
        if gate:
            z = 1 / (1 + np.exp(-r[i, Hq + h]))
            t = (t + 2.0 ** -8 * np.abs(o) + 2.0 ** -21 * np.abs(o)) * z
            o = o * z
        out[h], tol[h] = o, 1.01 * t        # second-order terms
    return out, tol


def check(got, proj, kc, vc, ctx, trees, N, Hq, Hkv, hd, gate, what, nodes=None):
    g = f64(host_u16(got)).reshape(len(ctx), N, Hq, hd)
    for b, par in enumerate(trees):
        for i in range(len(par)) if nodes is None else [n for n in nodes if n < len(par)]:
            ref, tol = reference(proj, kc, vc, ctx[b], par, b, N, i, Hq, Hkv, hd, gate)
            err = np.abs(g[b, i] - ref)
            assert (err <= tol).all(), f"{what}: sequence {b} node {i}: {np.nanmax(err / tol):.2f} of the bound"


@pytest.mark.parametrize("kind", ["chain", "star", "mixed", "forest", "pairs"])
def test_positions(xv, kind):
    rng = np.random.default_rng(3)
    counts, ctx = [64, 1, 0, 33, 50], [0, 7, 9, 100000, 63]
    trees = [tree(kind, n, rng) if n else [] for n in counts]
    pos = torch.full((5, 64), -9, dtype=torch.int32, device="cuda")
    xv.xv_tree_positions(parents(trees, 64), i32(counts), i32(ctx), pos)
    for b, t in enumerate(trees):
        want = [ctx[b] + len(chain_of(t, i)) - 1 for i in range(len(t))]
        assert pos[b].tolist() == want + [-9] * (64 - len(t))
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,N,ctx,kind,gate", [
    (256, 24, 4, 16, [2183], "mixed", True), (64, 2, 1, 8, [128, 1, 0, 63], "mixed", False),
    (128, 8, 2, 13, [511, 512, 513, 64, 700], "wide", False), (64, 6, 2, 64, [15, 16, 17, 448, 500], "star", False),
    (256, 6, 1, 64, [4090, 0, 4096], "mixed", True), (128, 5, 1, 1, [1, 300], "chain", False),
    (64, 1, 1, 64, [47, 4095], "chain", True), (256, 4, 4, 31, [6140, 100], "forest", False),
    (64, 128, 1, 5, [70], "pairs", False), (128, 96, 1, 7, [130, 64], "pairs", False), (64, 8, 8, 64, [65, 127], "wide", False)])
def test_attention_against_the_formula(xv, hd, Hq, Hkv, N, ctx, kind, gate):
    B = len(ctx)
    rng = np.random.default_rng(hd * N + B)
    counts = [N] + [int(rng.integers(0, N + 1)) for _ in ctx[1:]]
    trees = [tree(kind, n, rng) if n else [] for n in counts]
    Lmax = max(ctx) + 3
    proj, (kc, vc) = rows(1, B, N, Hq, Hkv, hd, f"f{hd}{Hq}{N}"), cache(1, B, Hkv, Lmax, hd, f"f{hd}{Hq}{N}")
    got = run(xv, dev(proj), dev(kc), dev(vc), ctx, parents(trees, N), i32(counts), N, Hq, Hkv, hd, gate=gate, fill=77)
    check(got, proj, kc, vc, ctx, trees, N, Hq, Hkv, hd, gate, "attn_tree")
    for b, n in enumerate(counts):
        assert (got.reshape(B, N, -1)[b, n:] == 77).all(), "rows past a tree's nodes were written"
    assert xv.xv_device_check() == 0


def decode_bits(xv, proj, kc, vc, ctx, par, b, N, i, Hq, Hkv, hd, gate):
    """xv_attn_decode_rows for node i of sequence b over a cache that holds its path at ctx.."""
    path = chain_of(par, i)
    r = proj.reshape(-1, N, 2 * Hq + 2 * Hkv, hd)[b]
    L = ctx + len(path)
    K, V = (np.concatenate([c[b, :, :ctx], r[path, o: o + Hkv].transpose(1, 0, 2)], 1)[None] for c, o in
            ((kc, 2 * Hq), (vc, 2 * Hq + Hkv)))
    one = dev(np.ascontiguousarray(proj.reshape(-1, proj.shape[1])[b * N + i][None]))
    out = torch.empty((1, Hq * hd), dtype=torch.int16, device="cuda")
    ws = xv.workspace(xv.xv_attn_workspace_size(1, 1, Hq, hd, L))
    W = proj.shape[1]
    xv.xv_attn_decode_rows(one, W, dev(K), dev(V), i32([L]), 1, 1, Hq, Hkv, hd, L, L, hd ** -0.5, out, Hq * hd, ws,
                           gate=one[:, Hq * hd:] if gate else None, gate_stride=W if gate else 0)
    return out[0]


@pytest.mark.parametrize("hd,Hq,Hkv,N,ctx,kind,gate", [
    (256, 24, 4, 16, [2183], "mixed", True), (64, 2, 1, 64, [128, 0, 63], "mixed", False),
    (64, 6, 2, 64, [15, 16, 17, 448, 470, 512], "star", False), (256, 6, 1, 64, [4090, 4064], "mixed", True),
    (64, 1, 1, 64, [47, 4095, 500], "chain", False), (256, 4, 4, 31, [6140, 100], "forest", False),
    (64, 128, 1, 9, [70], "pairs", False), (256, 12, 2, 40, [40, 33], "pairs", True), (64, 4, 2, 64, [30, 1], "wide", False)])
def test_rows_have_the_bits_of_decode_rows(xv, hd, Hq, Hkv, N, ctx, kind, gate):
    """Every node's row, at depths that cross 16-position groups, tiles and splits, has the bits of a
    decode row over a contiguous cache that holds its path."""
    B = len(ctx)
    rng = np.random.default_rng(hd + N)
    trees = [tree(kind, N - 3 * b, rng) for b in range(B)]
    proj, (kc, vc) = rows(5, B, N, Hq, Hkv, hd, f"b{hd}{Hq}{N}"), cache(5, B, Hkv, max(ctx) + 1, hd, f"b{hd}{Hq}{N}")
    got = run(xv, dev(proj), dev(kc), dev(vc), ctx, parents(trees, N), i32([len(t) for t in trees]), N, Hq, Hkv, hd, gate=gate)
    for b, par in enumerate(trees):
        for i in range(len(par)):
            one = decode_bits(xv, proj, kc, vc, ctx[b], par, b, N, i, Hq, Hkv, hd, gate)
            assert same_bits(got[b * N + i], one), f"sequence {b} (ctx {ctx[b]}) node {i}"
    assert xv.xv_device_check() == 0


def test_other_branches_and_garbage_change_nothing(xv):
    """NaN and infinities in the cache past ctx, and in the K and V of nodes off a row's path, leave
    the row's bits; rows whose path holds one give what a decode row gives."""
    hd, Hq, Hkv, N, ctx = 64, 4, 2, 24, 37
    rng = np.random.default_rng(2)
    par = tree("mixed", N, rng)
    proj, (kc, vc) = rows(6, 1, N, Hq, Hkv, hd, "nan"), cache(6, 1, Hkv, 80, hd, "nan")
    clean = run(xv, dev(proj), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd)
    kc[:, :, ctx:], vc[:, :, ctx:] = 0x7FC0, 0x7F80
    assert same_bits(clean, run(xv, dev(proj), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd))
    bad = proj.reshape(N, 2 * Hq + 2 * Hkv, hd).copy()
    spoiled = [9, 17, 23]
    bad[9, 2 * Hq + Hkv, 5], bad[17, 2 * Hq + Hkv + 1, 63], bad[23, 2 * Hq, 0] = 0x7F80, 0x7FC0, 0xFF80
    bad = bad.reshape(N, -1)
    got = run(xv, dev(bad), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd)
    for i in range(N):
        if not set(chain_of(par, i)) & set(spoiled):
            assert same_bits(got[i], clean[i]), i
        else:
            want = f64(host_u16(decode_bits(xv, bad, kc, vc, ctx, par, 0, N, i, Hq, Hkv, hd, False)))
            have = f64(host_u16(got[i]))
            assert np.array_equal(np.isnan(have), np.isnan(want)) and np.array_equal(have[~np.isnan(want)], want[~np.isnan(want)]), i
    vc[:, :, 33, 7] = 0xFF80      # visible to every row, in the group the tree starts in
    got = run(xv, dev(proj), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd)
    for i in range(N):
        want = f64(host_u16(decode_bits(xv, proj, kc, vc, ctx, par, 0, N, i, Hq, Hkv, hd, False)))
        have = f64(host_u16(got[i]))
        assert np.isneginf(have.reshape(Hq, hd)[:, 7]).all()
        assert np.array_equal(have, want), i


@pytest.mark.parametrize("hd,ctx", [(64, 37), (128, 37), (256, 37), (128, 1000), (256, 4133)])
def test_non_finite_values_reach_their_columns_only(xv, hd, ctx):
    """Infinities and NaN in V, of nodes and of a cache position in the tree's first group of 16: in
    the rows that see them their column, every other value with the bits of the clean run."""
    Hq, Hkv, N, g0 = 4, 2, 40, ctx & ~15
    par = tree("mixed", N, np.random.default_rng(4))
    proj, (kc, vc) = rows(9, 1, N, Hq, Hkv, hd, f"nf{hd}"), cache(9, 1, Hkv, ctx + 5, hd, f"nf{ctx}.{hd}")
    clean = host_u16(run(xv, dev(proj), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd)).reshape(N, Hq, hd)
    heads = proj.reshape(N, 2 * Hq + 2 * Hkv, hd)
    heads[9, 2 * Hq + Hkv, 5], heads[17, 2 * Hq + Hkv + 1, hd - 1], vc[0, 1, g0 + 1, 7] = 0x7F80, 0x7FC0, 0xFF80
    got = host_u16(run(xv, dev(proj), dev(kc), dev(vc), [ctx], parents([par], N), None, N, Hq, Hkv, hd)).reshape(N, Hq, hd)
    for i in range(N):
        path = chain_of(par, i)
        want = f64(clean[i])
        if 9 in path:
            want[:2, 5] = np.inf
        if 17 in path:
            want[2:, hd - 1] = np.nan
        want[2:, 7] = -np.inf
        have = f64(got[i])
        assert np.array_equal(np.isnan(have), np.isnan(want)) and np.array_equal(have[~np.isnan(want)], want[~np.isnan(want)]), i
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,N,page,ctx,kind", [(256, 24, 4, 16, 64, [2183, 640, 64], "mixed"), (64, 6, 2, 64, 128, [500, 1], "wide"),
                                                       (128, 8, 8, 9, 192, [191, 192, 193, 4100], "pairs")])
def test_paged_equals_contiguous(xv, hd, Hq, Hkv, N, page, ctx, kind):
    B, rng = len(ctx), np.random.default_rng(page)
    trees = [tree(kind, N, rng) for _ in ctx]
    Lmax = -(-max(ctx) // page) * page
    mp = Lmax // page
    proj, (kc, vc) = rows(7, B, N, Hq, Hkv, hd, f"p{hd}"), cache(7, B, Hkv, Lmax, hd, f"p{hd}")
    n_pages = B * mp + 3
    table = rng.permutation(n_pages)[: B * mp].reshape(B, mp).astype(np.int32)
    pools = []
    for c in (kc, vc):
        pool = np.zeros((n_pages, Hkv, page, hd), np.uint16)
        for b in range(B):
            for j in range(mp):
                pool[table[b, j]] = c[b, :, j * page:(j + 1) * page]
        pools.append(dev(pool))
    X, par = dev(proj), parents(trees, N)
    want = run(xv, X, dev(kc), dev(vc), ctx, par, None, N, Hq, Hkv, hd)
    tab, out = dev(table), torch.empty_like(want)
    xv.xv_attn_tree_paged(X, pools[0], pools[1], xv.kv_pages(tab, page, n_pages), i32(ctx), X[:, 2 * Hq * hd:], par, None, N, B, Hq,
                          Hkv, hd, max(ctx), hd ** -0.5, out, xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, max(ctx))))
    assert same_bits(out, want) and xv.xv_device_check() == 0


def test_batched_and_persistent_equal_alone(xv):
    """Mixed lengths and node counts in one call, enough items for persistent CTAs that cross
    sequences and reload Q between row tiles: every sequence's rows equal its own call's."""
    hd, Hq, Hkv, N = 256, 24, 4, 64
    ctx = [20000, 9001, 1, 513, 2183, 0, 64, 4096]
    rng = np.random.default_rng(5)
    counts = [64, 40, 64, 1, 64, 22, 0, 63]
    trees = [tree(["mixed", "wide", "pairs", "chain"][b % 4], n, rng) if n else [] for b, n in enumerate(counts)]
    B, Lmax = len(ctx), 20000
    proj, (kc, vc) = rows(8, B, N, Hq, Hkv, hd, "batch"), cache(8, B, Hkv, Lmax, hd, "batch")
    X, K, V = dev(proj), dev(kc), dev(vc)
    out = run(xv, X, K, V, ctx, parents(trees, N), i32(counts), N, Hq, Hkv, hd, gate=True, fill=3)
    for b in range(B):
        if not counts[b]:
            continue
        one = run(xv, X[b * N:(b + 1) * N].contiguous(), K[b:b + 1], V[b:b + 1], [ctx[b]], parents([trees[b]], N), i32([counts[b]]),
                  N, Hq, Hkv, hd, gate=True, fill=3)
        assert same_bits(out[b * N:(b + 1) * N], one), f"sequence {b}"
    check(out, proj, kc, vc, ctx, trees, N, Hq, Hkv, hd, True, "batch", nodes=(0, 13, 39, 62))
    for _ in range(20):
        assert same_bits(out, run(xv, X, K, V, ctx, parents(trees, N), i32(counts), N, Hq, Hkv, hd, gate=True, fill=3))
    assert xv.xv_device_check() == 0


def walk(par, tokens, argmax):
    kept = [0]
    while True:
        nxt = [i for i in range(len(par)) if par[i] == kept[-1] and tokens[i] == argmax[kept[-1]]]
        if not nxt:
            return kept
        kept.append(nxt[0])


@pytest.mark.parametrize("kind", ["chain", "star", "mixed", "wide", "pairs", "forest"])
def test_accept_walks_to_the_lowest_matching_child(xv, kind):
    """Every draft follows its parent's argmax with probability 0.8, from a vocabulary of 2 so that
    siblings often carry the same token."""
    rng = np.random.default_rng(11)
    B, N = 37, 64
    counts = [64, 1, 0, 33, 32, 31] + [int(rng.integers(0, 65)) for _ in range(B - 6)]
    trees = [tree(kind, n, rng) if n else [] for n in counts]
    am = rng.integers(0, 2, (B, N))
    tok = rng.integers(0, 2, (B, N))
    for b, t in enumerate(trees):
        for i in range(1, len(t)):
            if t[i] >= 0 and rng.random() < 0.8:
                tok[b, i] = am[b, t[i]]
    path, keep, nxt = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,)))
    xv.xv_tree_accept(i32(tok), parents(trees, N), i32(counts), i32(am), path, keep, nxt)
    longest = 0
    for b, t in enumerate(trees):
        want = walk(t, tok[b], am[b]) if t else []
        longest = max(longest, len(want))
        assert path[b].tolist() == want + [-1] * (N - len(want))
        assert keep[b].item() == len(want)
        assert nxt[b].item() == (am[b, want[-1]] if want else -1)
    assert longest > 1
    assert xv.xv_device_check() == 0


@pytest.mark.parametrize("paged", [False, True])
def test_append_path_places_the_kept_rows(xv, paged):
    B, N, Hkv, hd, page = 3, 16, 2, 64, 64
    ctx, keep = [60, 0, 130], [9, 1, 0]
    kv = synth.normal_bf16(2, synth.tid("path.kv"), (B * N, 2 * Hkv * hd + 16))
    path = np.full((B, N), -1, np.int32)
    path[0, :9], path[1, 0] = [0, 2, 3, 5, 6, 9, 11, 12, 15], 0
    Lmax = 192
    table = np.array([[5, 2, 7], [0, 6, 3], [1, 4, 8]], np.int32)
    shape = (9, Hkv, page, hd) if paged else (B, Hkv, Lmax, hd)
    kc = torch.full(shape, 5, dtype=torch.int16, device="cuda")
    vc = torch.full(shape, 6, dtype=torch.int16, device="cuda")
    src = dev(kv)[:, : 2 * Hkv * hd]
    if paged:
        tab = dev(table)
        xv.xv_kv_append_path_paged(src, dev(path), i32(keep), i32(ctx), N, B, Hkv, hd, xv.kv_pages(tab, page, 9), kc, vc)
    else:
        xv.xv_kv_append_path(src, dev(path), i32(keep), i32(ctx), N, B, Hkv, hd, Lmax, kc, vc)
    wk, wv = np.full(shape, 5, np.uint16), np.full(shape, 6, np.uint16)
    for b in range(B):
        for t in range(keep[b]):
            p, r = ctx[b] + t, kv[b * N + path[b, t]]
            a, o = (table[b, p // page], p % page) if paged else (b, p)
            wk[a, :, o], wv[a, :, o] = r[: Hkv * hd].reshape(Hkv, hd), r[Hkv * hd: 2 * Hkv * hd].reshape(Hkv, hd)
    assert np.array_equal(host_u16(kc), wk) and np.array_equal(host_u16(vc), wv)
    assert xv.xv_device_check() == 0


def bits(xv):
    import ctypes
    code = ctypes.c_uint(0)
    xv.lib().xv_device_check(None, ctypes.byref(code))
    return code.value


def test_bad_trees_counts_and_lengths_are_recorded(xv):
    """Nothing out of range is followed: a bad parent is read as none, a bad count clamped, a bad
    length's sequence skipped, a bad page read as page 0 or skipped."""
    N, Hq, Hkv, hd, B = 4, 2, 1, 64, 2
    proj, (kc, vc) = rows(3, B, N, Hq, Hkv, hd, "bad"), cache(3, B, Hkv, 64, hd, "bad")
    X, K, V = dev(proj), dev(kc), dev(vc)
    good, bad = i32([[-1, 0, 1, 2]] * 2), i32([[-1, 0, 2, 9], [-1, 0, 1, -5]])
    seen = run(xv, X, K, V, [8, 9], bad, None, N, Hq, Hkv, hd)
    assert bits(xv) == 32
    assert same_bits(seen, run(xv, X, K, V, [8, 9], i32([[-1, 0, -1, -1], [-1, 0, 1, -1]]), None, N, Hq, Hkv, hd))
    out = run(xv, X, K, V, [8, 9], good, i32([-1, 9]), N, Hq, Hkv, hd, fill=7)
    assert bits(xv) == 8
    assert (out[:N] == 7).all()
    assert same_bits(out[N:], run(xv, X, K, V, [8, 9], good, None, N, Hq, Hkv, hd)[N:])
    out = run(xv, X, K, V, [-1, 41], good, None, N, Hq, Hkv, hd, max_ctx=40, fill=7)
    assert bits(xv) == 4 and (out == 7).all()
    pos = torch.full((2, N), -9, dtype=torch.int32, device="cuda")
    xv.xv_tree_positions(bad, None, i32([5, 5]), pos)
    assert bits(xv) == 32 and pos.tolist() == [[5, 6, 5, 5], [5, 6, 7, 5]]
    path, keep, nxt = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, N), 2, 2))
    xv.xv_tree_accept(i32([[0, 1, 1, 1]] * 2), bad, i32([5, 3]), i32([[1, 1, 1, 1]] * 2), path, keep, nxt)
    assert bits(xv) == 32 | 8 and keep.tolist() == [2, 3]
    before = K.clone()
    xv.xv_kv_append_path(X[:, 2 * Hq * hd:], i32([[0, 4, -1, 1]] * 2), i32([3, 5]), i32([0, 62]), N, B, Hkv, hd, 64, K, V)
    assert bits(xv) == 8 | 4
    k = host_u16(K)
    assert np.array_equal(k[0, 0, 0], proj[0, 2 * Hq * hd: (2 * Hq + 1) * hd]) and same_bits(K[0, :, 1:], before[0, :, 1:])
    assert np.array_equal(k[1, 0, 62], proj[N, 2 * Hq * hd: (2 * Hq + 1) * hd]) and same_bits(K[1, :, 63:], before[1, :, 63:])
    table = i32([[3], [0]])
    pool_k, pool_v = dev(kc), dev(vc)
    out = torch.zeros((B * N, Hq * hd), dtype=torch.int16, device="cuda")
    xv.xv_attn_tree_paged(X, pool_k, pool_v, xv.kv_pages(table, 64, 2), i32([8, 8]), X[:, 2 * Hq * hd:], good, None, N, B, Hq, Hkv,
                          hd, 8, 0.125, out, xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, 8)))
    assert bits(xv) == 16 and torch.isfinite(out.view(torch.bfloat16).float()).all()
    xv.xv_kv_append_path_paged(X[:, 2 * Hq * hd:], i32([[0] * N] * 2), i32([1, 0]), i32([8, 8]), N, B, Hkv, hd,
                               xv.kv_pages(table, 64, 2), pool_k, pool_v)
    assert bits(xv) == 16 and same_bits(pool_k, dev(kc))
