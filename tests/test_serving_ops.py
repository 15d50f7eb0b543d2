"""Host side of the page-table, head-norm/rotation and draft-tree entry points: every refusal of a
bad argument happens before anything reaches the device (no GPU needed), the workspace sizes, and
the frequency table."""
import ctypes
import math
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def test_pages_update_refusals(xv):
    L = xv.lib()

    def call(table=P, page=64, max_pages=8, n_pages=100, free=P, n_free=P, B=4, slots=P, max_rows=32, ws=P, wsb=1 << 20):
        return L.xv_kv_pages_update(table, page, max_pages, n_pages, free, n_free, P, P, P, P, P, B, P, P, slots, max_rows,
                                    ws, wsb, None)

    assert call(table=None) == xv.XV_ERR_ARG
    assert call(free=None) == xv.XV_ERR_ARG
    assert call(n_free=None) == xv.XV_ERR_ARG
    assert call(slots=None) == xv.XV_ERR_ARG
    assert call(B=0) == xv.XV_ERR_ARG
    assert call(max_rows=0) == xv.XV_ERR_ARG
    assert call(max_pages=0) == xv.XV_ERR_ARG
    assert call(n_pages=0) == xv.XV_ERR_ARG
    assert call(page=96) == xv.XV_ERR_UNSUPPORTED
    assert call(page=0) == xv.XV_ERR_UNSUPPORTED
    assert call(B=65536) == xv.XV_ERR_UNSUPPORTED
    assert call(page=1 << 20, max_pages=1 << 12) == xv.XV_ERR_UNSUPPORTED
    assert call(ws=None) == xv.XV_ERR_WORKSPACE
    assert call(wsb=xv.xv_kv_pages_workspace_size(4) - 1) == xv.XV_ERR_WORKSPACE
    assert call(ws=ODD) == xv.XV_ERR_UNSUPPORTED
    assert xv.xv_kv_pages_workspace_size(0) == 0


def _rope(xv, q_norm=0x10000, freq=0x10000, rot=64):
    return xv.QkRope(q_norm, 0x10000, 1e-6, freq, rot, 0)


def test_qk_norm_rope_refusals(xv):
    L = xv.lib()

    def call(q=P, qs=1024, qo=P, k=P, ks=512, ko=P, rope=None, pos=P, M=2, Hq=4, Hkv=2, hd=256):
        r = rope or _rope(xv)
        return L.xv_qk_norm_rope(q, qs, qo, 1024, k, ks, ko, 512, ctypes.byref(r), pos, None, M, Hq, Hkv, hd, None)

    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None), dict(M=0), dict(Hq=0), dict(Hkv=0),
               dict(qs=1016), dict(ks=504), dict(rope=_rope(xv, rot=272)), dict(rope=_rope(xv, rot=-16)),
               dict(rope=_rope(xv, freq=None))):
        assert call(**kw) == xv.XV_ERR_ARG, kw
    for kw in (dict(hd=96), dict(hd=512), dict(rope=_rope(xv, rot=24)), dict(q=ODD), dict(k=ODD), dict(qs=1028),
               dict(rope=_rope(xv, q_norm=0x10004)), dict(Hq=65536, qs=1 << 40)):
        assert call(**kw) == xv.XV_ERR_UNSUPPORTED, kw
    assert L.xv_qk_norm_rope(P, 1024, P, 1024, P, 512, P, 512, None, P, None, 2, 4, 2, 256, None) == xv.XV_ERR_ARG


def test_qk_norm_rope_append_refusals(xv):
    L = xv.lib()

    def call(kvs=1024, slots=P, page=64, n_pages=4, kp=P):
        r = _rope(xv)
        return L.xv_qk_norm_rope_append(P, 1024, P, 1024, P, kvs, ctypes.byref(r), P, slots, None, 2, 4, 2, 256, page,
                                        n_pages, kp, P, None)

    assert call(kvs=1016) == xv.XV_ERR_ARG          # rows of k and v
    assert call(slots=None) == xv.XV_ERR_ARG
    assert call(kp=None) == xv.XV_ERR_ARG
    assert call(page=0) == xv.XV_ERR_ARG
    assert call(n_pages=0) == xv.XV_ERR_ARG
    assert call(kp=ODD) == xv.XV_ERR_UNSUPPORTED


def test_attn_tree_refusals(xv):
    L = xv.lib()

    def call(q=P, qs=1024, kc=P, src=P, ss=1024, parent=P, N=16, B=2, Hq=4, Hkv=2, hd=256, Lmax=512, max_ctx=500, gate=None,
             gs=0, os=1024, ws=P, wsb=1 << 40):
        return L.xv_attn_tree(q, qs, kc, P, P, src, ss, parent, None, N, B, Hq, Hkv, hd, Lmax, max_ctx, 0.0625, gate, gs, P,
                              os, ws, wsb, None)

    for kw in (dict(q=None), dict(kc=None), dict(src=None), dict(parent=None), dict(N=0), dict(B=0), dict(Hq=0), dict(Hkv=0),
               dict(Hq=5, qs=2048, os=2048), dict(max_ctx=513), dict(max_ctx=-1), dict(qs=1016), dict(ss=1016), dict(os=1016),
               dict(gate=P, gs=1000)):
        assert call(**kw) == xv.XV_ERR_ARG, kw
    for kw in (dict(N=xv.XV_KMAX + 1), dict(hd=96), dict(hd=512, qs=4096, os=4096, ss=4096), dict(q=ODD), dict(src=ODD),
               dict(kc=ODD), dict(qs=1028), dict(ws=ODD), dict(B=65536), dict(Hq=258, qs=1 << 20, os=1 << 20)):
        assert call(**kw) == xv.XV_ERR_UNSUPPORTED, kw
    assert call(ws=None) == xv.XV_ERR_WORKSPACE
    assert call(wsb=xv.xv_attn_tree_workspace_size(2, 16, 4, 256, 500) - 1) == xv.XV_ERR_WORKSPACE
    assert xv.xv_attn_tree_workspace_size(0, 16, 4, 256, 500) == 0
    assert xv.xv_attn_tree_workspace_size(2, 65, 4, 256, 500) == 0
    bad = xv.KvPages(0x10000, 96, 4, 8)
    assert L.xv_attn_tree_paged(P, 1024, P, P, ctypes.byref(bad), P, P, 1024, P, None, 16, 2, 4, 2, 256, 300, 0.0625, None, 0,
                                P, 1024, P, 1 << 40, None) == xv.XV_ERR_UNSUPPORTED
    good = xv.KvPages(0x10000, 64, 4, 8)
    assert L.xv_attn_tree_paged(P, 1024, P, P, ctypes.byref(good), P, P, 1024, P, None, 16, 2, 4, 2, 256, 257, 0.0625, None, 0,
                                P, 1024, P, 1 << 40, None) == xv.XV_ERR_ARG


def test_tree_walk_refusals(xv):
    L = xv.lib()
    pos = lambda parent=P, N=16, B=2, out=P: L.xv_tree_positions(parent, None, P, N, B, out, None)   # noqa: E731
    acc = lambda tok=P, N=16, B=2, path=P: L.xv_tree_accept(tok, P, None, P, N, B, path, P, P, None)   # noqa: E731
    app = lambda src=P, ss=1024, N=16, B=2, Hkv=2, hd=256, Lmax=64, kc=P: L.xv_kv_append_path(   # noqa: E731
        src, ss, P, P, P, N, B, Hkv, hd, Lmax, kc, P, None)
    assert pos(parent=None) == xv.XV_ERR_ARG and pos(out=None) == xv.XV_ERR_ARG and pos(N=0) == xv.XV_ERR_ARG
    assert pos(N=65) == xv.XV_ERR_UNSUPPORTED and pos(B=65536) == xv.XV_ERR_UNSUPPORTED
    assert acc(tok=None) == xv.XV_ERR_ARG and acc(path=None) == xv.XV_ERR_ARG and acc(B=0) == xv.XV_ERR_ARG
    assert acc(N=65) == xv.XV_ERR_UNSUPPORTED
    assert app(src=None) == xv.XV_ERR_ARG and app(ss=1016) == xv.XV_ERR_ARG and app(hd=12) == xv.XV_ERR_ARG
    assert app(Lmax=0) == xv.XV_ERR_ARG and app(N=65) == xv.XV_ERR_UNSUPPORTED
    assert app(src=ODD) == xv.XV_ERR_UNSUPPORTED and app(ss=1028) == xv.XV_ERR_UNSUPPORTED and app(kc=ODD) == xv.XV_ERR_UNSUPPORTED
    assert L.xv_kv_append_path_paged(P, 1024, P, P, P, 16, 2, 2, 256, ctypes.byref(xv.KvPages(0x10000, 96, 4, 8)), P, P,
                                     None) == xv.XV_ERR_UNSUPPORTED


@pytest.mark.parametrize("rot,base", [(64, 1e4), (128, 1e7), (16, 500000.0)])
def test_rope_freqs_are_turns_in_binary_fractions(xv, rot, base):
    """Each entry is within 2^-50 of its frequency's turns (a double's own error in it), so the angle
    at position 2^20 is exact to 2^-28 of a radian."""
    f = xv.rope_freqs(rot, base, device="cpu").tolist()
    assert len(f) == rot // 2
    for i, x in enumerate(f):
        turns = Fraction(x % 2 ** 64, 2 ** 64)
        want = base ** (-2 * i / rot) / (2 * math.pi)
        assert abs(float(turns) - want) <= want * 2.0 ** -50 + 2.0 ** -64
