"""Head norms with the rotation against the formula in 64 bits.

Tolerance, before any run: y is a value a cos - b sin of normed a, b.  Up to the final rounding the
kernel works in fp32: the sum of hd squares (8 products per lane and a 5-step tree) is off by at most
13 roundings, half of that after the root; root, reciprocal, mean, eps, the two products of the norm
and 1 + w add 7; the rotation's products and sum 2; cos and sin are within 2^-24 * 4 of 1 (the
angle's conversion 2^-25 of a half turn, the functions' own 2 units).  So |err| <= e with
e = 20 * 2^-24 * (|a| + |b|), and the final rounding is at most half a step: 2^-8 of the value."""
import math

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


def reference(x, w, pos, rot, base, inter):
    """x [M, H, hd] -> (y, |a| + |b|) in 64 bits."""
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + 1e-6) * (1 + w) if w is not None else x.copy()
    mag = np.abs(y)
    if rot:
        ang = np.asarray(pos, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        i = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
        j = i + 1 if inter else i + rot // 2
        a, b = y[..., i].copy(), y[..., j].copy()
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        mag[..., i] = mag[..., j] = np.abs(a) + np.abs(b)
    return y, mag


def close(got, ref, mag, what):
    e = 20 * 2.0 ** -24 * mag
    tol = 2.0 ** -8 * (np.abs(ref) + e) + e
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values off, worst {np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)):.2f} of the bound"


def inputs(seed, M, Hq, Hkv, hd, sigma=1.0):
    proj = synth.normal_bf16(seed, synth.tid(f"rope{M}.{Hq}.{hd}"), (M, (2 * Hq + 2 * Hkv) * hd), sigma)
    qn, kn = (synth.normal_bf16(seed, synth.tid(n), (hd,), 0.3) for n in ("rope.qn", "rope.kn"))
    return proj, qn, kn


@pytest.mark.parametrize("hd,Hq,Hkv,M,rot,inter,base", [
    (256, 24, 4, 8, 64, False, 1e7), (256, 24, 4, 3, 256, True, 1e4), (128, 32, 8, 1, 128, False, 1e6),
    (128, 5, 1, 70, 16, True, 1e4), (64, 2, 1, 9, 64, False, 1e4), (64, 7, 7, 1100, 48, True, 1e5),
    (256, 3, 3, 1030, 32, False, 1e7), (64, 1, 1, 1, 0, False, 1e4), (128, 40, 2, 4, 96, False, 1e4),
    # several rows to a CTA
    (64, 7, 7, 5001, 48, True, 1e5), (128, 12, 4, 4870, 128, False, 1e6), (64, 1, 1, 20011, 16, False, 1e4)])
def test_rows_against_the_formula(xv, hd, Hq, Hkv, M, rot, inter, base):
    """Positions from 0 through 500000, negative ones among them."""
    proj, qn, kn = inputs(1, M, Hq, Hkv, hd)
    pos = np.random.default_rng(M).integers(-5, 500001, M).astype(np.int32)
    pos[: 3] = [131071, 0, -5][: min(M, 3)]
    X = dev(proj)
    q, kv = X[:, : Hq * hd], X[:, 2 * Hq * hd:]
    qo = torch.empty((M, Hq * hd), dtype=torch.int16, device="cuda")
    ko = torch.empty((M, Hkv * hd + 8), dtype=torch.int16, device="cuda")[:, : Hkv * hd]
    xv.xv_qk_norm_rope(q, kv, dev(pos), Hq, Hkv, hd, qo, ko, q_norm=dev(qn), k_norm=dev(kn),
                       freqs=xv.rope_freqs(rot, base) if rot else None, interleaved=inter)
    heads = f64(proj).reshape(M, -1, hd)
    for got, x, w, what in ((qo, heads[:, :Hq], qn, "q"), (ko, heads[:, 2 * Hq: 2 * Hq + Hkv], kn, "k")):
        ref, mag = reference(x, f64(w), pos, rot, base, inter)
        close(f64(host_u16(got)).reshape(ref.shape), ref, mag, what)
    # in place: the same bits, and the gate and v columns as they were
    Y = X.clone()
    xv.xv_qk_norm_rope(Y[:, : Hq * hd], Y[:, 2 * Hq * hd:], dev(pos), Hq, Hkv, hd, Y[:, : Hq * hd], Y[:, 2 * Hq * hd:],
                       q_norm=dev(qn), k_norm=dev(kn), freqs=xv.rope_freqs(rot, base) if rot else None, interleaved=inter)
    assert same_bits(Y[:, : Hq * hd].contiguous(), qo)
    assert same_bits(Y[:, 2 * Hq * hd: (2 * Hq + Hkv) * hd].contiguous(), ko.contiguous())
    assert same_bits(Y[:, Hq * hd: 2 * Hq * hd].contiguous(), X[:, Hq * hd: 2 * Hq * hd].contiguous())
    assert same_bits(Y[:, (2 * Hq + Hkv) * hd:].contiguous(), X[:, (2 * Hq + Hkv) * hd:].contiguous())
    assert xv.xv_device_check() == 0


def test_without_norm_weights_the_head_is_only_rotated(xv):
    hd, Hq, Hkv, M, rot = 128, 4, 2, 5, 64
    proj, _, _ = inputs(2, M, Hq, Hkv, hd, 30.0)
    pos = np.arange(M, dtype=np.int32) * 1000
    X = dev(proj)
    qo, ko = (torch.empty((M, h * hd), dtype=torch.int16, device="cuda") for h in (Hq, Hkv))
    xv.xv_qk_norm_rope(X[:, : Hq * hd], X[:, 2 * Hq * hd:], dev(pos), Hq, Hkv, hd, qo, ko, freqs=xv.rope_freqs(rot))
    heads = f64(proj).reshape(M, -1, hd)
    for got, x in ((qo, heads[:, :Hq]), (ko, heads[:, 2 * Hq: 2 * Hq + Hkv])):
        ref, mag = reference(x, None, pos, rot, 1e4, False)
        close(f64(host_u16(got)).reshape(ref.shape), ref, mag, "rotation alone")


def test_zero_heads_and_non_finite_values_stay_in_their_head(xv):
    """A zero head normalises to zeros; a NaN or an infinity spoils its own head only."""
    hd, Hq, Hkv, M = 64, 6, 2, 4
    proj, qn, kn = inputs(3, M, Hq, Hkv, hd)
    clean = dev(proj)
    dirty = proj.copy()
    dirty[0, : hd] = 0
    dirty[1, hd + 5] = 0x7FC0
    dirty[2, 3 * hd + 63] = 0x7F80
    pos, f = dev(np.arange(M, dtype=np.int32)), xv.rope_freqs(64)
    outs = []
    for X in (clean, dev(dirty)):
        qo, ko = (torch.empty((M, h * hd), dtype=torch.int16, device="cuda") for h in (Hq, Hkv))
        xv.xv_qk_norm_rope(X[:, : Hq * hd], X[:, 2 * Hq * hd:], pos, Hq, Hkv, hd, qo, ko, q_norm=dev(qn), k_norm=dev(kn), freqs=f)
        outs.append((host_u16(qo).reshape(M, Hq, hd), host_u16(ko)))
    a, b = outs[0][0].copy(), outs[1][0]
    assert not (b[0, 0] & 0x7FFF).any()
    assert np.isnan(f64(b[1, 1])).any() and not np.isfinite(f64(b[2, 3])).all()
    for r, h in ((0, 0), (1, 1), (2, 3)):
        a[r, h] = b[r, h]
    assert np.array_equal(a, b) and np.array_equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("hd,Hq,Hkv,M,page,inter", [(256, 24, 4, 9, 64, False), (128, 8, 2, 1500, 128, True), (64, 3, 1, 33, 192, False),
                                                       (128, 32, 8, 4870, 128, True)])
def test_append_writes_the_rows_bits_to_their_slots(xv, hd, Hq, Hkv, M, page, inter):
    """K as xv_qk_norm_rope gives it and V as it is, at the slots and nowhere else; a row with slot -1
    and rows from *n_rows on write no K or V (the latter no q either)."""
    proj, qn, kn = inputs(4, M, Hq, Hkv, hd)
    n_pages = (M + page - 1) // page + 4
    rng = np.random.default_rng(7)
    slots = rng.permutation(n_pages * page)[:M].astype(np.int64)
    slots[1] = -1
    live = M - 2
    X, pos, f = dev(proj), dev(rng.integers(0, 200000, M).astype(np.int32)), xv.rope_freqs(64 if hd > 64 else 32)
    kw = dict(q_norm=dev(qn), k_norm=dev(kn), freqs=f, interleaved=inter)
    q, kv = X[:, : Hq * hd], X[:, 2 * Hq * hd:]
    qo, ko = (torch.zeros((M, h * hd), dtype=torch.int16, device="cuda") for h in (Hq, Hkv))
    xv.xv_qk_norm_rope(q, kv, pos, Hq, Hkv, hd, qo, ko, **kw)
    qa = torch.full_like(qo, 77)
    kp = torch.full((n_pages, Hkv, page, hd), 99, dtype=torch.int16, device="cuda")
    vp = torch.full_like(kp, 98)
    xv.xv_qk_norm_rope_append(q, kv, pos, dev(slots), Hq, Hkv, hd, qa, kp, vp, page, n_pages, n_rows=dev(np.array([live], np.int32)), **kw)
    assert same_bits(qa[:live], qo[:live]) and (qa[live:] == 77).all()
    want_k, want_v = np.full((n_pages, Hkv, page, hd), 99, np.uint16), np.full((n_pages, Hkv, page, hd), 98, np.uint16)
    K, V = host_u16(ko).reshape(M, Hkv, hd), proj[:, (2 * Hq + Hkv) * hd:].reshape(M, Hkv, hd)
    for r in range(live):
        if slots[r] >= 0:
            want_k[slots[r] // page, :, slots[r] % page], want_v[slots[r] // page, :, slots[r] % page] = K[r], V[r]
    assert np.array_equal(host_u16(kp), want_k) and np.array_equal(host_u16(vp), want_v)
    assert xv.xv_device_check() == 0


def test_a_slot_outside_the_pool_is_recorded_and_skipped(xv):
    hd, Hq, Hkv, M, page = 64, 2, 1, 3, 64
    proj, qn, kn = inputs(5, M, Hq, Hkv, hd)
    X = dev(proj)
    kp = torch.zeros((2, Hkv, page, hd), dtype=torch.int16, device="cuda")
    vp, qo = torch.zeros_like(kp), torch.zeros((M, Hq * hd), dtype=torch.int16, device="cuda")
    xv.xv_qk_norm_rope_append(X[:, : Hq * hd], X[:, 2 * Hq * hd:], dev(np.arange(M, dtype=np.int32)),
                              dev(np.array([128, -2, 5], np.int64)), Hq, Hkv, hd, qo, kp, vp, page, 2, freqs=xv.rope_freqs(64))
    with pytest.raises(xv.XVError, match="0x10"):
        xv.xv_device_check()
    assert int((host_u16(vp).reshape(2, page, hd) != 0).any(-1).sum()) == 1 and (qo != 0).any(-1).all()


def test_far_positions_turn_by_the_exact_angle(xv):
    """At 2^30 - 1 positions the angle is still right: an fp32 product would be off by whole turns."""
    hd, rot, base = 64, 64, 1e4
    proj, _, _ = inputs(6, 2, 1, 1, hd)
    pos = np.array([2 ** 30 - 1, 2 ** 24 + 1], dtype=np.int32)
    X = dev(proj)
    qo, ko = (torch.empty((2, hd), dtype=torch.int16, device="cuda") for _ in range(2))
    xv.xv_qk_norm_rope(X[:, :hd], X[:, 2 * hd:], dev(pos), 1, 1, hd, qo, ko, freqs=xv.rope_freqs(rot, base))
    x = f64(proj).reshape(2, -1, hd)[:, :1]
    y = np.empty_like(x)
    freqs = [v % 2 ** 64 for v in xv.rope_freqs(rot, base, device="cpu").tolist()]
    for r in range(2):
        for i in range(rot // 2):
            a = 2 * math.pi * (((int(pos[r]) * freqs[i]) % 2 ** 64) / 2.0 ** 64)     # whole turns dropped in integers
            y[r, 0, i] = x[r, 0, i] * math.cos(a) - x[r, 0, i + 32] * math.sin(a)
            y[r, 0, i + 32] = x[r, 0, i + 32] * math.cos(a) + x[r, 0, i] * math.sin(a)
    mag = np.concatenate([np.abs(x[..., :32]) + np.abs(x[..., 32:])] * 2, -1)
    close(f64(host_u16(qo)).reshape(2, 1, hd), y, mag, "far positions")
