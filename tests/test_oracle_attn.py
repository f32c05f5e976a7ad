"""Pins of the attention oracle (oracle/attn.py) to facts outside it: the
rotation against complex multiplication and relative positions, the norm's
size, the softmax against torch's in float64, the join of two halves by their
log sums, masks, pages in any order, and planted mistakes that each fail one of
these."""
import math

import numpy as np
import pytest
import torch

from oracle import attn as orc


def rot_tables(S, R):
    rate = 10000.0 ** (-np.arange(0, R, 2) / R)
    ang = np.arange(S)[:, None] * rate
    return np.cos(ang), np.sin(ang)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_complex_multiplication(inter):
    r = np.random.default_rng(1)
    x, R = r.standard_normal(64), 32
    cos, sin = rot_tables(50, R)
    got = orc.norm_rotate(x, cos=cos[37], sin=sin[37], interleaved=inter)
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    z = (x[a] + 1j * x[b]) * np.exp(1j * 37 * 10000.0 ** (-2 * i / R))
    np.testing.assert_allclose(got[a] + 1j * got[b], z, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(got[R:], x[R:])


@pytest.mark.parametrize("inter", [False, True])
def test_scores_depend_on_the_distance_only(inter):
    r = np.random.default_rng(2)
    q, k = r.standard_normal((2, 64))
    cos, sin = rot_tables(100, 64)
    turn = lambda x, p: orc.norm_rotate(x, cos=cos[p], sin=sin[p], interleaved=inter)
    assert math.isclose(turn(q, 20) @ turn(k, 13), turn(q, 97) @ turn(k, 90), rel_tol=1e-10)
    assert abs(turn(q, 20) @ turn(k, 13) - turn(q, 20) @ turn(k, 14)) > 1e-3


def test_norm_has_unit_mean_square_and_ignores_size():
    r = np.random.default_rng(3)
    x = r.standard_normal(128) * 7
    y = orc.norm_rotate(x, weight=np.ones(128), eps=0.0)
    assert math.isclose(np.mean(y * y), 1.0, rel_tol=1e-12)
    np.testing.assert_allclose(orc.norm_rotate(5 * x, weight=np.ones(128), eps=0.0), y, rtol=1e-12)


def paged(r, n, Hkv, D, ps):
    """Contiguous keys and values, and the same in shuffled pages."""
    K, V = r.standard_normal((2, n, Hkv, D))
    M = -(-n // ps)
    pages = r.permutation(M + 2)[:M]
    kp, vp = np.full((2, M + 2, Hkv, ps, D), np.nan)
    for j in range(n):
        kp[pages[j // ps], :, j % ps] = K[j]
        vp[pages[j // ps], :, j % ps] = V[j]
    return K, V, kp, vp, pages


@pytest.mark.parametrize("T,window", [(1, 0), (4, 0), (3, 5)])
def test_attention_equals_torch_softmax(T, window):
    r = np.random.default_rng(4)
    n, Hkv, G, D, ps = 23, 2, 3, 16, 5
    K, V, kp, vp, pages = paged(r, n, Hkv, D, ps)
    q = r.standard_normal((1, T, Hkv * G, D))
    out, lse, *_ = orc.paged_attention(q, kp, vp, pages[None], [n], window=window)
    for h in range(Hkv * G):
        s = torch.tensor(q[0, :, h] @ K[:, h // G].T / math.sqrt(D))
        e = torch.arange(n - T, n)[:, None]
        j = torch.arange(n)[None]
        s = s.masked_fill((j > e) | ((j <= e - window) if window else (j < 0)), -math.inf)
        np.testing.assert_allclose(out[0, :, h], (s.softmax(-1) @ torch.tensor(V[:, h // G])).numpy(), rtol=1e-12)
        np.testing.assert_allclose(lse[0, :, h], s.logsumexp(-1).numpy(), rtol=1e-12)


def test_halves_join_by_their_log_sums():
    r = np.random.default_rng(5)
    K, V, kp, vp, pages = paged(r, 24, 1, 16, 4)
    q = r.standard_normal((1, 1, 2, 16))
    whole, lse, *_ = orc.paged_attention(q, kp, vp, pages[None], [24])
    a, la, *_ = orc.paged_attention(q, kp, vp, pages[None, :3], [12])
    b, lb, *_ = orc.paged_attention(q, kp, vp, pages[None, 3:], [12])
    wa, wb = np.exp(la - lse)[..., None], np.exp(lb - lse)[..., None]
    np.testing.assert_allclose(a * wa + b * wb, whole, rtol=1e-12)


def test_rows_without_positions_and_missing_pages():
    r = np.random.default_rng(6)
    K, V, kp, vp, pages = paged(r, 8, 1, 16, 4)
    q = r.standard_normal((2, 3, 1, 16))
    table = np.stack([pages, pages])
    out, lse, *_ = orc.paged_attention(q, kp, vp, table, [0, 2])
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (out[1, 0] == 0).all() and np.isneginf(lse[1, 0]).all()      # e = -1
    np.testing.assert_allclose(out[1, 1, 0], V[0, 0], rtol=1e-12)       # sees itself only
    gone = np.array([[-1, pages[1]]])
    out2, *_ = orc.paged_attention(q[:1, :1], kp, vp, gone, [8])
    ref, *_ = orc.paged_attention(q[:1, :1], kp, vp, pages[None, 1:], [4])
    np.testing.assert_allclose(out2, ref, rtol=1e-12)


def test_append_then_read_returns_the_rows():
    r = np.random.default_rng(7)
    T, Hkv, D, ps = 9, 2, 16, 4
    q, (k, v) = r.standard_normal((T, 4, D)), r.standard_normal((2, T, Hkv, D))
    pages = np.array([3, 0, 2])
    slots = np.array([pages[i // ps] * ps + i % ps for i in range(T)])
    slots[4] = -1
    out, held = orc.kv_append(q, k, v, slots, 16)
    assert np.isnan(out[4]).all() and len(held) == T - 1
    np.testing.assert_array_equal(out[5], q[5])
    pool = np.zeros((4, Hkv, ps, D))
    for s, (kr, _) in held.items():
        pool[s // ps, :, s % ps] = kr
    got = orc.kv_read(pool, None, pages[None], [0, T], T + 1)
    ref = np.concatenate([k, np.zeros((1, Hkv, D))])
    ref[4] = 0
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("mistake", ["direction", "pairs", "mean", "future", "window", "group"])
def test_pins_reject_planted_mistakes(mistake):
    r = np.random.default_rng(8)
    if mistake in ("direction", "pairs"):
        x = r.standard_normal(32)
        cos, sin = rot_tables(9, 32)
        good = orc.norm_rotate(x, cos=cos[5], sin=sin[5])
        bad = orc.norm_rotate(x, cos=cos[5], sin=-sin[5]) if mistake == "direction" else \
            orc.norm_rotate(x, cos=cos[5], sin=sin[5], interleaved=True)
        i = np.arange(16)
        z = (x[i] + 1j * x[i + 16]) * np.exp(1j * 5 * 10000.0 ** (-2 * i / 32))
        assert np.allclose(good[i] + 1j * good[i + 16], z)
        assert not np.allclose(bad[i] + 1j * bad[i + 16], z)
        return
    if mistake == "mean":
        x = r.standard_normal(32)
        y = x / math.sqrt(float(np.sum(x * x)))          # the sum in place of the mean
        assert not math.isclose(np.mean(y * y), 1.0, rel_tol=1e-3)
        return
    K, V, kp, vp, pages = paged(r, 12, 2, 16, 4)
    q = r.standard_normal((1, 2, 4, 16))
    good, *_ = orc.paged_attention(q, kp, vp, pages[None], [12], window=4)
    if mistake == "future":       # every row sees every position
        bad, *_ = orc.paged_attention(q[:, 1:], kp, vp, pages[None], [12], window=5)
        bad = np.concatenate([orc.paged_attention(q[:, :1], kp, vp, pages[None], [12], window=4)[0], bad], 1)
    elif mistake == "window":
        bad, *_ = orc.paged_attention(q, kp, vp, pages[None], [12], window=5)
    else:                         # heads taken in turn instead of in runs
        bad, *_ = orc.paged_attention(q[:, :, [0, 2, 1, 3]], kp, vp, pages[None], [12], window=4)
        bad = bad[:, :, [0, 2, 1, 3]]
    assert np.abs(bad - good).max() > 1e-3
