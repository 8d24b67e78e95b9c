"""Pins of the attention oracle: closed forms, a brute-force softmax, and the
page operations' invariants."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import nvfp4

F32 = np.float32


def test_tree_sum_adds_neighbours_first():
    # 2^24 + 1 rounds to 2^24 in fp32: the order of the sum is visible
    x = np.array([2.0 ** 24, 1.0, 1.0, 1.0], F32)
    assert oa.tree_sum(x) == F32(2.0 ** 24) + F32(2.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation_closed_forms(interleaved):
    D, rot = 64, 32
    x = np.full((1, 1, D), 3.0, F32)
    one = np.ones(D, F32)
    # position 0: no rotation; a constant vector normalises to ones
    y = oa.norm_rope(x, one, 0.0, np.ones((1, rot // 2), F32), np.zeros((1, rot // 2), F32), interleaved)
    np.testing.assert_allclose(y, 1.0, rtol=1e-6)
    # a quarter turn: (a, b) -> (-b, a)
    z = np.arange(D, dtype=F32).reshape(1, 1, D)
    y = oa.norm_rope(z, None, 0.0, np.zeros((1, rot // 2), F32), np.ones((1, rot // 2), F32), interleaved)
    a, b = oa.rope_pairs(D, rot, interleaved)
    assert (y[..., a] == -z[..., b]).all() and (y[..., b] == z[..., a]).all() and (y[..., rot:] == z[..., rot:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_norm_is_near_fp64(interleaved):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 128)).astype(F32)
    w = (1 + 0.1 * rng.normal(size=128)).astype(F32)
    ang = rng.uniform(0, 6, size=(5, 64))
    c, s = np.cos(ang).astype(F32), np.sin(ang).astype(F32)
    got = oa.norm_rope(x, w, 1e-6, c, s, interleaved)
    # about a dozen roundings of 2^-24 on values of a few units
    np.testing.assert_allclose(got, oa.norm_rope_f64(x, w, 1e-6, c, s, interleaved), rtol=0, atol=16 * 2.0 ** -24 * 8)


def test_attention_against_brute_force():
    rng = np.random.default_rng(1)
    P, D, Hkv, G, n, N = 32, 64, 2, 3, 50, 4
    pool = np.zeros((N, Hkv, oa.record_bytes(P, D)), np.uint8)
    pages = [3, 1]
    k, v = (rng.normal(size=(n, Hkv, D)).astype(F32) for _ in range(2))
    gk, gv = np.full(Hkv, 0.002, F32), np.full(Hkv, 0.003, F32)
    for t in range(n):
        oa.write_token(pool, pages[t // P] * P + t % P, k[t], v[t], gk, gv, P)
    q = rng.normal(size=(4, Hkv * G, D))
    out, lse, *_ = oa.attention(q, pool, gk, gv, [0, 4], [n], [pages], 0.1, P, window=20)
    for h in range(Hkv * G):
        kd = np.stack([nvfp4.dequantize(*nvfp4.quantize(k[t, h // G][None], gk[h // G]))[0] for t in range(n)])
        vd = np.stack([nvfp4.dequantize(*nvfp4.quantize(v[t, h // G][None], gv[h // G]))[0] for t in range(n)])
        for i in range(4):
            p = n - 4 + i
            z = torch.tensor(q[i, h] @ kd.T * 0.1)
            z[torch.arange(n) > p] = -torch.inf
            z[torch.arange(n) <= p - 20] = -torch.inf
            np.testing.assert_allclose(out[i, h], (torch.softmax(z, 0).numpy()[None] @ vd)[0], atol=1e-12)
            assert abs(lse[i, h] - torch.logsumexp(z, 0).item()) < 1e-12


def test_attention_without_keys_is_zero():
    pool = np.zeros((1, 1, oa.record_bytes(32, 64)), np.uint8)
    out, lse, *_ = oa.attention(np.ones((2, 1, 64)), pool, [1.0], [1.0], [0, 2], [1], [[0]], 1.0, 32)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and np.isfinite(lse[1, 0])


def _counts(s):
    refs = [0] * len(s.refs)
    for r, n in zip(s.table, s.lens):
        for j in range(s.used(n)):
            refs[r[j]] += 1
    return refs


def test_pages_keep_their_counts():
    rng = np.random.default_rng(2)
    s = oa.Pages([[-1] * 6 for _ in range(8)], [0] * 8, [0] * 40, 32)
    for _ in range(200):
        op = rng.integers(4)
        if op == 0:
            s.extend([int(n) for n in rng.integers(0, 40, 8) * (rng.random(8) < 0.4)])
        elif op == 1:
            empty = [r for r in range(8) if s.lens[r] == 0][:2]
            full = [r for r in range(8) if s.lens[r] > 0]
            if full and empty:
                s.fork([int(rng.choice(full)) for _ in empty], empty)
        elif op == 2:
            s.free([int(rng.integers(8))])
        else:
            remap, moves = s.compact()
            live = sum(r > 0 for r in s.refs)
            assert all(r > 0 for r in s.refs[:live]) and not any(s.refs[live:])
        assert s.refs == _counts(s)
        # partial pages are never shared
        for r, n in zip(s.table, s.lens):
            assert n % 32 == 0 or s.refs[r[n // 32]] == 1
