"""Pins of the key/value cache oracle: the rotation against complex multiplication, the
cache's byte places as a bijection, attention against torch's float64 softmax and closed
forms, and the error bound against an fp32 emulation.  CPU only."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import nvfp4 as O


def test_rotation_is_complex_multiplication():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64)).astype(np.float32)
    ang = rng.uniform(0, 6, (5, 16))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    z = (cos.astype(np.float64) + 1j * sin)[:, None]
    y = KV.rotate_f32(x, cos, sin, True)
    w = (x[..., 0:32:2] + 1j * x[..., 1:32:2].astype(np.float64)) * z
    assert np.allclose(y[..., 0:32:2] + 1j * y[..., 1:32:2], w, atol=1e-6) and np.array_equal(y[..., 32:], x[..., 32:])
    y = KV.rotate_f32(x, cos, sin, False)
    w = (x[..., :16] + 1j * x[..., 16:32].astype(np.float64)) * z
    assert np.allclose(y[..., :16] + 1j * y[..., 16:32], w, atol=1e-6) and np.array_equal(y[..., 32:], x[..., 32:])


@pytest.mark.parametrize("D,page,H", [(64, 16, 2), (128, 32, 3), (256, 64, 1)])
def test_every_byte_of_a_page_has_one_owner(D, page, H):
    size = H * page * D * 9 // 8
    seen = np.zeros(2 * size, dtype=int)
    for slot in range(2 * page):
        for h in range(H):
            for at in KV.byte_places(slot, h, H, page, D):
                seen[at] += 1
    assert np.all(seen == 1)


def test_append_and_gather_round_trip():
    rng = np.random.default_rng(1)
    T, H, D, page = 21, 2, 64, 16
    k, v = rng.standard_normal((2, T, H, D)).astype(np.float32)
    kg, vg = np.float32([0.002, 0.003]), np.float32([0.0015, 0.001])
    cache = np.full(3 * H * page * D * 9 // 8, 0xAB, dtype=np.uint8)
    slots = rng.permutation(3 * page)[:T].astype(np.int64)
    slots[[2, 5]] = [-1, 3 * page]
    KV.append(cache, k, v, slots, kg, vg, page)
    gk, gv = KV.gather(cache, slots, H, D, kg, vg, page)
    for x, y, g in ((k, gk, kg), (v, gv, vg)):
        c, s = KV.quantize_heads(x, g)
        want = O.dequantize_rows(c.reshape(T * H, -1), s.reshape(T * H, -1), np.tile(g, T)).reshape(T, H, D)
        want[[2, 5]] = 0
        assert np.array_equal(y, want)
        live = np.delete(np.arange(T), [2, 5])
        assert np.linalg.norm((x - y)[live]) < 0.12 * np.linalg.norm(x[live])


@pytest.mark.parametrize("m,n,window", [(1, 9, 0), (7, 7, 0), (5, 30, 4), (6, 3, 0), (1, 0, 0), (3, 12, 100)])
def test_attention_matches_masked_softmax(m, n, window):
    rng = np.random.default_rng(m * 31 + n)
    q, k, v = rng.standard_normal((m, 6, 16)), rng.standard_normal((n, 2, 16)), rng.standard_normal((n, 2, 16))
    o, lse, w = KV.attention(q, k, v, 0.25, window)
    t = torch.from_numpy
    s = 0.25 * torch.einsum("mhd,nhd->mhn", t(q), t(np.repeat(k, 3, 1)))
    pos = n - m + torch.arange(m)[:, None]
    j = torch.arange(n)[None]
    ok = (j <= pos) & ((j > pos - window) if window else True)
    s = s.masked_fill(~ok[:, None], -float("inf"))
    p = torch.softmax(s, -1).nan_to_num(0)
    assert np.allclose(w, p.numpy(), atol=1e-14)
    assert np.allclose(o, torch.einsum("mhn,nhd->mhd", p, t(np.repeat(v, 3, 1))).numpy(), atol=1e-13)
    empty = ~ok.any(-1).numpy() if n else np.ones(m, bool)
    assert np.all(np.isneginf(lse[empty])) and np.all(o[empty] == 0)
    if n:
        assert np.allclose(lse[~empty], torch.logsumexp(s, -1).numpy()[~empty], atol=1e-13)


def test_equal_scores_average_the_values():
    v = np.random.default_rng(3).standard_normal((8, 1, 4))
    o, lse, _ = KV.attention(np.zeros((1, 1, 4)), np.ones((8, 1, 4)), v, 0.5)
    assert np.allclose(o[0, 0], v[:, 0].mean(0)) and np.isclose(lse[0, 0], np.log(8))


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_bound_admits_a_narrow_emulation_and_rejects_a_planted_error(out_dtype):
    rng = np.random.default_rng(4)
    m, n, H, D = 3, 200, 2, 64
    q = rng.standard_normal((m, H, D)).astype(np.float32)
    k, v = rng.standard_normal((2, n, H, D))
    o, lse, w = KV.attention(q, k, v, 0.125)
    bo, bl = KV.attention_bounds(q, k, v, w, 0.125, out_dtype)
    s = np.einsum("mhd,nhd->mhn", q, k.astype(np.float32)).astype(np.float32) * np.float32(0.125)
    s = np.where(w > 0, s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True)).astype(np.float32)
    p2 = p.astype(np.float16).astype(np.float64) if out_dtype == "bf16" else p.astype(np.float64)
    got = np.einsum("mhn,nhd->mhd", p2, v) / p.sum(-1, dtype=np.float64)[..., None]
    assert np.all(np.abs(got - o) <= bo)
    assert not np.all(np.abs(got * 1.01 - o) <= bo)
    assert np.all(np.abs(s.max(-1) + np.log(p.sum(-1, dtype=np.float64)) - lse) <= bl)
    w2 = w.copy()
    w2[..., 0] = 0                                        # a token left out
    assert not np.all(np.abs(np.einsum("mhn,nhd->mhd", w2, v) - o) <= bo)
