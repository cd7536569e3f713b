"""Cache and attention at the edges of their ranges: bytes that were never written, scores
of any size, scales of either sign, bounds far above the lengths, many sequences, rows
beyond the caches.  Tolerances as in test_gpu_kv.py."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import nvfp4 as O
from tests.test_gpu_kv import Problem

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _held(x, g):
    """The values that the cache holds for x [n, H, D] under g [H], float64."""
    n, H, D = x.shape
    codes, scales = KV.quantize_heads(x, g)
    return O.dequantize_rows(codes.reshape(n * H, -1), scales.reshape(n * H, -1), np.tile(g, n)).reshape(n, H, D)


def _cache(nv, k, v, g, page, written=None):
    """(cache, table) of one sequence k, v fp32 [n, H, D] in pages in reverse order, with bytes
    that decode to NaN where nothing (or not `written`) is."""
    n, H, D = k.shape
    pages = -(-n // page)
    table = np.arange(pages, dtype=np.int32)[::-1].copy()
    slots = table[np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    if written is not None:
        slots[~written] = -1
    cache = nv.empty_kv_cache(pages, H, page, D).fill_(0x7F)
    nv.nvfp4_rope_append_kv(None, _dev(k.reshape(n, -1)), _dev(v.reshape(n, -1)), None, None,
                            torch.zeros(n, dtype=torch.int32, device="cuda"), _dev(slots), cache, _dev(g), _dev(g), page, None)
    return cache, _dev(table)[None]


def _attend(nv, q, cache, table, n, g, page, Hkv, most=None, window=0, scale=None):
    """q [m, Hq, D] of the dtype on the CPU -> (o, lse) float64."""
    m, Hq, D = q.shape
    x = q.reshape(m, -1).cuda()
    o, lse = torch.full_like(x, 3.0), torch.full((m, Hq), 3.0, device="cuda")
    most = most or n
    ws = torch.empty(nv.nvfp4_kv_attention_workspace(m, 1, Hq, Hkv, D, m, most, q.dtype), dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    nv.nvfp4_kv_attention(x, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), _dev(g), _dev(g), page, o, most,
                          ws, cu_q=cu, max_q_len=m, scale=scale, window=window, lse=lse)
    torch.cuda.synchronize()
    return o.double().cpu().numpy().reshape(m, Hq, D), lse.double().cpu().numpy()


def _check(q, k, v, got, scale, window, dtype):
    o, lse = got
    wo, wl, w = KV.attention(q.float().numpy(), k, v, scale, window)
    bo, bl = KV.attention_bounds(q.float().numpy(), k, v, w, scale, dtype)
    assert np.all(np.abs(o - wo) <= bo + O.ulp(wo, dtype)), np.max(np.abs(o - wo))
    assert np.all(np.abs(lse - wl) <= bl + 4 * 2.0 ** -24 * np.abs(wl))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,m,n,window,most", [
    (64, 1, 300, 33, 0), (128, 1, 301, 34, 0), (256, 1, 302, 35, 0), (128, 3, 300, 36, 0),
    (128, 1, 4096, 3001, 8192),                     # cut along the keys
    (64, 70, 300, 33, 0), (128, 70, 301, 34, 0), (256, 71, 300, 36, 0),   # prompts (bf16), cut
    (64, 70, 300, 33, -1), (128, 70, 301, 34, -1), (256, 71, 300, 36, -1)])   # and whole items
def test_slots_before_every_window_may_be_unwritten(nv, dtype, D, m, n, window, most):
    rng = np.random.default_rng(n + m + D)
    Hkv, Hq = (1, 4) if most >= 0 else (192, 768)
    most = max(most, n)
    k, v = rng.standard_normal((2, n, Hkv, D)).astype(np.float32)
    g = np.full(Hkv, 5 / 2688, dtype=np.float32)
    first = n - m - window + 1                      # of the first query's window
    assert first % 4 and first > 0
    cache, table = _cache(nv, k, v, g, 16, np.arange(n) >= first)
    q = torch.from_numpy(rng.standard_normal((m, Hq, D)).astype(np.float32)).to(DT[dtype])
    o, lse = _attend(nv, q, cache, table, n, g, 16, Hkv, most, window)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    kh = min(Hkv, 2)                                # heads whose values are checked
    _check(q[:, :4 * kh], _held(k[:, :kh], g[:kh]), _held(v[:, :kh], g[:kh]), (o[:, :4 * kh], lse[:, :4 * kh]), D ** -0.5,
           window, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,m,n,most", [
    (64, 1, 300, 0), (128, 1, 301, 0), (256, 2, 302, 0), (128, 9, 300, 0),
    (128, 1, 3000, 8192),                           # cut along the keys
    (64, 70, 300, 0), (128, 70, 301, 0), (256, 71, 300, 0), (128, 300, 333, 8192)])   # prompts (bf16)
@pytest.mark.parametrize("gain", [1e6, 1e8, 1e10, 1e20, 3e33, -1e8, -1e20, -3e33])
def test_scores_of_any_size(nv, dtype, D, m, n, most, gain):
    """Queries so long that a key stands out, or several are alike within the scores' rounding;
    gain < 0: all scores negative, the lowest near -1e35."""
    rng = np.random.default_rng(n + m + D)
    k, v = rng.standard_normal((2, n, 2, D)).astype(np.float32)
    x = rng.standard_normal((m, 6, D))
    if gain < 0:
        k, x = np.abs(k) + 0.25, np.abs(x)
    x[m // 2, 0] /= gain                            # a row of ordinary scores beside them
    g = np.full(2, 5 / 2688, dtype=np.float32)
    q = torch.from_numpy((x * gain).astype(np.float32)).to(DT[dtype])
    cache, table = _cache(nv, k, v, g, 16)
    o, lse = _attend(nv, q, cache, table, n, g, 16, 2, max(most, n))
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    kk, vv, scale = _held(k, g), _held(v, g), D ** -0.5
    qn = q.double().numpy()
    wo, wl, w = KV.attention(qn, kk, vv, scale)
    bo, bl = KV.attention_bounds(qn, kk, vv, w, scale, dtype)
    # the score's error with every key's magnitudes, not those of positive weights alone
    mag = scale * np.einsum("mhd,nhd->mhn", np.abs(qn), np.abs(np.repeat(kk, 3, 1))).max(-1)
    ds = ((D + 16) * 2.0 ** -24 + (2.0 ** -21 if dtype == "f32" else 0)) * mag + 16 * 2.0 ** -24
    assert np.all(np.abs(lse - wl) <= ds + np.log(n) + 1e-6 * np.abs(wl))
    ordinary = (m // 2, 0)
    assert np.all(np.abs(o[ordinary] - wo[ordinary]) <= bo[ordinary] + O.ulp(wo[ordinary], dtype))
    most_v = np.abs(vv).max()
    alone = 0
    for i in range(m):
        for h in range(6):
            s = scale * (kk[:n - m + i + 1, h // 3] @ qn[i, h])
            values = vv[:len(s), h // 3]
            # keys that the scores' error may make the largest: a mean of their values
            near = values[s >= s.max() - 4 * ds[i, h] - 40]
            alone += len(near) == 1
            slack = 2.0 ** -8 * most_v if dtype == "bf16" else 2.0 ** -19 * most_v
            assert np.all(o[i, h] <= near.max(0) + slack) and np.all(o[i, h] >= near.min(0) - slack)
    assert alone >= m                               # most rows have one such key


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 128)])
def test_bounds_far_above_the_lengths(nv, dtype, D):
    """65536 sequences, one of them with all 32768 queries: planned for what the bounds allow, the
    grid would have 2^23 workgroups of 512 threads (2^25 of 256), more than a launch takes."""
    rng = np.random.default_rng(D)
    batch, m, n, page = 1 << 16, 1 << 15, 600, 16
    k, v = rng.standard_normal((2, n, 1, D)).astype(np.float32)
    g = np.full(1, 5 / 2688, dtype=np.float32)
    cache, one = _cache(nv, k, v, g, page)
    q = torch.from_numpy(rng.standard_normal((m, D)).astype(np.float32)).to(DT[dtype])
    x = q.cuda()
    o, lse = torch.full_like(x, 3.0), torch.full((m, 1), 3.0, device="cuda")
    at = batch // 3
    table = torch.zeros(batch, one.shape[1], dtype=torch.int32, device="cuda")
    table[at] = one[0]
    kv_len = torch.full((batch,), 5, dtype=torch.int32, device="cuda")
    kv_len[at] = n
    cu = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    cu[at + 1:] = m
    need = nv.nvfp4_kv_attention_workspace(m, batch, 1, 1, D, m, n, q.dtype)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    nv.nvfp4_kv_attention(x, cache, table, kv_len, _dev(g), _dev(g), page, o, n, ws, cu_q=cu, max_q_len=m, lse=lse)
    torch.cuda.synchronize()
    o, lse = o.double().cpu().numpy()[:, None], lse.double().cpu().numpy()
    seen = m - n                                    # rows before it have no key
    assert np.all(o[:seen] == 0) and np.all(np.isneginf(lse[:seen]))
    kk, vv = _held(k, g), _held(v, g)
    for i in [seen, seen + 1, m - 257, m - 256, m - 255, m - 64, m - 2, m - 1]:
        end = i - seen + 1
        _check(q[i:i + 1, None], kk[:end], vv[:end], (o[i:i + 1], lse[i:i + 1]), D ** -0.5, 0, dtype)


def test_prompts_between_replays_of_a_captured_step(nv):
    """examples/attention_layer.py: prompt, capture, prompts that need more workspace, replay; the
    replays equal eager steps and write nowhere else."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    gen = torch.Generator("cuda").manual_seed(5)

    def rows(n):
        return torch.randn(n, 256, generator=gen, device="cuda").bfloat16()
    layer = example.AttentionLayer(256, 8, 2, 64, 3, 5000, 3000, page=16, seed=3)
    layer.cache.zero_()
    x, y = rows(33), torch.empty(3000, 256, dtype=torch.bfloat16, device="cuda")
    layer.prompt(x, [30, 2, 1], y[:33])
    x1, y1 = rows(3), torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    layer.decode(x1, y1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(x1, y1)
    held = layer.workspace.numel()
    for lens in ([100, 200, 300], [2000, 10, 900]):
        x = rows(sum(lens))
        layer.prompt(x, lens, y[:sum(lens)])
        torch.cuda.synchronize()
        guards = [torch.full((max(held, 1 << 20),), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
        steps = [rows(3) for _ in range(4)]
        got = []
        for s in steps:
            x1.copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            got.append(y1.clone())
        assert all(bool((t == 0x5A).all()) for t in guards)
        layer.prompt(x, lens, y[:sum(lens)])                      # again, then the same steps eagerly
        for s, want in zip(steps, got):
            x1.copy_(s)
            layer.decode(x1, y1)
            assert torch.equal(y1, want)
    assert layer.workspace.numel() > held


def test_strides_of_single_rows_and_columns_mean_nothing(nv):
    rng = np.random.default_rng(3)
    D, page, n = 64, 16, 16
    x = _dev(rng.standard_normal((1, 2 * D)).astype(np.float32))
    g = torch.full((2,), 0.002, device="cuda")
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(odd):
        one = (lambda t: t.as_strided(t.shape, (odd, 1))) if odd is not None else (lambda t: t)
        cache = nv.empty_kv_cache(1, 2, page, D).zero_()
        table = i32[:, None] if odd is None else i32.as_strided((1, 1), (odd, odd))
        outs = [torch.empty_like(x) for _ in range(4)]
        nv.nvfp4_rope_append_kv(one(x), one(x), one(x), None, None, i32, slots, cache, g, g, page, one(outs[0]))
        nv.nvfp4_kv_gather(cache, slots, g, g, page, one(outs[1]), one(outs[2]))
        nv.nvfp4_kv_attention(one(outs[0]), cache, table, i32 + 1, g, g, page, one(outs[3]), n)
        return outs + [cache]
    plain = step(None)
    for odd in (0, 1, 7, 1000):
        assert all(torch.equal(a, b) for a, b in zip(step(odd), plain))
    # several rows keep theirs: a table of one column, and rows that overlap are refused
    many = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = x.expand(3, -1).contiguous()
    o = [torch.empty_like(q) for _ in range(2)]
    for out, table in zip(o, (many[:, None], many.as_strided((3, 1), (1, 0)))):
        nv.nvfp4_kv_attention(q, plain[-1], table, many + 1, g, g, page, out, n)
    assert torch.equal(*o)
    for bad in (many.as_strided((3, 1), (0, 1)), many.as_strided((2, 2), (1, 1))):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_kv_attention(q[:bad.shape[0]], plain[-1], bad, many[:bad.shape[0]], g, g, page, o[0][:bad.shape[0]], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, -0.0])
@pytest.mark.parametrize("D,Hq,Hkv,kv,m", [
    (128, 4, 2, [130, 40], [1, 3]), (64, 4, 1, [3000, 70], [1, 1]), (256, 2, 1, [2500, 20], [2, 1]),
    (128, 4, 1, [300, 100], [90, 70]), (256, 4, 1, [200], [130]), (64, 56, 56, [300, 65, 7], [290, 65, 7])])
def test_scales_that_are_not_positive(nv, dtype, scale, D, Hq, Hkv, kv, m):
    p = Problem(nv, kv, m, Hq, Hkv, D, 16, dtype, seed=sum(kv))
    p.check(p.run(nv, scale=scale), scale=scale, rows=sorted({0, 1, 63, 64, 89, 129, 289}))


@pytest.mark.parametrize("batch,Hq,Hkv,D,dtype,most_m", [
    (65, 4, 1, 128, "bf16", 1), (100, 2, 2, 64, "bf16", 3), (130, 3, 1, 64, "f32", 1), (130, 4, 2, 128, "bf16", 2),
    (129, 20, 1, 64, "f32", 4), (66, 2, 1, 256, "bf16", 1)])
def test_many_sequences_cut_along_the_keys(nv, batch, Hq, Hkv, D, dtype, most_m):
    # more sequences than a wave's lanes: each lane counts the steps of several
    rng = np.random.default_rng(batch + D)
    kv = [int(n) for n in rng.integers(1, 400, batch)]
    m = [int(x) for x in rng.integers(0, most_m + 1, batch)] if most_m > 1 else [1] * batch
    for b in range(0, batch, 7):
        kv[b] = int(rng.integers(900, 1500))
    for b in (3, batch // 2 + 1, batch - 2):
        kv[b] = 0
    kv[-1] = 1400
    p = Problem(nv, kv, m, Hq, Hkv, D, 16, dtype, seed=batch)
    hints = (most_m, 9000)
    assert nv.nvfp4_kv_attention_workspace(p.T, batch, Hq, Hkv, D, *hints, p.q.dtype) > 0
    p.check(p.run(nv, hints=hints))
    p.check(p.run(nv, window=700, hints=hints), window=700)
    if most_m == 1:
        p.check(p.run(nv, hints=hints, use_cu=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,Hq,Hkv,rot,inter", [(64, 33, 2, 64, False), (128, 17, 1, 96, True), (256, 9, 1, 64, False),
                                                (256, 8, 2, 256, True), (64, 32, 1, 0, False)])
def test_append_beyond_the_caches(nv, dtype, D, Hq, Hkv, rot, inter):
    """Queries of more than 32 MiB, which are read and written past the caches."""
    size = 2 if dtype == "bf16" else 4
    T = (32 << 20) // (Hq * D * size) + 5
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, Hq + 2 * Hkv, D), dtype=np.float32)
    x = torch.from_numpy(x).to(DT[dtype]).float().numpy()
    g = np.full(Hkv, 5 / 2688, dtype=np.float32)
    pad, page, n_pos = 8, 64, 300
    buf = torch.full((T, (Hq + 2 * Hkv) * D + pad), float("nan"), dtype=DT[dtype], device="cuda")
    buf[:, :-pad] = _dev(x.reshape(T, -1))
    q, k, v = buf[:, :-pad].split([Hq * D, Hkv * D, Hkv * D], 1)
    n_pages = -(-T // page) + 1
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    slots[7] = -1
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    ang = rng.uniform(0, 50, (n_pos, max(rot // 2, 1)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    c, s = (_dev(cos), _dev(sin)) if rot else (None, None)
    rotate = (lambda a: KV.rotate_f32(a, cos[pos], sin[pos], inter)) if rot else (lambda a: a)
    want = torch.from_numpy(rotate(x[:, :Hq])).to(DT[dtype]).reshape(T, -1)
    wk, wv = _held(rotate(x[:, Hq:Hq + Hkv]), g), _held(x[:, Hq + Hkv:], g)
    wk[7], wv[7] = 0, 0
    out = torch.full((T, Hq * D + pad), 3.0, dtype=DT[dtype], device="cuda")
    for q_out in (out[:, :-pad], q):                # apart, then in place
        cache = nv.empty_kv_cache(n_pages, Hkv, page, D).fill_(0x7F)
        nv.nvfp4_rope_append_kv(q, k, v, c, s, _dev(pos), _dev(slots), cache, _dev(g), _dev(g), page, q_out, interleaved=inter)
        assert torch.equal(q_out.cpu().view(torch.int16 if size == 2 else torch.int32),
                           want.view(torch.int16 if size == 2 else torch.int32))
        k_out, v_out = torch.empty(2, T, Hkv * D, device="cuda")
        nv.nvfp4_kv_gather(cache, _dev(slots), _dev(g), _dev(g), page, k_out, v_out)
        for got, w in ((k_out, wk), (v_out, wv)):
            assert np.array_equal(got.cpu().numpy(), w.astype(np.float32).reshape(T, -1))
    assert bool((out[:, -pad:] == 3.0).all()) and bool(buf[:, -pad:].isnan().all())
