"""The attention layer of examples/attention_layer.py on the GPU, stage by stage against the
CPU oracle: prompts, then generated tokens eagerly and from a replayed graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import nvfp4 as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _np(t):
    return t.float().cpu().numpy()


def _linear(layer, x):
    codes, scales, g = O.quantize_activation(_np(x).astype(np.float64), float(layer.gscale.item()))
    y, _ = O.linear_reference(codes, scales, g, layer.codes.cpu().numpy(), layer.scales.cpu().numpy(), layer.seg_end,
                              layer.seg_gscale.cpu().numpy(), "bf16")
    return y


class Mirror:
    """The layer's cache as the oracle appends to it, from the layer's own projections."""

    def __init__(self, layer):
        self.layer = layer
        self.cache = layer.cache.cpu().numpy().reshape(-1).copy()
        self.cos, self.sin = _np(layer.cos), _np(layer.sin)
        self.kg, self.vg = _np(layer.k_gscale), _np(layer.v_gscale)

    def slots(self, b, n):
        t = np.arange(n)
        return self.layer.table.cpu().numpy()[b][t // self.layer.page].astype(np.int64) * self.layer.page + t % self.layer.page

    def check(self, x, y, lens, total):
        """The layer's last call: lens new tokens per sequence, total with them."""
        la = self.layer
        T, n_q, n_kv, d = x.shape[0], la.n_q, la.n_kv, la.d
        want = _linear(la.qkv, x)
        rows = _np(la.qkv_rows[:T])                               # its queries are rotated by now
        kv = rows[:, n_q * d:]
        assert np.linalg.norm(kv - want[:, n_q * d:]) <= 1e-3 * np.linalg.norm(want[:, n_q * d:])
        pos = np.concatenate([np.arange(t - m, t) for m, t in zip(lens, total)])
        slots = np.concatenate([self.slots(b, t)[t - m:] for b, (m, t) in enumerate(zip(lens, total))])
        qr = KV.rotate_f32(want[:, :n_q * d].reshape(T, n_q, d).astype(np.float32), self.cos[pos], self.sin[pos], False)
        # the projection's 1e-3 and the rotated queries' own rounding, 2^-9 at most
        assert np.linalg.norm(rows[:, :n_q * d] - qr.reshape(T, -1)) <= 4e-3 * np.linalg.norm(qr)
        k, v = kv.reshape(T, 2, n_kv, d).transpose(1, 0, 2, 3)
        KV.append(self.cache, KV.rotate_f32(k, self.cos[pos], self.sin[pos], False), v, slots, self.kg, self.vg, la.page)
        assert np.array_equal(la.cache.cpu().numpy().reshape(-1), self.cache)
        q, o, at = rows[:, :n_q * d].reshape(T, n_q, d), _np(la.o_rows[:T]).reshape(T, n_q, d), 0
        for b, (m, n) in enumerate(zip(lens, total)):
            k, v = KV.gather(self.cache, self.slots(b, n), n_kv, d, self.kg, self.vg, la.page)
            wo, _, w = KV.attention(q[at:at + m], k, v, d ** -0.5, 0)
            bo, _ = KV.attention_bounds(q[at:at + m], k, v, w, d ** -0.5, "bf16")
            assert np.all(np.abs(o[at:at + m] - wo) <= bo + O.ulp(wo, "bf16"))
            at += m
        want = _linear(la.out, la.o_rows[:T])
        assert np.linalg.norm(_np(y) - want) <= 1e-3 * np.linalg.norm(want)


def test_prompts_then_generation(example):
    hidden, lens = 256, [70, 1, 33]
    layer = example.AttentionLayer(hidden, 8, 2, 64, 3, 160, sum(lens), page=16, seed=3)
    layer.cache.zero_()
    mirror = Mirror(layer)
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(sum(lens), hidden, generator=gen, device="cuda").bfloat16()
    y = torch.empty_like(x)
    layer.prompt(x, lens, y)
    torch.cuda.synchronize()
    mirror.check(x, y, lens, lens)

    total = list(lens)
    x1 = torch.empty(3, hidden, dtype=torch.bfloat16, device="cuda")
    y1 = torch.empty_like(x1)
    layer.reserve(3, 1)

    def step(run):
        nonlocal total
        x1.copy_(torch.randn(3, hidden, generator=gen, device="cuda"))
        run()
        torch.cuda.synchronize()
        total = [t + 1 for t in total]
        assert layer.kv_len.tolist() == total
        mirror.check(x1, y1, [1, 1, 1], total)

    for _ in range(2):
        step(lambda: layer.decode(x1, y1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(x1, y1)
    for _ in range(4):
        step(graph.replay)
