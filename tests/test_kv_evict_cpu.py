"""Accepted paths, attention weights and eviction over the key/value cache on the CPU: the entry
points' refusals, all before the GPU is touched, and pins of the oracle."""

import ctypes

import numpy as np
import pytest

from oracle import kv as KV
from tests.test_kv_abi_cpu import FAKE, ODD, nv  # noqa: F401  (the fixture)

F32 = ctypes.c_float


def at(offset):
    return ctypes.c_void_p(FAKE.value + offset)


def _accept(nv, cache=FAKE, pages=4, page=16, hkv=2, d=128, batch=2, kv=FAKE, cu=FAKE, table=FAKE, mp=4, ldt=4, acc=FAKE,  # noqa: F811
            most=3, lda=3, n=FAKE, out=FAKE):
    return nv.lib.nvfp4_kv_accept(cache, pages, page, hkv, d, batch, kv, cu, table, mp, ldt, acc, most, lda, n, out, None)


def test_accept_validation(nv):  # noqa: F811
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("cache", "kv", "table", "acc", "n", "out"):
        assert _accept(nv, **{name: None}) == inv, name
    assert _accept(nv, cache=ODD) == uns and _accept(nv, d=96) == uns and _accept(nv, page=24) == uns
    assert _accept(nv, batch=0) == inv and _accept(nv, hkv=0) == inv and _accept(nv, pages=0) == inv
    assert _accept(nv, most=0) == inv and _accept(nv, lda=2) == inv and _accept(nv, most=257, lda=257) == uns
    assert _accept(nv, mp=0) == inv and _accept(nv, ldt=3) == inv and _accept(nv, mp=1 << 30, ldt=1 << 30) == inv
    assert _accept(nv, out=at(4)) == inv and "overlaps" in nv.nvfp4_last_error()
    assert _accept(nv, batch=1 << 22, hkv=2) == uns


def _weights(nv, q=FAKE, dt=1, ldq=512, T=2, hq=4, hkv=2, d=128, batch=2, cu=None, mq=1, kv=FAKE, mk=10, table=FAKE, mp=4,  # noqa: F811
             ldt=4, cache=FAKE, pages=4, page=16, kg=FAKE, scale=0.1, window=0, lse=FAKE, w=FAKE, decay=1.0):
    return nv.lib.nvfp4_kv_attention_weights(q, dt, ldq, T, hq, hkv, d, batch, cu, mq, kv, mk, table, mp, ldt, cache, pages,
                                             page, kg, F32(scale), window, lse, w, F32(decay), None)


def test_weights_validation(nv):  # noqa: F811
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("q", "kv", "table", "cache", "kg", "lse", "w"):
        assert _weights(nv, **{name: None}) == inv, name
    assert _weights(nv, w=ODD) == uns and _weights(nv, q=ODD) == uns and _weights(nv, cache=ODD) == uns
    assert _weights(nv, T=3) == inv and _weights(nv, T=0) == inv and _weights(nv, hq=3) == inv and _weights(nv, batch=0) == inv
    assert _weights(nv, mq=0) == inv and _weights(nv, mk=-1) == inv and _weights(nv, window=-1) == inv
    for bad in (float("nan"), float("inf")):
        assert _weights(nv, scale=bad) == inv and _weights(nv, decay=bad) == inv
    assert _weights(nv, dt=3) == uns and _weights(nv, d=80) == uns and _weights(nv, page=20) == uns
    assert _weights(nv, mp=0) == inv and _weights(nv, ldt=1) == inv and _weights(nv, ldq=256) == inv


def _evict(nv, cache=FAKE, pages=4, page=16, hkv=2, d=128, w=FAKE, wo=None, batch=2, kv=FAKE, mk=60, table=FAKE, mp=4, ldt=4,  # noqa: F811
           budget=20, first=1, last=2, kept=None, out=FAKE, ws=FAKE, wsb=1 << 20):
    return nv.lib.nvfp4_kv_evict(cache, pages, page, hkv, d, w, wo, batch, kv, mk, table, mp, ldt, budget, first, last, kept,
                                 out, ws, wsb, None)


def test_evict_validation(nv):  # noqa: F811
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("cache", "w", "kv", "table", "out", "ws"):
        assert _evict(nv, **{name: None}) == inv, name
    assert _evict(nv, cache=ODD) == uns and _evict(nv, w=ODD) == uns and _evict(nv, wo=ODD) == uns and _evict(nv, ws=ODD) == uns
    assert _evict(nv, wo=at(16)) == inv and "overlaps" in nv.nvfp4_last_error()
    assert _evict(nv, out=at(4)) == inv and _evict(nv, out=at(-4)) == inv
    assert _evict(nv, budget=0) == inv and _evict(nv, budget=(1 << 30) + 1) == inv
    assert _evict(nv, first=-1) == inv and _evict(nv, last=-1) == inv and _evict(nv, first=10, last=11) == inv
    assert _evict(nv, first=1 << 62, last=1 << 62) == inv and _evict(nv, mk=-1) == inv
    assert _evict(nv, wsb=100) == inv and "workspace" in nv.nvfp4_last_error()
    assert _evict(nv, d=32) == uns and _evict(nv, page=17) == uns and _evict(nv, batch=0) == inv and _evict(nv, mp=0) == inv
    assert _evict(nv, batch=1 << 22, hkv=2) == uns


def test_evict_workspace(nv):  # noqa: F811
    need = nv.nvfp4_kv_evict_workspace(3, 4, 100, 5000)
    assert need >= 3 * 4 * 100 * 4
    assert nv.nvfp4_kv_evict_workspace(2, 4, 100, 5000) <= need and nv.nvfp4_kv_evict_workspace(3, 4, 100, 50) <= need
    for bad in ((0, 4, 100, 10), (1, 0, 100, 10), (1, 4, 0, 10), (1, 4, 100, -1), (1 << 22, 2, 10, 10)):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_kv_evict_workspace(*bad)
    assert nv.lib.nvfp4_kv_evict_workspace(1, 1, 1, 1, None) == nv.NVFP4_ERR_INVALID_ARG


@pytest.mark.parametrize("window", [0, 3])
def test_oracle_weights_sum_to_rows(window):
    """Under the attention's own log-sums every row's weights sum to 1 (rows that see nothing: 0)."""
    rng = np.random.default_rng(window)
    m, n, Hq, Hkv, D = 7, 5, 6, 2, 8                     # more query tokens than tokens: two rows are empty
    q, k = rng.standard_normal((m, Hq, D)), rng.standard_normal((n, Hkv, D))
    _, lse, w = KV.attention(q, k, k, 0.4, window)
    total, bound = KV.attention_weights(q, k, lse, 0.4, window)
    assert np.isclose(total.sum(), (m - 2) * Hq) and np.all(bound > 0)
    want = w.reshape(m, Hkv, Hq // Hkv, n).sum((0, 2)).T
    assert np.allclose(total, want)


def test_oracle_weights_bound_admits_fp32_and_no_more():
    rng = np.random.default_rng(1)
    m, n, Hq, D = 20, 50, 2, 64
    q, k = rng.standard_normal((m, Hq, D)).astype(np.float32), rng.standard_normal((n, 1, D)).astype(np.float32)
    _, lse, _ = KV.attention(q, k, k, 0.125)
    lse = lse.astype(np.float32)
    total, bound = KV.attention_weights(q, k, lse, 0.125)
    got = np.zeros((n, 1), np.float32)
    for i in range(m):
        for h in range(Hq):
            p = n - m + i + 1
            s = (k[:p, 0] @ q[i, h]) * np.float32(0.125)
            got[:p, 0] += np.exp(s - lse[i, h])
    assert np.all(np.abs(got - total) <= bound)
    assert not np.all(np.abs(got * (1 + 1e-4) - total) <= bound)


@pytest.mark.parametrize("n,budget,first,last", [(9, 9, 1, 1), (10, 4, 0, 0), (10, 4, 1, 2), (10, 4, 2, 2), (50, 49, 3, 20),
                                                 (50, 10, 0, 10), (50, 10, 10, 0), (33, 1, 0, 0)])
def test_oracle_eviction(n, budget, first, last):
    rng = np.random.default_rng(n + budget)
    w = rng.integers(0, 5, n).astype(float)               # many ties
    w[rng.integers(0, n, 3)] = np.nan
    kept = KV.evicted(w, n, budget, first, last)
    assert len(kept) == len(set(kept)) == min(n, budget)
    if n <= budget:
        assert kept == list(range(n))
        return
    assert kept[:first] == list(range(first)) and (last == 0 or kept[-last:] == list(range(n - last, n)))
    key = [(np.inf if np.isnan(w[t]) else -w[t], t) for t in range(n)]
    middle, out = kept[first:budget - last], set(range(first, n - last)) - set(kept)
    if middle and out:
        assert max(key[t] for t in middle) < min(key[t] for t in out)
    moved = [t for place, t in enumerate(kept) if t != place and place < budget - last]
    assert moved == sorted(moved) and all(t >= budget - last for t in moved)
