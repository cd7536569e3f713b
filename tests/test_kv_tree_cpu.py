"""Drafted trees over the key/value cache on the CPU: the entry point's refusals, all before
the GPU is touched, and pins of the oracle."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv as KV
from tests.test_kv_abi_cpu import FAKE, ODD, nv  # noqa: F401  (the fixture)


def _tree(nv, mask=FAKE, words=1, ldm=1, mq=4, T=6, batch=2, cu=FAKE, q=FAKE, o=FAKE, window=0, d=128, mk=10):  # noqa: F811
    return nv.lib.nvfp4_kv_tree_attention(q, 1, 512, T, 4, 2, d, batch, cu, mq, FAKE, mk, FAKE, 4, 4, FAKE, 4, 16, FAKE, FAKE,
                                          ctypes.c_float(0.1), window, mask, words, ldm, o, 512, None, None, 0, None)


def test_tree_validation(nv):  # noqa: F811
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    assert _tree(nv, mask=None) == inv and "tree_mask" in nv.nvfp4_last_error()
    assert _tree(nv, words=0) == inv and _tree(nv, words=65, ldm=65) == uns and _tree(nv, words=2) == inv
    assert _tree(nv, mq=65) == inv and "bits" in nv.nvfp4_last_error()
    assert _tree(nv, mask=ODD) == uns
    assert _tree(nv, q=None) == inv and _tree(nv, o=None) == inv and _tree(nv, cu=None) == inv
    assert _tree(nv, window=-1) == inv and _tree(nv, d=96) == uns and _tree(nv, mk=-1) == inv and _tree(nv, T=0) == inv


def _case(rng, n, m, Hq, Hkv, D):
    return rng.standard_normal((m, Hq, D)), rng.standard_normal((n, Hkv, D)), rng.standard_normal((n, Hkv, D))


@pytest.mark.parametrize("n,m,window", [(9, 4, 0), (9, 4, 3), (6, 6, 0), (3, 5, 2), (7, 7, 1)])
def test_oracle_chain_is_causal(n, m, window):
    q, k, v = _case(np.random.default_rng(n), n, m, 4, 2, 8)
    chain = [range(i + 1) for i in range(m)]
    for a, b in zip(KV.tree_attention(q, k, v, 0.3, chain, window), KV.attention(q, k, v, 0.3, window)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("window", [0, 1, 3, 100])
def test_oracle_against_dense_masks(window):
    rng = np.random.default_rng(window)
    n, m, Hq, Hkv, D = 11, 6, 4, 2, 8
    q, k, v = _case(rng, n, m, Hq, Hkv, D)
    paths = [{0}, {0, 1}, {0, 2}, {0, 2, 3}, set(), {1, 5}]
    o, lse, w = KV.tree_attention(q, k, v, 0.3, paths, window)
    for i, p in enumerate(paths):
        sees = [t < n - m or t - (n - m) in p for t in range(n)]
        if window:                                    # the last `window` of those seen
            for t in np.flatnonzero(sees)[:-window]:
                sees[t] = False
        for h in range(Hq):
            e = np.where(sees, np.exp(0.3 * k[:, h // 2] @ q[i, h]), 0)
            assert np.allclose(w[i, h], e / e.sum()) and np.isclose(lse[i, h], np.log(e.sum()))
            assert np.allclose(o[i, h], (e / e.sum()) @ v[:, h // 2])


def test_oracle_empty_rows():
    q, k, v = _case(np.random.default_rng(0), 2, 2, 2, 1, 8)
    o, lse, w = KV.tree_attention(q, k, v, 1.0, [set(), {0, 1}])
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.all(w[0] == 0) and np.all(np.isfinite(lse[1]))


@pytest.mark.skipif(torch.cuda.is_available(), reason="its buffers are not real: where there is a GPU the calls would be launched")
def test_workspace_covers_every_window(nv):  # noqa: F811
    """A window may change how a tree's call is planned: the workspace that is asked for without
    one is enough (the call is not refused for it: without a GPU it goes on to look for the
    device)."""
    for T, batch, hq, hkv, d, mq, mk in ((480, 8, 32, 8, 128, 60, 4096), (64, 2, 32, 8, 128, 32, 131072), (256, 8, 16, 2, 256, 32, 8192),
                                         (40, 5, 15, 5, 64, 8, 100000), (960, 16, 32, 8, 128, 60, 8192)):
        for dt, dtype in ((1, torch.bfloat16), (0, torch.float32)):
            need = nv.nvfp4_kv_attention_workspace(T, batch, hq, hkv, d, mq, mk, dtype)
            for window in (0, 1, 17, 300, 2000, 20000):
                st = nv.lib.nvfp4_kv_tree_attention(FAKE, dt, hq * d, T, hq, hkv, d, batch, FAKE, mq, FAKE, mk, FAKE, mk // 16 + 1,
                                                    mk // 16 + 1, FAKE, 1 << 20, 16, FAKE, FAKE, ctypes.c_float(0.1), window, FAKE, 1, 1,
                                                    FAKE, hq * d, None, FAKE, need, None)
                assert st in (nv.NVFP4_ERR_HIP, nv.NVFP4_ERR_DEVICE), (T, window, nv.nvfp4_last_error())
