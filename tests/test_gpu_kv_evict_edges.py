"""Edges of the attention weights and of eviction over the paged NVFP4 key/value cache, against the
CPU oracle: rows that are taken out, bounds below the lengths, pages that are not there."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from tests.test_gpu_kv_evict import Eviction, WeightProblem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


# ----------------------------------------------------------------------------- attention weights

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,m,Hq,Hkv,window,hints", [
    ([400, 70], [1, 1], 8, 2, 0, None),                  # a generated token each
    ([400, 70], [3, 2], 8, 2, 90, None),
    ([400, 70], [5, 4], 9, 1, 0, None),                  # blocks of 16 columns whose last is not full
    ([400, 70], [30, 9], 4, 2, 0, (1, 400)),             # more columns than announced
    ([900, 40], [70, 40], 8, 2, 0, None),                # many columns
    ([900, 40], [70, 40], 5, 1, 300, None),              # tiles of less than 32 rows
    ([600], [11], 40, 1, 0, None),                       # more heads of a group than a tile's rows
])
def test_queries_of_rows_of_no_weight(nv, dtype, D, kv, m, Hq, Hkv, window, hints):
    """Rows whose log-sum is -inf have no weights whatever their queries hold, as the rows of a batch that
    is padded to a fixed size do: NaN, infinities, values whose products overflow."""
    p = WeightProblem(nv, kv, m, Hq, Hkv, D, 16, dtype, seed=D + Hq)
    lse = p.lse_of(nv, window)
    rng = np.random.default_rng(Hq)
    gone = rng.random((p.T, Hq)) < 0.3
    gone[0] = True                                       # a whole query token
    gone[-1, 0] = True
    lse[torch.from_numpy(gone)] = -np.inf
    for i, h in np.argwhere(gone):
        kind = (i + h) % 4
        p.q[i, h] = (float("nan"), float("inf"), 3e38, -float("inf"))[kind]
        if kind == 3:
            p.q[i, h, ::2] = 1.0                         # products of both signs, and ordinary ones
    got = p.run_weights(nv, lse, window, 0.5, hints=hints)
    p.check_weights(got, lse, window, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 700])
@pytest.mark.parametrize("kv,m,Hq,Hkv,window", [
    ([2500, 310], [90, 310], 8, 2, 0),
    ([2500, 310], [90, 310], 8, 2, 400),                 # a window that leaves whole turns of tokens out
    ([2500, 310], [40, 17], 40, 1, 0),                   # more heads of a group than a tile's rows
    ([1200, 300] + [20] * 6, [9] * 8, 128, 16, 0),       # waves that have tokens each, of many heads
])
def test_many_columns_of_more_tokens_than_announced(nv, dtype, D, most, kv, m, Hq, Hkv, window):
    """A workgroup takes tokens again and again where the lengths are above their bound."""
    p = WeightProblem(nv, kv, m, Hq, Hkv, D, 32, dtype, seed=D + Hq)
    lse = p.lse_of(nv, window)
    got = p.run_weights(nv, lse, window, 0.5, hints=(max(m), most))
    p.check_weights(got, lse, window, 0.5)


# ----------------------------------------------------------------------------- eviction

def ranked(s, b, t, h, missing):
    """A token whose page is not there ranks last."""
    return -np.inf if b == 0 and t // s.page == missing else s.weight(s.weights, b, t, h)


@pytest.mark.parametrize("kv,budget,first,last,page", [
    ([100, 60], 50, 2, 10, 16),                          # a workgroup a row
    ([4000, 3100], 2000, 4, 200, 64),                    # chosen and moved in two launches
    ([20000, 700], 2000, 2, 300, 64),                    # in parts
    ([20000, 700], 19900, 2, 300, 64),                   # and places that overlap
])
@pytest.mark.parametrize("gone", ["source", "place"])
def test_every_place_of_kept_is_written(nv, kv, budget, first, last, page, gone):
    """A row whose page, or whose place's page, is not in the cache does not move: kept has the place itself
    there, and no place of kept is left as it was."""
    s = Eviction(nv, kv, 2, 64, page, "plain", seed=budget)
    n = kv[0]
    token = n - last // 2 if gone == "source" else budget - last // 2      # among the last ones
    missing = token // page
    s.dtable[0, missing] = -1 if gone == "source" else 10 ** 6
    s.run(nv, budget, first, last, out="none")
    for b, n in enumerate(kv):
        for h in range(2):
            w = np.array([ranked(s, b, t, h, missing) for t in range(n)])
            want = np.array(KV.evicted(w, n, budget, first, last))
            if b == 0 and n > budget:
                place = np.arange(budget)
                still = (want // page == missing) | (place // page == missing)
                assert still[budget - last:].any()
                want = np.where(still, place, want)
            got = s.kept[b, h].cpu().numpy()
            assert np.array_equal(got[:len(want)], want) and np.all(got[len(want):] == -1), (b, h)
