"""GPU parity of drafted trees' attention in every form of the prompts' kernel with the CPU oracle: two groups of waves
for up to 128 columns and one for more, items whole and cut along the keys, windows, more than 64 sequences,
column tiles past the planned ones, words that LDS does not hold (tests/test_kv_tree_forms_cpu.py has the sizes, and
checks that they are planned for that kernel)."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from tests.test_gpu_kv_tree import TreeProblem, mask_of
from tests.test_kv_tree_forms_cpu import FORMS, form_id

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


def rows_of(f):
    edges = (f.tile // f.group, 2 * (f.tile // f.group))
    return sorted({0, 1, 5, 31, 32, 39, 63, 64, max(f.m) // 2, max(f.m) - 2, max(f.m) - 1}
                  | {r + d for r in edges for d in (-1, 0)})


def problem(nv, f, kinds):
    return TreeProblem(nv, list(f.kv), list(f.m), f.group * f.Hkv, f.Hkv, f.D, 16, "bf16", seed=f.D + f.tile + len(f.kv),
                       kinds=kinds, words=f.words)


@pytest.mark.parametrize("f", FORMS, ids=form_id)
def test_form_matches_oracle(nv, f):
    p = problem(nv, f, ("tree", "any"))
    hints = (f.most_q, f.most_kv)
    got = p.run_tree(nv, f.window, hints=hints)
    p.check_tree(got, f.window, rows=rows_of(f))
    again = p.run_tree(nv, f.window, hints=hints)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("f", FORMS, ids=form_id)
def test_form_of_unwritten_nodes(nv, f):
    """Slots of nodes without a bit in any row, in several granules of 16 tokens, and those before every window
    may hold what decodes to NaN: nothing of it is in a result."""
    p = problem(nv, f, ("tree", "chain"))
    rng = np.random.default_rng(1)
    hidden = [set(np.flatnonzero(rng.random(m) < 0.3).tolist()) for m in p.m]
    p.paths = [[q - h for q in paths] for paths, h in zip(p.paths, hidden)]
    p.mask = mask_of(rng, p.paths, p.words, noise=False)
    hints = (f.most_q, f.most_kv)
    want = p.run_tree(nv, f.window, hints=hints)
    flat, ka, gone = p.cache.view(-1), 0, 0
    for n, m, paths, h in zip(p.kv, p.m, p.paths, hidden):
        own = [len([j for j in q if n - m + j >= 0]) for q in paths]
        at = [n - m + j for j in h if n - m + j >= 0]
        if f.window and m and max(own) < f.window:
            at += range(n - m - (f.window - min(own)))
        for t in at:
            for head in range(p.Hkv):
                for places in KV.byte_places(int(p.slots[ka + t]), head, p.Hkv, 16, p.D):
                    flat[torch.from_numpy(places).cuda()] = 0x7F
        ka, gone = ka + n, gone + len(at)
    assert gone > 10
    got = p.run_tree(nv, f.window, hints=hints)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    p.check_tree(got, f.window, rows=rows_of(f))


SOME = [f for f in FORMS if f.most_q >= max(f.m) <= 64]


@pytest.mark.parametrize("f", SOME, ids=form_id)
def test_form_of_pages_out_of_range(nv, f):
    """A sequence whose pages are not in the cache gets results without a meaning and nothing else changes; table
    entries past a sequence's pages are never looked at."""
    p = problem(nv, f, ("tree", "any"))
    hints = (f.most_q, f.most_kv)
    want = p.run_tree(nv, f.window, hints=hints)
    rest = np.arange(p.T) >= p.m[0]                      # the rows of the other sequences
    for bad in (-1, 2 ** 31 - 1, -2 ** 31, p.cache.shape[0]):
        p.table[0, :] = bad
        got = p.run_tree(nv, f.window, hints=hints)
        assert np.array_equal(got[0][rest], want[0][rest]) and np.array_equal(got[1][rest], want[1][rest])


@pytest.mark.parametrize("D,Hq,Hkv,m,hints", [
    (64, 8, 1, [9, 70], None),                           # k_kv_attn
    (64, 8, 2, [20, 12], (20, 1000000)),                 # two groups of waves
    (128, 16, 2, [20, 12], (20, 1000000)),               # one
])
@pytest.mark.parametrize("kv", [[-5, 50], [10 ** 6, 2 ** 31 - 1], [3, -2 ** 31]])
def test_lengths_out_of_range_are_clamped(nv, D, Hq, Hkv, m, hints, kv):
    """Lengths outside their range give what the clamped ones do; rows of a sequence without tokens are empty."""
    p = TreeProblem(nv, [100, 50], m, Hq, Hkv, D, 16, "bf16", seed=D)
    p.table.clamp_(0, p.cache.shape[0] - 1)
    p.cache.fill_(0x22)                                  # every slot has a value
    hints = hints or (max(m), 100)
    lens = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    p.kv_len = lens(kv)
    got = p.run_tree(nv, hints=hints)
    most = p.table.shape[1] * 16
    p.kv_len = lens([min(max(n, 0), most) for n in kv])
    want = p.run_tree(nv, hints=hints)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    rows = np.concatenate([[0], np.cumsum(m)])
    for b, n in enumerate(kv):
        own = slice(rows[b], rows[b + 1])
        if n <= 0:
            assert np.all(got[0][own] == 0) and np.all(np.isneginf(got[1][own]))
        else:
            assert np.all(np.isfinite(got[0][own]))


@pytest.mark.parametrize("D,Hq,Hkv,hints", [(64, 8, 1, (30, 100)), (64, 8, 2, (20, 1000000)), (128, 16, 2, (20, 1000000))])
def test_query_bounds_out_of_range_are_clamped(nv, D, Hq, Hkv, hints):
    """cu_q past q's rows ends with them, and a falling one gives a sequence without rows, whose outputs stay."""
    p = TreeProblem(nv, [100, 50], [20, 12], Hq, Hkv, D, 16, "bf16", seed=D + 1, kinds=("any",))
    lens = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    for bad, good in (([0, 20, 1000], [0, 20, 32]), ([-9, 20, 32], [0, 20, 32]), ([0, 20, -7], [0, 20, 20])):
        p.cu = lens(bad)
        got = p.run_tree(nv, hints=hints)
        p.cu = lens(good)
        want = p.run_tree(nv, hints=hints)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert np.all(got[0][good[2]:] == 3.0) and np.all(got[1][good[2]:] == 3.0)
