"""GPU parity of the attention of drafted trees over the paged NVFP4 key/value cache with the
CPU oracle (oracle.kv.tree_attention), within the per-element bound of attention_bounds plus
the output's own rounding."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import nvfp4 as O
from tests.test_gpu_kv import Problem


pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


def draw_paths(rng, m, kind="tree"):
    """The numbers of the query tokens that each of m query tokens attends to."""
    paths = []
    for j in range(m):
        if kind == "chain":
            paths.append(set(range(j + 1)))
        elif kind == "self":
            paths.append({j})
        elif kind == "none":
            paths.append(set())
        elif kind == "any":                       # any bits at all, later tokens among them
            paths.append(set(np.flatnonzero(rng.random(m) < 0.3).tolist()))
        else:
            paths.append((paths[rng.integers(max(0, j - 8), j)] if j else set()) | {j})
    return paths


def mask_of(rng, paths_of, words, noise=True):
    """tree_mask [T, words]; with noise, bits that no query token has are set at random."""
    rows = []
    for paths in paths_of:
        for p in paths:
            x = sum(1 << j for j in p)
            if noise:
                extra = int(rng.integers(0, 2 ** 62)) << max(len(paths), 0)
                x |= extra & ((1 << 64 * words) - 1)
            rows.append([(x >> 64 * w) & (2 ** 64 - 1) for w in range(words)])
    return torch.from_numpy(np.array(rows, dtype=np.uint64).reshape(len(rows), words).view(np.int64)).cuda()


class TreeProblem(Problem):
    def __init__(self, nv, kv, m, Hq, Hkv, D, page, dtype, seed, kinds=("tree",), words=None, **kw):
        super().__init__(nv, kv, m, Hq, Hkv, D, page, dtype, seed, **kw)
        rng = np.random.default_rng(seed + 1)
        self.paths = [draw_paths(rng, mm, kinds[i % len(kinds)]) for i, mm in enumerate(m)]
        self.words = words or -(-max(max(m), 1) // 64)
        self.mask = mask_of(rng, self.paths, self.words)

    def run_tree(self, nv, window=0, scale=None, hints=None, use_cu=True, mask=None, stream=None):
        q = self.q.reshape(self.T, -1).cuda()
        o = torch.full_like(q, 3.0)
        lse = torch.full((self.T, self.Hq), 3.0, device="cuda")
        mq, mk = hints or (max(self.m), max(self.kv))
        ws = torch.empty(nv.nvfp4_kv_attention_workspace(self.T, len(self.kv), self.Hq, self.Hkv, self.D, mq, mk, q.dtype),
                         dtype=torch.uint8, device="cuda")
        nv.nvfp4_kv_tree_attention(q, self.cache, self.table, self.kv_len, self.dkg, self.dvg, self.page, o, mk,
                                   self.mask if mask is None else mask, ws, cu_q=self.cu if use_cu else None,
                                   max_q_len=mq, scale=scale, window=window, lse=lse, stream=stream)
        torch.cuda.synchronize()
        return o.float().cpu().numpy().reshape(self.T, self.Hq, self.D).astype(np.float64), \
            lse.cpu().numpy().astype(np.float64)

    def check_tree(self, got, window=0, scale=None, rows=None):
        """rows: query tokens of each sequence to check (None: all)."""
        scale = self.D ** -0.5 if scale is None else scale
        o, lse = got
        qa = ka = 0
        for n, m, paths in zip(self.kv, self.m, self.paths):
            k, v = self.k[ka:ka + n], self.v[ka:ka + n]
            which = np.arange(m) if rows is None else np.array([r for r in rows if r < m], dtype=int)
            if len(which):
                q = self.q[qa:qa + m].float().numpy()
                if rows is None:
                    wo, wl, w = KV.tree_attention(q, k, v, scale, paths, window)
                else:                             # the oracle of single rows
                    parts = [self._row(q[i:i + 1], k, v, scale, paths[i], m, window) for i in which]
                    wo, wl, w = (np.concatenate([p[x] for p in parts]) for x in range(3))
                q = q[which]
                go, gl = o[qa:qa + m][which], lse[qa:qa + m][which]
                bo, bl = KV.attention_bounds(q, k, v, w, scale, self.dtype)
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
                fin = np.isfinite(wl)
                assert np.all(np.abs(go - wo) <= bo + O.ulp(wo, self.dtype)), np.max(np.abs(go - wo))
                assert np.all(np.abs(gl - np.where(fin, wl, 0))[fin] <= (bl + 4 * 2.0 ** -24 * np.abs(wl))[fin])
                assert np.all(go[~fin] == 0)
            qa, ka = qa + m, ka + n

    @staticmethod
    def _row(q, k, v, scale, path, m, window):
        c = k.shape[0] - m
        at = list(range(c)) + [c + j for j in sorted(path) if c + j >= 0]
        return KV._attend(q, k, v, scale, [at[-window:] if window else at])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,m,Hq,Hkv,D,page,window", [
    ([1], [1], 1, 1, 64, 16, 0),                                   # one node, one head, no context
    ([9], [9], 4, 2, 128, 16, 0),                                  # a tree without context
    ([300, 45], [8, 5], 8, 2, 128, 64, 0),
    ([17, 0, 64, 129], [3, 0, 7, 16], 6, 3, 64, 16, 0),            # an empty sequence among them
    ([200, 100], [33, 64], 8, 2, 256, 32, 0),                      # a whole word of bits
    ([500, 150], [65, 100], 4, 2, 128, 64, 0),                     # two words
    ([170], [130], 2, 2, 64, 128, 0),                              # three
    ([400, 90], [60, 90], 5, 5, 128, 32, 40),                      # windows that end inside the tree, or before it
    ([80, 33], [30, 20], 4, 1, 64, 16, 3),                         # windows shorter than the paths
    ([50], [40], 3, 3, 256, 16, 1),                                # one token each
    ([5, 30], [12, 4], 4, 2, 128, 16, 0),                          # more nodes than tokens
    ([5, 30], [12, 4], 4, 2, 64, 16, 2),
    ([90, 60, 40], [70, 30, 9], 20, 2, 128, 16, 0),                # more columns than a tile
])
def test_tree_matches_oracle(nv, dtype, kv, m, Hq, Hkv, D, page, window):
    p = TreeProblem(nv, kv, m, Hq, Hkv, D, page, dtype, seed=sum(kv) + D, kinds=("tree", "any"))
    p.check_tree(p.run_tree(nv, window), window)


@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 16, 2, 32), (128, 8, 1, 16), (256, 8, 2, 64)])
@pytest.mark.parametrize("window", [0, 37, 700])
def test_many_columns(nv, D, Hq, Hkv, page, window):
    """Trees of 256 columns a kv head and more: the kernel of prompts, whole and in pieces."""
    p = TreeProblem(nv, [1500, 70, 900], [70, 64, 129], Hq, Hkv, D, page, "bf16", seed=D + window,
                    kinds=("tree", "any", "tree"))
    rows = [0, 1, 17, 40, 63, 64, 69, 100, 128]
    p.check_tree(p.run_tree(nv, window), window, rows=rows)
    p.check_tree(p.run_tree(nv, window, hints=(129, 1)), window, rows=rows)         # a bound far below the lengths
    p.check_tree(p.run_tree(nv, window, hints=(192, 100000)), window, rows=rows)    # and above them (the mask's bits)


@pytest.mark.parametrize("kv,m,D", [([9000], [20], 128), ([20000], [70], 64), ([6000], [130], 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts_are_cut(nv, dtype, kv, m, D):
    p = TreeProblem(nv, kv, m, 4, 2, D, 128, dtype, seed=D)
    p.check_tree(p.run_tree(nv), rows=[0, 1, m[0] // 2, m[0] - 1])
    p.check_tree(p.run_tree(nv, 5000), 5000, rows=[0, m[0] // 2, m[0] - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_bits(nv, dtype):
    """Rows without a bit attend to the context alone; without context they are empty."""
    p = TreeProblem(nv, [40, 6, 7], [7, 6, 5], 4, 2, 64, 16, dtype, seed=3, kinds=("none", "none", "self"))
    for window in (0, 4):
        got = p.run_tree(nv, window)
        p.check_tree(got, window)
        assert np.all(np.isneginf(got[1][7:13])) and np.all(got[0][7:13] == 0)


@pytest.mark.parametrize("dtype,m", [("bf16", [5, 3]), ("bf16", [70, 64]), ("f32", [9, 1])])
@pytest.mark.parametrize("window", [0, 21])
def test_a_chain_is_causal_attention(nv, dtype, m, window):
    p = TreeProblem(nv, [333, 80], m, 8, 2, 128, 16, dtype, seed=m[0], kinds=("chain",))
    got = p.run_tree(nv, window)
    p.check(got, window)
    p.check_tree(got, window)


def test_one_token_each_without_cu_q(nv):
    p = TreeProblem(nv, [100, 31, 1], [1, 1, 1], 4, 2, 128, 32, "bf16", seed=9)
    a, b = p.run_tree(nv, use_cu=False), p.run_tree(nv)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    p.check_tree(a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_gain,scale", [(1e4, None), (1.0, -3.0), (3.0, 1e7), (1.0, 0.0), (1e-30, None)])
def test_scores_of_any_size(nv, dtype, q_gain, scale):
    p = TreeProblem(nv, [60, 33], [20, 33], 4, 2, 64, 16, dtype, seed=4, q_gain=q_gain)
    o, lse = p.run_tree(nv, scale=scale)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse))
    if not (q_gain > 1 or (scale or 0) > 1):
        p.check_tree((o, lse), scale=scale)


@pytest.mark.parametrize("Hq,words", [(2, 64), (16, 64)])
def test_widest_masks(nv, Hq, words):
    """64 words of bits a row, of which the sequences use a part, in rows that lie apart."""
    p = TreeProblem(nv, [700, 20], [300, 7], Hq, 2, 64, 16, "bf16", seed=Hq, kinds=("any", "tree"), words=words)
    wide = torch.full((p.T, words + 3), -1, dtype=torch.int64, device="cuda")
    wide[:, :words] = p.mask
    p.check_tree(p.run_tree(nv, hints=(300, 700), mask=wide[:, :words]), rows=[0, 6, 63, 64, 150, 255, 256, 299])


@pytest.mark.parametrize("D,Hq,m", [(64, 2, 600), (128, 1, 700), (256, 2, 330)])
@pytest.mark.parametrize("window", [0, 50])
def test_words_that_are_not_kept(nv, D, Hq, m, window):
    """Trees of so many words that a tile's are read where they are used."""
    p = TreeProblem(nv, [m + 100], [m], Hq, 1, D, 16, "bf16", seed=D + m, kinds=("any",))
    p.check_tree(p.run_tree(nv, window), window, rows=[0, 63, 64, 128, 255, 256, m // 2, m - 1])


@pytest.mark.parametrize("D,Hq,Hkv,m", [(64, 4, 2, 3), (128, 8, 1, 11), (128, 16, 1, 12), (256, 8, 1, 20)])
@pytest.mark.parametrize("window", [0, 19])
def test_more_sequences_than_lanes(nv, D, Hq, Hkv, m, window):
    """66 to 70 trees, of up to 24, 88, 192 and 160 columns a kv head."""
    rng = np.random.default_rng(m)
    kv = rng.integers(m, 200, 66 + D % 5).tolist()
    p = TreeProblem(nv, kv, rng.integers(0, m + 1, len(kv)).tolist(), Hq, Hkv, D, 16, "bf16", seed=m, kinds=("tree", "any"))
    p.check_tree(p.run_tree(nv, window, hints=(m, 200)), window, rows=[0, 1, m // 2, m - 1])


@pytest.mark.parametrize("Hq,Hkv,m", [(8, 1, 9), (8, 1, 16), (8, 1, 17), (4, 1, 32), (4, 1, 33), (3, 1, 41), (9, 1, 14), (5, 1, 26)])
@pytest.mark.parametrize("kv", [[190], [900, 60, 400] * 24])
def test_columns_about_a_tile(nv, Hq, Hkv, m, kv):
    """Just below and above the columns where another kernel or form of it takes over, whole and cut."""
    p = TreeProblem(nv, kv, [m] * len(kv), Hq, Hkv, 64, 16, "bf16", seed=Hq * m)
    p.check_tree(p.run_tree(nv), rows=[0, m // 2, m - 1])


@pytest.mark.parametrize("Hq,m", [(4, 9), (16, 40)])
@pytest.mark.parametrize("window", [0, 30])
def test_nodes_that_no_row_sees_may_be_unwritten(nv, Hq, m, window):
    """The slots of nodes without a bit in any row hold what decodes to NaN: nothing of it is
    in a result (and nothing of slots before every window)."""
    n = 100
    p = TreeProblem(nv, [n], [m], Hq, 2, 128, 16, "bf16", seed=m + window)
    hidden = set(range(1, m, 3))
    p.paths[0] = [q - hidden for q in p.paths[0]]
    p.mask = mask_of(np.random.default_rng(0), p.paths, 1, noise=False)
    want = p.run_tree(nv, window)
    gone = [n - m + j for j in sorted(hidden)]
    if window:
        most = max(len(q) for q in p.paths[0])
        least = min(len(q) for q in p.paths[0])
        assert most < window
        gone += list(range(n - m - (window - least)))
    # a granule's bytes of the token: keys, key scales, values, value scales
    flat = p.cache.view(-1)
    for h in range(2):
        for t in gone:
            for at in KV.byte_places(int(p.slots[t]), h, 2, 16, 128):
                flat[torch.from_numpy(at).cuda()] = 0x7F
    got = p.run_tree(nv, window)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    p.check_tree(got, window)


def test_lengths_and_tables_out_of_range(nv):
    """Lengths past the table, negative ones and pages outside the cache are clamped."""
    p = TreeProblem(nv, [100, 50], [9, 70], 8, 1, 64, 16, "bf16", seed=2)
    for bad in ([-5, 50], [10 ** 6, 2 ** 31 - 1], [3, -2 ** 31]):
        p.kv_len = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = p.run_tree(nv)
        assert o.shape == (79, 8, 64)
    p.cu = torch.tensor([0, 1000, -7], dtype=torch.int32, device="cuda")
    p.run_tree(nv)


@pytest.mark.parametrize("Hq,m", [(8, [9, 3]), (32, [64, 20])])
def test_graph_replays(nv, Hq, m):
    p = TreeProblem(nv, [600, 90], m, Hq, 2, 128, 64, "bf16", seed=11)
    q = p.q.reshape(p.T, -1).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(p.T, Hq, device="cuda")
    ws = torch.empty(nv.nvfp4_kv_attention_workspace(p.T, 2, Hq, 2, 128, max(m), 1000), dtype=torch.uint8, device="cuda")
    mask = p.mask.clone()

    def call():
        nv.nvfp4_kv_tree_attention(q, p.cache, p.table, p.kv_len, p.dkg, p.dvg, 64, o, 1000, mask, ws, cu_q=p.cu,
                                   max_q_len=max(m), lse=lse)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    rng = np.random.default_rng(5)
    for kind in ("tree", "any", "self"):
        p.paths = [draw_paths(rng, mm, kind) for mm in m]
        mask.copy_(mask_of(rng, p.paths, p.words))
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        call()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        p.mask = mask
        p.check_tree((o.float().cpu().numpy().reshape(p.T, Hq, 128).astype(np.float64), lse.cpu().numpy().astype(np.float64)),
                     rows=[0, 2, 8, 19, 63])


def test_two_calls_at_once(nv):
    """Two trees on two streams, each call with its own workspace."""
    a, b = (TreeProblem(nv, [5000, 300], [m, 9], 8, 2, 128, 32, "bf16", seed=m) for m in (40, 12))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for p, stream in ((a, None), (b, side)):
        q = p.q.reshape(p.T, -1).cuda()
        torch.cuda.synchronize()
        o, lse = torch.empty_like(q), torch.empty(p.T, 8, device="cuda")
        ws = torch.empty(nv.nvfp4_kv_attention_workspace(p.T, 2, 8, 2, 128, 40, 5000), dtype=torch.uint8, device="cuda")
        outs.append((p, stream, q, o, lse, ws))
    torch.cuda.synchronize()
    for p, stream, q, o, lse, ws in outs:
        nv.nvfp4_kv_tree_attention(q, p.cache, p.table, p.kv_len, p.dkg, p.dvg, 32, o, 5000, p.mask, ws, cu_q=p.cu, max_q_len=40,
                                   lse=lse, stream=stream)
    torch.cuda.synchronize()
    for p, _, _, o, lse, _ in outs:
        p.check_tree((o.float().cpu().numpy().reshape(p.T, 8, 128).astype(np.float64), lse.cpu().numpy().astype(np.float64)),
                     rows=[0, 5, 39])


def test_on_another_stream(nv):
    p = TreeProblem(nv, [200, 64], [17, 8], 8, 2, 64, 32, "bf16", seed=6)
    want = p.run_tree(nv)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = p.run_tree(nv)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    got = p.run_tree(nv, stream=side)
    assert np.array_equal(got[0], want[0])


def test_refusals(nv):
    p = TreeProblem(nv, [50, 9], [4, 2], 4, 2, 64, 16, "bf16", seed=1)
    q = p.q.reshape(p.T, -1).cuda()
    o = torch.empty_like(q)

    def call(mask=p.mask, q=q, o=o, mq=4, window=0, cu=p.cu):
        nv.nvfp4_kv_tree_attention(q, p.cache, p.table, p.kv_len, p.dkg, p.dvg, 16, o, 50, mask, None, cu_q=cu,
                                   max_q_len=mq, window=window)
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    call()
    for bad, status in ((dict(mask=None), inv), (dict(mask=p.mask.int()), uns), (dict(mask=p.mask.view(-1)), inv),
                        (dict(mask=p.mask[:3]), inv), (dict(mask=p.mask.cpu()), inv), (dict(mq=65), inv),
                        (dict(mask=torch.zeros(6, 65, dtype=torch.int64, device="cuda")), uns),
                        (dict(mask=torch.zeros(6, 0, dtype=torch.int64, device="cuda")), inv),
                        (dict(mask=torch.zeros(2, 6, dtype=torch.int64, device="cuda").t()), inv),
                        (dict(window=-1), inv), (dict(o=o.float()), uns), (dict(cu=None), inv), (dict(mq=0), inv)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call(**bad)
        assert e.value.status == status, (bad, str(e.value))
