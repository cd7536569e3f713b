"""GPU parity of accepted paths, attention weights and eviction over the paged NVFP4 key/value
cache with the CPU oracle: rows and their weights move bit for bit, which tokens stay is equal,
weights are within the bound that oracle.kv.attention_weights derives."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from tests.test_gpu_kv import DT, Problem
from tests.test_gpu_kv_tree import draw_paths, mask_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


def dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x if dtype is None else np.asarray(x, dtype=dtype))).cuda()


class Sequences:
    """Sequences of the given lengths in shuffled pages of random bytes, every slot with a
    random weight per head; table entries past each end out of range."""

    def __init__(self, nv, kv, Hkv, D, page, seed, extra=2):
        rng = np.random.default_rng(seed)
        self.kv, self.Hkv, self.D, self.page = kv, Hkv, D, page
        need = [-(-n // page) for n in kv]
        self.n_pages = sum(need) + extra
        order = rng.permutation(self.n_pages)
        self.table = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, self.n_pages], (len(kv), max(need + [1]) + 1))
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.bytes = rng.integers(0, 256, (self.n_pages, Hkv * page * D * 9 // 8), dtype=np.uint8)
        self.weights = rng.standard_normal((self.n_pages, Hkv, page)).astype(np.float32)
        self.cache, self.dweights = dev(self.bytes), dev(self.weights)
        self.dtable, self.kv_len = dev(self.table, np.int32), dev(kv, np.int32)

    def slot(self, b, t):
        return int(self.table[b, t // self.page]) * self.page + t % self.page

    def row(self, flat, b, t, h):
        return np.concatenate(KV.byte_places(self.slot(b, t), h, self.Hkv, self.page, self.D))

    def weight(self, w, b, t, h):
        return w[self.table[b, t // self.page], h, t % self.page]

    def moved(self, rows):
        """The cache's bytes and the weights after token `old` of head h went to `place`, for
        rows (b, h, old, place), all read before any is written."""
        flat, w = self.bytes.reshape(-1).copy(), self.weights.copy()
        for b, h, old, place in rows:
            flat[self.row(flat, b, place, h)] = self.bytes.reshape(-1)[self.row(flat, b, old, h)]
            w[self.table[b, place // self.page], h, place % self.page] = self.weight(self.weights, b, old, h)
        return flat, w


# ----------------------------------------------------------------------------- accepted paths

@pytest.mark.parametrize("kv,m,paths,Hkv,D,page", [
    ([1], [1], [[0]], 1, 64, 16),
    ([30], [8], [[0, 2, 5]], 2, 128, 16),                             # across pages
    ([30, 7, 64, 50], [9, 7, 3, 20], [[0, 3, 4, 8], [], [1], [0, 1, 2, 3, 4]], 3, 64, 16),
    ([90, 66], [64, 60], [[0, 7, 20, 33, 34, 50, 63], [59]], 2, 256, 32),
    ([300, 20], [17, 2], [[3, 1, 2, 0], [1, 1]], 1, 128, 64),         # any order, the same one twice
    ([700], [300], [list(range(0, 300, 2))], 5, 64, 64),              # more rows than are held at a time
    ([520], [256], [list(range(255, -1, -1))], 2, 256, 16),           # the most, reversed
    ([16, 40], [0, 6], [[], [0, 5]], 64, 64, 16),                     # a sequence without a tree; many heads
])
@pytest.mark.parametrize("in_place", [False, True])
def test_accept(nv, kv, m, paths, Hkv, D, page, in_place):
    s = Sequences(nv, kv, Hkv, D, page, seed=sum(kv))
    most = max(max(map(len, paths)), 1)
    acc = np.full((len(kv), most + 2), -7)
    for b, p in enumerate(paths):
        acc[b, :len(p)] = p
    acc, count = dev(acc, np.int32)[:, :most], dev([len(p) for p in paths], np.int32)
    cu = dev(np.concatenate([[0], np.cumsum(m)]), np.int32)
    out = s.kv_len if in_place else torch.full_like(s.kv_len, -1)
    nv.nvfp4_kv_accept(s.cache, s.dtable, s.kv_len, cu, acc, count, Hkv, page, out)
    flat, _ = s.moved([(b, h, kv[b] - m[b] + a, kv[b] - m[b] + i) for b, p in enumerate(paths) for h in range(Hkv)
                       for i, a in enumerate(p)])
    assert np.array_equal(s.cache.cpu().numpy().reshape(-1), flat)
    assert out.tolist() == [n - mm + len(p) for n, mm, p in zip(kv, m, paths)]
    if not in_place:
        assert s.kv_len.tolist() == kv


def test_accept_one_token_each(nv):
    s = Sequences(nv, [20, 33], 2, 64, 16, seed=1)
    nv.nvfp4_kv_accept(s.cache, s.dtable, s.kv_len, None, dev([[0], [0]], np.int32), dev([1, 0], np.int32), 2, 16, s.kv_len)
    assert np.array_equal(s.cache.cpu().numpy(), s.bytes) and s.kv_len.tolist() == [20, 32]


def test_accept_clamps(nv):
    """Numbers and counts out of range, trees longer than their sequence, pages that are not there:
    nothing outside the sequence's own places is written."""
    s = Sequences(nv, [20, 40, 5], 2, 64, 16, seed=2)
    cu = dev([0, 6, 12, 20], np.int32)                                # the last tree has 8 nodes of 5 tokens
    s.dtable[1, 2] = 10 ** 6                                          # tokens 32 on have no page
    out = torch.zeros_like(s.kv_len)
    acc = dev([[-5, 100, 2 ** 31 - 1], [0, 3, 5], [4, 7, -2 ** 31]], np.int32)
    nv.nvfp4_kv_accept(s.cache, s.dtable, s.kv_len, cu, acc, dev([3, 99, -4], np.int32), 2, 16, out)
    flat, _ = s.moved([(0, h, 14 + a, 14 + i) for h in range(2) for i, a in enumerate([0, 5, 5])])
    assert np.array_equal(s.cache.cpu().numpy().reshape(-1), flat)
    assert out.tolist()[:2] == [17, 37] and 0 <= out.tolist()[2] <= 5


# ----------------------------------------------------------------------------- attention weights

class WeightProblem(Problem):
    def __init__(self, nv, kv, m, Hq, Hkv, D, page, dtype, seed, **kw):
        super().__init__(nv, kv, m, Hq, Hkv, D, page, dtype, seed, **kw)
        rng = np.random.default_rng(seed + 5)
        n_pages = self.cache.shape[0]
        self.old = np.full((n_pages, Hkv, page), np.nan, dtype=np.float32)
        used = self.slots
        self.old[used // page, :, used % page] = rng.random((len(used), Hkv)).astype(np.float32)

    def lse_of(self, nv, window, scale=None):
        return torch.from_numpy(self.run(nv, window, scale)[1].astype(np.float32))

    def run_weights(self, nv, lse, window=0, decay=1.0, scale=None, hints=None, use_cu=True, weights=None, pad=0):
        weights = dev(self.old) if weights is None else weights
        wide = torch.full((self.T, self.Hq * self.D + pad), float("nan"), dtype=DT[self.dtype], device="cuda")
        q = wide[:, :self.Hq * self.D]
        q.copy_(self.q.reshape(self.T, -1))
        mq, mk = hints or (max(self.m), max(self.kv))
        nv.nvfp4_kv_attention_weights(q, self.cache, self.table, self.kv_len, self.dkg, self.page, lse.cuda(), weights, mk,
                                      cu_q=self.cu if use_cu else None, max_q_len=mq, scale=scale, window=window, decay=decay)
        torch.cuda.synchronize()
        return weights.cpu().numpy()

    def check_weights(self, got, lse, window=0, decay=1.0, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        want, bound = self.old.astype(np.float64), np.zeros_like(self.old, dtype=np.float64)
        lse = lse.double().numpy()
        qa = ka = 0
        for n, m in zip(self.kv, self.m):
            if n and m:
                q = self.q[qa:qa + m].float().numpy()
                w, e = KV.attention_weights(q, self.k[ka:ka + n], lse[qa:qa + m], scale, window, self.dtype)
                s = self.slots[ka:ka + n]
                at = (s // self.page, slice(None), s % self.page)
                d = np.float64(np.float32(decay))
                old = np.where((np.arange(n) < n - m)[:, None], d * want[at], 0)
                if decay == 0:
                    old = np.zeros_like(old)
                want[at] = old + w
                bound[at] = e + 2.0 ** -24 * (np.abs(old) + np.abs(want[at])) * 1.01
            qa, ka = qa + m, ka + n
        assert np.array_equal(np.isnan(got), np.isnan(want))
        some = ~np.isnan(want)
        bad = np.abs(got - want)[some] > bound[some]
        assert not bad.any(), (np.abs(got - want)[some][bad].max(), bad.sum())
        untouched = bound == 0
        assert np.array_equal(got[untouched & some], self.old[untouched & some])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,m,Hq,Hkv,D,page,window,decay", [
    ([1], [1], 1, 1, 64, 16, 0, 1.0),
    ([0, 3, 17], [1, 1, 1], 4, 2, 64, 16, 0, 1.0),                   # an empty sequence
    ([15, 16, 17, 63, 64, 65, 129], [1] * 7, 8, 2, 128, 16, 0, 0.9),
    ([200, 31], [1, 1], 6, 2, 256, 32, 0, 0.5),
    ([300, 40, 5], [1, 1, 1], 5, 5, 128, 64, 33, 1.0),               # weights before the window stay
    ([300, 40, 5], [1, 1, 1], 5, 5, 128, 64, 33, 0.25),              # or fade
    ([700], [1], 20, 1, 64, 128, 0, 0.0),                            # more heads than a block; nothing of before
    ([90, 20, 64], [4, 1, 7], 4, 2, 128, 16, 0, 1.0),
    ([3, 50], [8, 2], 2, 1, 64, 16, 0, 0.5),                         # rows that see nothing
    ([40, 100, 7], [0, 100, 7], 3, 3, 128, 32, 9, 0.7),              # a sequence without queries keeps its weights
    ([150], [150], 4, 1, 256, 16, 0, 1.0),
    ([290, 333], [120, 333], 7, 7, 64, 64, 1, 0.9),                  # each token sees itself alone
    ([610, 40], [270, 40], 16, 2, 128, 32, 0, 1.0),                  # many query columns
    ([610, 40], [270, 40], 16, 2, 256, 32, 100, 0.9),
    ([500, 1], [333, 1], 12, 2, 64, 16, 77, 1.0),
])
def test_weights_match_oracle(nv, dtype, kv, m, Hq, Hkv, D, page, window, decay):
    p = WeightProblem(nv, kv, m, Hq, Hkv, D, page, dtype, seed=sum(kv) + D)
    lse = p.lse_of(nv, window)
    got = p.run_weights(nv, lse, window, decay)
    p.check_weights(got, lse, window, decay)
    if all(x == 1 for x in m):
        assert np.array_equal(p.run_weights(nv, lse, window, decay, use_cu=False), got, equal_nan=True)
    again = p.run_weights(nv, lse, window, decay, pad=8)             # the same order of sums
    assert np.array_equal(again, got, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,m,Hq,Hkv,D,window", [
    ([70, 33], [20, 5], 40, 1, 64, 0),                               # more heads of a group than a tile's rows
    ([150], [9], 66, 2, 128, 12),
    ([300, 2], [40, 2], 36, 1, 256, 0),
    ([2100], [17], 1, 1, 128, 0),                                    # one head
])
def test_weights_of_wide_groups(nv, dtype, kv, m, Hq, Hkv, D, window):
    p = WeightProblem(nv, kv, m, Hq, Hkv, D, 32, dtype, seed=Hq + D)
    lse = p.lse_of(nv, window)
    p.check_weights(p.run_weights(nv, lse, window, 0.75), lse, window, 0.75)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,batch", [(64, 40), (128, 40), (256, 20)])
@pytest.mark.parametrize("window", [0, 100])
def test_weights_of_runs(nv, dtype, D, batch, window):
    """Sequences so many that a wave has several steps of 64 tokens, of any length."""
    rng = np.random.default_rng(D)
    kv = rng.integers(1, 600, batch).tolist()
    kv[0], kv[1] = 128, 129
    p = WeightProblem(nv, kv, [1] * batch, 4, 4, D, 16, dtype, seed=D)
    lse = p.lse_of(nv, window)
    # as announced, and as for lengths of 20000 (a run of 3 to 16 steps)
    for most in (None, 20000, 150000):
        got = p.run_weights(nv, lse, window, 0.5, hints=most and (1, most))
        p.check_weights(got, lse, window, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,m", [(4, 4), (4, 5), (4, 8), (3, 11), (4, 16), (1, 17), (1, 33), (1, 64), (5, 13)])
def test_weights_of_paths(nv, dtype, D, Hq, m):
    """Up to one, two and four blocks of 16 query columns, and just past them; some sequences have fewer."""
    p = WeightProblem(nv, [300, 70, 64, 1000], [m, m - 1, 1, m], Hq, 1, D, 16, dtype, seed=D + m)
    for window, hints in ((0, None), (20, None), (0, (m, 200000))):
        lse = p.lse_of(nv, window)
        p.check_weights(p.run_weights(nv, lse, window, 0.5, hints=hints), lse, window, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hints", [(1, 1), (500, 100000), (2, 3)])
def test_weights_with_other_bounds(nv, dtype, hints):
    p = WeightProblem(nv, [1200, 77], [40, 60], 6, 2, 64, 16, dtype, seed=8)
    lse = p.lse_of(nv, 0)
    p.check_weights(p.run_weights(nv, lse, hints=hints), lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,scale", [(1, -0.3), (1, 0.0), (90, 0.5), (90, -0.1)])
def test_weights_of_other_scales(nv, dtype, m, scale):
    p = WeightProblem(nv, [130], [m], 8, 2, 64, 16, dtype, seed=3)
    lse = p.lse_of(nv, 0, scale)
    p.check_weights(p.run_weights(nv, lse, scale=scale), lse, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 60])
def test_rows_of_no_weight(nv, dtype, m):
    """A log-sum of -inf takes its row out, whatever its scores."""
    p = WeightProblem(nv, [100], [m], 8, 2, 128, 16, dtype, seed=4)
    lse = p.lse_of(nv, 0)
    lse[::2, 1] = -np.inf
    lse[1, :] = -np.inf
    p.check_weights(p.run_weights(nv, lse), lse)


@pytest.mark.parametrize("m", [1, 70])
def test_weights_pages_out_of_range(nv, m):
    """Weights whose page is not in the cache are not written."""
    p = WeightProblem(nv, [100], [m], 8, 1, 64, 16, "bf16", seed=6)
    lse = p.lse_of(nv, 0)
    whole = p.run_weights(nv, lse)
    gone = int(p.table[0, 1])
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        p.table[0, 1] = bad
        got = p.run_weights(nv, lse)
        rest = np.arange(got.shape[0]) != gone
        assert np.array_equal(got[rest], whole[rest], equal_nan=True)
        assert np.array_equal(got[gone], p.old[gone], equal_nan=True)


@pytest.mark.parametrize("m", [1, 40])
def test_weights_replayed(nv, m):
    """A captured call adds its weights at every replay."""
    p = WeightProblem(nv, [300, 80], [m, m], 8, 2, 128, 16, "bf16", seed=7)
    lse = p.lse_of(nv, 0).cuda()
    q, w = p.q.reshape(p.T, -1).cuda(), dev(p.old)

    def call(w):
        nv.nvfp4_kv_attention_weights(q, p.cache, p.table, p.kv_len, p.dkg, 16, lse, w, 300, cu_q=p.cu, max_q_len=m, decay=0.5)
    call(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w)
    w.copy_(dev(p.old))
    eager = dev(p.old)
    for _ in range(3):
        graph.replay()
        call(eager)
        torch.cuda.synchronize()
        assert np.array_equal(w.cpu().numpy(), eager.cpu().numpy(), equal_nan=True)


def test_weights_refusals(nv):
    p = WeightProblem(nv, [50, 9], [4, 2], 4, 2, 64, 16, "bf16", seed=1)
    q, lse, w = p.q.reshape(p.T, -1).cuda(), torch.zeros(6, 4, device="cuda"), dev(p.old)

    def call(q=q, lse=lse, w=w, cu=p.cu, kg=p.dkg, table=p.table, kv=p.kv_len, page=16, **kw):
        nv.nvfp4_kv_attention_weights(q, p.cache, table, kv, kg, page, lse, w, 50, **{"cu_q": cu, "max_q_len": 4, **kw})
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    call()
    for bad, status in ((dict(lse=lse[:5]), inv), (dict(lse=lse.double()), inv), (dict(lse=None), inv), (dict(w=None), inv),
                        (dict(w=w[:-1]), inv), (dict(w=w.double()), inv), (dict(w=w.transpose(1, 2)), inv),
                        (dict(q=q.half()), uns), (dict(q=q[:, :100]), inv), (dict(cu=None), inv), (dict(kg=p.dkg[:1]), inv),
                        (dict(table=p.table.long()), uns), (dict(kv=p.kv_len[:1]), inv), (dict(page=32), inv),
                        (dict(decay=float("nan")), inv), (dict(decay="x"), inv), (dict(window=-2), inv),
                        (dict(scale=float("inf")), inv), (dict(max_q_len=0), inv), (dict(w=w.cpu()), inv)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call(**bad)
        assert e.value.status == status, (bad, str(e.value))


# ----------------------------------------------------------------------------- eviction

def draw_weights(rng, shape, kind):
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.zeros(shape, np.float32) * np.where(rng.random(shape) < 0.5, -1, 1).astype(np.float32)   # 0 and -0
    w = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "odd":
        odd = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38, -1.0], dtype=np.float32)
        w = np.where(rng.random(shape) < 0.5, rng.choice(odd, shape), w)
    if kind == "signed":
        w = w * np.where(rng.random(shape) < 0.5, -1, 1).astype(np.float32)
    return w


class Eviction(Sequences):
    def __init__(self, nv, kv, Hkv, D, page, kind, seed):
        super().__init__(nv, kv, Hkv, D, page, seed)
        self.weights = draw_weights(np.random.default_rng(seed + 9), self.weights.shape, kind)
        self.dweights = dev(self.weights)

    def run(self, nv, budget, first, last, out="same", most=None, kept=True, in_place=False):
        ws = torch.empty(nv.nvfp4_kv_evict_workspace(len(self.kv), self.Hkv, budget, most or max(self.kv)),
                         dtype=torch.uint8, device="cuda")
        self.w_out = {"same": self.dweights, "none": None, "other": torch.full_like(self.dweights, -8.0)}[out]
        self.kept = torch.full((len(self.kv), self.Hkv, budget), -9, dtype=torch.int32, device="cuda") if kept else None
        self.len_out = self.kv_len if in_place else torch.full_like(self.kv_len, -1)
        nv.nvfp4_kv_evict(self.cache, self.dweights, self.dtable, self.kv_len, self.page, budget, self.len_out,
                          max(self.kv) if most is None else most, ws, keep_first=first, keep_last=last, weights_out=self.w_out,
                          kept=self.kept)

    def check(self, budget, first, last, out="same"):
        rows, same = [], []
        for b, n in enumerate(self.kv):
            for h in range(self.Hkv):
                w = [self.weight(self.weights, b, t, h) for t in range(n)]
                want = KV.evicted(w, n, budget, first, last)
                if self.kept is not None:
                    got = self.kept[b, h].tolist()
                    assert got[:len(want)] == want and all(x == -1 for x in got[len(want):]), (b, h)
                rows += [(b, h, old, place) for place, old in enumerate(want) if old != place]
                same += [(b, h, old, place) for place, old in enumerate(want) if old == place]
        flat, w = self.moved(rows)
        assert np.array_equal(self.cache.cpu().numpy().reshape(-1), flat)
        assert self.len_out.tolist() == [min(n, budget) for n in self.kv]
        bits = lambda x: x.cpu().numpy().view(np.uint32)              # noqa: E731
        if out == "same":
            assert np.array_equal(bits(self.w_out), w.view(np.uint32))
        else:
            assert np.array_equal(bits(self.dweights), self.weights.view(np.uint32))
        if out == "other":
            want = np.full_like(self.weights, -8.0)
            for b, h, old, place in rows + same:
                want[self.table[b, place // self.page], h, place % self.page] = self.weight(self.weights, b, old, h)
            assert np.array_equal(bits(self.w_out), want.view(np.uint32))


@pytest.mark.parametrize("kv,budget,first,last,Hkv,D,page", [
    ([2], 1, 0, 0, 1, 64, 16),
    ([10, 9, 0, 11], 10, 2, 3, 2, 64, 16),                           # one goes over by one
    ([40, 100, 64], 33, 1, 7, 2, 128, 16),
    ([40, 100, 64], 33, 0, 0, 2, 256, 32),
    ([300], 200, 4, 190, 3, 64, 64),                                 # the last tokens overlap their new places
    ([300], 200, 0, 200, 2, 128, 64),                                # nothing but the last ones
    ([300], 200, 200, 0, 2, 64, 16),                                 # nothing but the first ones
    ([1500, 700], 600, 10, 500, 1, 256, 128),                        # the last in more than a piece
    ([1100, 90, 1025], 64, 0, 16, 5, 64, 16),
    ([2100], 2099, 3, 1000, 2, 64, 256),                             # one goes, the rest moves by one
])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "signed"])
def test_evict(nv, kv, budget, first, last, Hkv, D, page, kind):
    s = Eviction(nv, kv, Hkv, D, page, kind, seed=sum(kv) + budget)
    s.run(nv, budget, first, last)
    s.check(budget, first, last)


@pytest.mark.parametrize("out", ["same", "none", "other"])
@pytest.mark.parametrize("most", [0, 100, 900, 50000])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_outputs_and_bounds(nv, out, most, in_place):
    s = Eviction(nv, [900, 31, 500], 2, 64, 16, "ties", seed=5)
    s.run(nv, 300, 5, 40, out, most, kept=out != "none", in_place=in_place)
    s.check(300, 5, 40, out)


@pytest.mark.parametrize("kv,budget,first,last", [([45000, 37000], 9000, 4, 300), ([70001], 70000, 0, 64), ([40000], 39000, 0, 0)])
@pytest.mark.parametrize("kind", ["plain", "ties"])
def test_evict_long(nv, kv, budget, first, last, kind):
    """More weights than a workgroup's memory holds."""
    s = Eviction(nv, kv, 1, 64, 128, kind, seed=budget)
    s.run(nv, budget, first, last)
    s.check(budget, first, last)


@pytest.mark.parametrize("n,budget,first,last,most", [
    (45000, 700, 3, 64, 100),                            # one workgroup a row, its keys not in registers
    (45000, 44000, 3, 1200, 16384),
    (70001, 3000, 0, 100, 17000),                        # parts far longer than announced
    (70001, 69000, 10, 2000, 20000),
    (30000, 29999, 0, 3000, 40000),                      # parts, the last tokens move by one
    (30000, 4000, 3000, 1000, 30000),                    # nothing but the first and the last ones
    (17000, 16400, 0, 16400, 17000),
])
@pytest.mark.parametrize("kind", ["ties", "equal", "odd", "signed"])
def test_evict_long_beside_its_bounds(nv, n, budget, first, last, most, kind):
    s = Eviction(nv, [n, 200], 1, 64, 128, kind, seed=budget)
    s.run(nv, budget, first, last, most=most)
    s.check(budget, first, last)


@pytest.mark.parametrize("out", ["none", "other"])
@pytest.mark.parametrize("D,Hkv", [(128, 2), (256, 1)])
def test_evict_long_outputs(nv, out, D, Hkv):
    s = Eviction(nv, [20000, 5000, 0], Hkv, D, 64, "ties", seed=D)
    s.run(nv, 6000, 2, 333, out, kept=out != "none", in_place=True)
    s.check(6000, 2, 333, out)


def test_evict_in_parts_replayed(nv):
    """The launches of a long eviction in a graph, replayed with eager calls between."""
    kv = [20000, 700]
    s = Eviction(nv, kv, 1, 64, 64, "ties", seed=12)
    s.run(nv, 2000, 2, 100, in_place=True)
    ws = torch.empty(nv.nvfp4_kv_evict_workspace(2, 1, 2000, 20000), dtype=torch.uint8, device="cuda")
    kept = torch.zeros(2, 1, 2000, dtype=torch.int32, device="cuda")

    def call():
        nv.nvfp4_kv_evict(s.cache, s.dweights, s.dtable, s.kv_len, 64, 2000, s.kv_len, 20000, ws, keep_first=2, keep_last=100,
                          weights_out=s.dweights, kept=kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, seed in enumerate((1, 2, 3, 4)):
        e = Eviction(nv, kv, 1, 64, 64, "ties", seed=12)
        e.weights = draw_weights(np.random.default_rng(seed), e.weights.shape, ("ties", "signed")[i % 2])
        for name, x in (("cache", e.bytes), ("dweights", e.weights), ("kv_len", np.array(e.kv, dtype=np.int32))):
            getattr(s, name).copy_(dev(x))
        torch.cuda.synchronize()
        call() if i == 2 else graph.replay()
        torch.cuda.synchronize()
        e.cache, e.dweights, e.w_out, e.kept, e.len_out = s.cache, s.dweights, s.dweights, kept, s.kv_len
        e.check(2000, 2, 100)


def test_two_evictions_at_once(nv):
    """Calls of different caches on two streams, each with its own workspace."""
    a, b = (Eviction(nv, [20000, 3000], 1, 64, 64, kind, seed=i) for i, kind in enumerate(("plain", "ties")))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a.run(nv, 1500, 1, 50)
    with torch.cuda.stream(side):
        b.run(nv, 1500, 1, 50)
    torch.cuda.synchronize()
    a.check(1500, 1, 50)
    b.check(1500, 1, 50)


@pytest.mark.parametrize("kv,budget,first,last,most", [
    ([4000, 3100, 700], 2000, 4, 64, None),
    ([9000, 2100], 1500, 0, 1000, None),
    ([2600, 2590], 1300, 5, 1290, None),                 # the last tokens' places meet or overlap their old ones
    ([30000, 5000], 2000, 1, 50, 4000),                  # longer than announced
    ([1999, 5000, 2001], 2000, 2000, 0, None),
])
@pytest.mark.parametrize("kind", ["ties", "odd"])
@pytest.mark.parametrize("out", ["same", "other"])
def test_evict_much_of_few(nv, kv, budget, first, last, most, kind, out):
    """Few rows of which much moves: chosen and moved in two launches."""
    s = Eviction(nv, kv, 2, 64, 64, kind, seed=budget)
    s.run(nv, budget, first, last, out, most=most)
    s.check(budget, first, last, out)


def test_evict_many_short_sequences(nv):
    rng = np.random.default_rng(0)
    kv = rng.integers(0, 60, 400).tolist()
    s = Eviction(nv, kv, 2, 64, 16, "plain", seed=3)
    s.run(nv, 24, 1, 6)
    s.check(24, 1, 6)


def test_evict_pages_out_of_range(nv):
    """Entries outside the cache and lengths past the table: only the sequence's own pages change."""
    s = Eviction(nv, [100, 60], 2, 64, 16, "plain", seed=4)
    other = s.table[1, :4].astype(int)
    s.dtable[0, 2], s.dtable[0, 5] = -5, 10 ** 6
    s.kv_len[0] = 2 ** 31 - 1
    s.run(nv, 50, 2, 10, most=100)
    torch.cuda.synchronize()
    got = s.cache.cpu().numpy()
    spare = [p for p in range(s.n_pages) if p not in s.table[0, :7].astype(int).tolist() and p not in other.tolist()]
    assert np.array_equal(got[spare], s.bytes[spare])
    s.kv_len[0] = -7
    s.run(nv, 50, 2, 10, most=100)
    assert s.len_out.tolist()[0] == 0


def test_evict_replayed(nv):
    """A captured eviction, its lengths in place: replays on new weights and lengths."""
    s = Eviction(nv, [500, 90, 260], 2, 128, 16, "plain", seed=6)
    s.run(nv, 120, 2, 30, in_place=True)                              # the modules are loaded
    fresh = Eviction(nv, [500, 90, 260], 2, 128, 16, "plain", seed=6)
    for name in ("cache", "dweights", "kv_len"):
        getattr(s, name).copy_(getattr(fresh, name))
    ws = torch.empty(nv.nvfp4_kv_evict_workspace(3, 2, 120, 500), dtype=torch.uint8, device="cuda")
    kept = torch.zeros(3, 2, 120, dtype=torch.int32, device="cuda")

    def call():
        nv.nvfp4_kv_evict(s.cache, s.dweights, s.dtable, s.kv_len, 16, 120, s.kv_len, 500, ws, keep_first=2, keep_last=30,
                          weights_out=s.dweights, kept=kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (6, 7, 8):
        e = Eviction(nv, [500, 90, 260], 2, 128, 16, "plain", seed=6)
        e.weights = draw_weights(np.random.default_rng(seed), e.weights.shape, "ties")
        for name, x in (("cache", e.bytes), ("dweights", e.weights), ("kv_len", np.array(e.kv, dtype=np.int32))):
            getattr(s, name).copy_(dev(x))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e.cache, e.dweights, e.w_out, e.kept, e.len_out = s.cache, s.dweights, s.dweights, kept, s.kv_len
        e.check(120, 2, 30)


def test_evict_and_accept_refusals(nv):
    s = Eviction(nv, [50, 9], 2, 64, 16, "plain", seed=1)
    ws = torch.empty(nv.nvfp4_kv_evict_workspace(2, 2, 20, 50), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out, kept = torch.zeros(2, **i32), torch.zeros(2, 2, 20, **i32)

    def evict(cache=s.cache, w=s.dweights, table=s.dtable, kv=s.kv_len, page=16, budget=20, out=out, ws=ws, **kw):
        nv.nvfp4_kv_evict(cache, w, table, kv, page, budget, out, 50, ws, **kw)

    acc, count = torch.zeros(2, 3, **i32), torch.ones(2, **i32)
    cu = torch.tensor([0, 3, 5], **i32)

    def accept(cache=s.cache, table=s.dtable, kv=s.kv_len, cu=cu, acc=acc, count=count, heads=2, page=16, out=out):
        nv.nvfp4_kv_accept(cache, table, kv, cu, acc, count, heads, page, out)
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for call, bad, status in (
            (evict, dict(cache=s.cache[:, :-1]), inv), (evict, dict(cache=s.cache.float()), inv), (evict, dict(w=s.dweights[0]), inv),
            (evict, dict(w=s.dweights.half()), inv), (evict, dict(table=s.dtable.long()), uns), (evict, dict(kv=s.kv_len.long()), inv),
            (evict, dict(budget=0), inv), (evict, dict(keep_first=15, keep_last=6), inv), (evict, dict(keep_last=-1), inv),
            (evict, dict(out=out[:1]), inv), (evict, dict(ws=None), inv), (evict, dict(ws=ws[:16]), inv), (evict, dict(page=8), inv),
            (evict, dict(weights_out=s.dweights[:-1]), inv), (evict, dict(kept=kept[:, :, :19]), inv),
            (evict, dict(kept=kept.long()), inv), (evict, dict(w=s.dweights.cpu()), inv), (evict, dict(ws=ws[::2]), inv),
            (accept, dict(cu=cu[:2]), inv), (accept, dict(acc=acc.long()), uns), (accept, dict(acc=acc[:1]), inv),
            (accept, dict(acc=acc[0]), inv), (accept, dict(count=count.float()), inv), (accept, dict(heads=3), inv),
            (accept, dict(heads=0), inv), (accept, dict(page=32), uns),   # the bytes are those of heads of 32
             (accept, dict(out=None), inv), (accept, dict(heads="2"), inv),
            (accept, dict(acc=torch.zeros(2, 257, **i32)), uns), (accept, dict(cache=s.cache.view(-1)), inv)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call(**bad)
        assert e.value.status == status, (bad, str(e.value))


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,D,group", [("bf16", 128, 4), ("f32", 64, 2), ("bf16", 256, 16)])
def test_generation_with_drafts_and_eviction(nv, dtype, D, group):
    """Prompts are attended to, weighed and cut; then rounds of drafted trees are appended, checked,
    accepted and weighed, with a cut when a sequence is over the budget.  Every attention output
    is the oracle's over the rows that each head should hold."""
    rng = np.random.default_rng(D)
    Hkv, page, budget, first, last, nodes = 2, 16, 48, 2, 9, 13
    Hq, B, prompts = Hkv * group, 3, [90, 40, 61]
    n_pages = 24
    table = rng.permutation(n_pages)[:B * 8].reshape(B, 8)
    cache = nv.empty_kv_cache(n_pages, Hkv, page, D)
    cache.fill_(0x7F)
    weights = torch.full((n_pages, Hkv, page), float("nan"), device="cuda")
    kg, vg = ((12 + rng.random(Hkv)) / 2688).astype(np.float32), ((11 + rng.random(Hkv)) / 2688).astype(np.float32)
    dkg, dvg, dtable = dev(kg), dev(vg), dev(table, np.int32)
    kv_len = dev(np.zeros(B), np.int32)
    held = [[[] for _ in range(Hkv)] for _ in range(B)]               # rows (k, v) of each head, by place
    wsum = [[[] for _ in range(Hkv)] for _ in range(B)]
    most = 128

    def append(m):
        """m new tokens of each sequence go behind its tokens; returns their queries."""
        T = sum(m)
        n = kv_len.tolist()
        slots = np.array([table[b, (n[b] + i) // page] * page + (n[b] + i) % page for b in range(B) for i in range(m[b])])
        x = rng.standard_normal((3, T, Hq, D)).astype(np.float32)
        q = torch.from_numpy(x[0]).to(DT[dtype]).cuda().view(T, -1)
        k, v = (torch.from_numpy(y[:, :Hkv]).to(DT[dtype]).cuda().reshape(T, -1) for y in x[1:])
        nv.nvfp4_rope_append_kv(None, k, v, None, None, torch.zeros(T, dtype=torch.int32, device="cuda"), dev(slots, np.int64),
                                cache, dkg, dvg, page, None)
        kv_len.add_(dev(m, np.int32))
        gk, gv = KV.gather(cache.cpu().numpy().reshape(-1), slots, Hkv, D, kg, vg, page)
        at = 0
        for b in range(B):
            for h in range(Hkv):
                held[b][h] += [(gk[at + i, h], gv[at + i, h]) for i in range(m[b])]
            at += m[b]
        return q, dev(np.concatenate([[0], np.cumsum(m)]), np.int32)

    def attend(q, cu, m, paths=None):
        o, lse = torch.empty_like(q), torch.empty(q.shape[0], Hq, device="cuda")
        ws = torch.empty(nv.nvfp4_kv_attention_workspace(q.shape[0], B, Hq, Hkv, D, max(m), most), dtype=torch.uint8, device="cuda")
        if paths is None:
            nv.nvfp4_kv_attention(q, cache, dtable, kv_len, dkg, dvg, page, o, most, ws, cu_q=cu, max_q_len=max(m), lse=lse)
        else:
            nv.nvfp4_kv_tree_attention(q, cache, dtable, kv_len, dkg, dvg, page, o, most, mask_of(rng, paths, 1), ws, cu_q=cu,
                                       max_q_len=max(m), lse=lse)
        host = q.float().cpu().numpy().reshape(-1, Hq, D)
        got, glse = o.float().cpu().numpy().reshape(-1, Hq, D), lse.cpu().numpy()
        at = 0
        for b in range(B):
            rows = slice(at, at + m[b])
            for h in range(Hkv):
                heads = slice(h * group, (h + 1) * group)
                k, v = (np.array([r[i] for r in held[b][h]])[:, None] for i in (0, 1))
                args = (host[rows, heads], k, v, D ** -0.5)
                wo, wl, w = KV.attention(*args) if paths is None else KV.tree_attention(*args, paths[b])
                bo, bl = KV.attention_bounds(host[rows, heads], k, v, w, D ** -0.5, dtype)
                half = torch.finfo(DT[dtype]).eps / 2
                assert np.all(np.abs(got[rows, heads] - wo) <= bo + half * np.abs(wo) * 1.01 + 1e-37)
                assert np.all(np.abs(glse[rows, heads] - wl) <= bl + 4 * 2.0 ** -24 * np.abs(wl))
            at += m[b]
        return lse

    def weigh(q, cu, m, lse):
        nv.nvfp4_kv_attention_weights(q, cache, dtable, kv_len, dkg, page, lse, weights, most, cu_q=cu, max_q_len=max(m))
        got = weights.cpu().numpy()
        for b in range(B):
            n = len(held[b][0])
            for h in range(Hkv):
                wsum[b][h] = [got[table[b, t // page], h, t % page] for t in range(n)]
                assert np.all(np.isfinite(wsum[b][h]))

    def cut():
        ws = torch.empty(nv.nvfp4_kv_evict_workspace(B, Hkv, budget, most), dtype=torch.uint8, device="cuda")
        nv.nvfp4_kv_evict(cache, weights, dtable, kv_len, page, budget, kv_len, most, ws, keep_first=first, keep_last=last,
                          weights_out=weights)
        for b in range(B):
            for h in range(Hkv):
                kept = KV.evicted(wsum[b][h], len(held[b][h]), budget, first, last)
                held[b][h] = [held[b][h][t] for t in kept]
        assert kv_len.tolist() == [len(held[b][0]) for b in range(B)]

    q, cu = append(prompts)
    weigh(q, cu, prompts, attend(q, cu, prompts))
    cut()
    for step in range(3):
        m = [nodes, nodes - step, 1]
        q, cu = append(m)
        paths = [draw_paths(rng, x) for x in m]
        lse = attend(q, cu, m, paths)
        # the path of the last node
        taken = [sorted(p[-1]) for p in paths]
        acc = np.zeros((B, max(map(len, taken))))
        for b, p in enumerate(taken):
            acc[b, :len(p)] = p
        nv.nvfp4_kv_accept(cache, dtable, kv_len, cu, dev(acc, np.int32), dev([len(p) for p in taken], np.int32), Hkv, page, kv_len)
        rows, at = [], 0
        for b, p in enumerate(taken):
            for h in range(Hkv):
                c = len(held[b][h]) - m[b]
                held[b][h] = held[b][h][:c] + [held[b][h][c + j] for j in p]
            rows += [at + j for j in p]
            at += m[b]
        assert kv_len.tolist() == [len(held[b][0]) for b in range(B)]
        # the accepted queries are now a chain
        rows = torch.tensor(rows, device="cuda")
        q, lse, m = q[rows].contiguous(), lse[rows].contiguous(), [len(p) for p in taken]
        cu = dev(np.concatenate([[0], np.cumsum(m)]), np.int32)
        again = attend(q, cu, m)
        assert torch.allclose(again, lse, atol=1e-4)
        weigh(q, cu, m, lse)
        cut()
