"""GPU parity of the paged NVFP4 key/value cache through the C ABI against the CPU oracle:
appended bytes, rotated queries and read-back values bit-exact; attention within the
per-element bound that oracle.kv.attention_bounds derives (plus the output's own
rounding)."""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from oracle import nvfp4 as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _draw(rng, shape, dtype):
    """Values of the dtype (as fp32) with a few large channels."""
    x = rng.standard_normal(shape).astype(np.float32)
    x[..., :: 13] *= 5
    return torch.from_numpy(x).to(DT[dtype]).float().numpy()


def _gscales(rng, H):
    return ((12 + rng.random(H)) / 2688).astype(np.float32), ((11 + rng.random(H)) / 2688).astype(np.float32)


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


# ----------------------------------------------------------------------------- append, gather

@pytest.mark.parametrize("T,dtype,D,Hq,Hkv,page,rot,inter", [
    (1, "bf16", 128, 4, 1, 64, 128, False),       # one token
    (7, "f32", 64, 6, 2, 16, 64, False),          # a granule cut short
    (33, "bf16", 64, 3, 3, 32, 32, True),         # partial interleaved rotation
    (50, "f32", 256, 4, 2, 16, 64, False),        # a quarter of the head rotated
    (70, "bf16", 256, 2, 1, 256, 256, True),
    (129, "f32", 128, 5, 5, 128, 96, False),      # rotated width that is no power of two
    (40, "bf16", 128, 0, 2, 16, 0, False),        # no queries, no rotation
])
def test_append_is_bit_exact(nv, T, dtype, D, Hq, Hkv, page, rot, inter):
    rng = np.random.default_rng(T * 7 + D)
    x = _draw(rng, (T, Hq + 2 * Hkv, D), dtype)
    x[T // 2, Hq, :16] = 0.0                                  # a zero block
    x[T // 2, Hq, 16:32] = -0.0
    x[0, -1, :16] = 1e4                                       # saturates its block scale
    kg, vg = _gscales(rng, Hkv)
    n_pages = -(-T // page) + 2
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    if T > 5:
        slots[3], slots[5] = -1, n_pages * page               # tokens that are not appended
    n_pos = 512
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    ang = rng.uniform(0, 50, (n_pos, max(rot // 2, 1)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)

    pad = 8                                                   # one fused projection, rows longer than their data
    buf = torch.full((T, (Hq + 2 * Hkv) * D + pad), float("nan"), dtype=DT[dtype], device="cuda")
    buf[:, :-pad] = torch.from_numpy(x.reshape(T, -1))
    q, k, v = buf[:, :-pad].split([Hq * D, Hkv * D, Hkv * D], 1)
    cache = nv.empty_kv_cache(n_pages, Hkv, page, D)
    cache.fill_(0xAB)
    q_out = torch.empty(T, Hq * D, dtype=DT[dtype], device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()               # noqa: E731
    c, s = (dev(cos), dev(sin)) if rot else (None, None)
    args = (dev(pos), dev(slots), cache, dev(kg), dev(vg), page)
    nv.nvfp4_rope_append_kv(q if Hq else None, k, v, c, s, *args, q_out if Hq else None, interleaved=inter)

    rotate = (lambda a: KV.rotate_f32(a, cos[pos], sin[pos], inter)) if rot else (lambda a: a)
    want = np.full(cache.numel(), 0xAB, dtype=np.uint8)
    KV.append(want, rotate(x[:, Hq:Hq + Hkv]), x[:, Hq + Hkv:], slots, kg, vg, page)
    assert np.array_equal(cache.cpu().numpy().reshape(-1), want)
    if Hq:
        wq = torch.from_numpy(rotate(x[:, :Hq])).to(DT[dtype]).reshape(T, -1)
        assert np.array_equal(_bits(q_out), _bits(wq))
        nv.nvfp4_rope_append_kv(q, k, v, c, s, *args, q, interleaved=inter)      # in place
        assert np.array_equal(_bits(q.contiguous()), _bits(wq))

    for out in ("f32", "bf16"):
        k_out = torch.full((T, Hkv * D + 8), 7.0, dtype=DT[out], device="cuda")[:, :Hkv * D]
        v_out = torch.full_like(k_out, 7.0)
        nv.nvfp4_kv_gather(cache, args[1], args[3], args[4], page, k_out, v_out)
        wk, wv = KV.gather(want, slots, Hkv, D, kg, vg, page)
        for got, w in ((k_out, wk), (v_out, wv)):
            w = torch.from_numpy(w.astype(np.float32)).to(DT[out]).reshape(T, -1)
            assert torch.equal(got.cpu(), w)


def test_positions_outside_the_table_are_clamped(nv):
    T, D = 4, 64
    x = torch.randn(T, D, device="cuda")
    cos, sin = torch.rand(2, 10, 32, device="cuda")
    g = torch.full((1,), 0.002, device="cuda")
    slots = torch.arange(T, device="cuda")
    outs = []
    for pos in ([-5, 0, 9, 1000], [0, 0, 9, 9]):
        cache = nv.empty_kv_cache(1, 1, 16, D).zero_()
        q = torch.empty_like(x)
        nv.nvfp4_rope_append_kv(x, x, x, cos, sin, torch.tensor(pos, dtype=torch.int32, device="cuda"), slots, cache, g,
                                g, 16, q)
        outs.append((q.cpu(), cache.cpu()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_binding_refusals(nv):
    cuda = dict(device="cuda")
    cache = nv.empty_kv_cache(4, 2, 16, 64)
    g, x = torch.ones(2, **cuda), torch.zeros(3, 128, **cuda)
    i32, slots = torch.zeros(3, dtype=torch.int32, **cuda), torch.zeros(3, dtype=torch.int64, **cuda)
    half = torch.rand(5, 32, **cuda)
    cu = torch.arange(4, dtype=torch.int32, **cuda)

    def append(q=x, k=x, v=x, cos=half, sin=half, pos=i32, slots=slots, cache=cache, kg=g, vg=g, page=16, out=x):
        nv.nvfp4_rope_append_kv(q, k, v, cos, sin, pos, slots, cache, kg, vg, page, out)

    def gather(cache=cache, slots=slots, kg=g, vg=g, page=16, k=x, v=x):
        nv.nvfp4_kv_gather(cache, slots, kg, vg, page, k, v)

    def attend(q=x, cache=cache, table=i32[:, None], kv_len=i32, kg=g, page=16, o=x, most=10, ws=None, **kw):
        nv.nvfp4_kv_attention(q, cache, table, kv_len, kg, g, page, o, most, ws, **kw)

    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for call, bad, status in (
            (append, dict(k=x[:, :64]), inv), (append, dict(v=x[:2]), inv), (append, dict(v=x.bfloat16()), uns),
            (append, dict(k=x.half(), v=x.half()), uns), (append, dict(q=x.t()), inv), (append, dict(q=None), inv),
            (append, dict(out=None), inv), (append, dict(q=x[:, :100], out=x[:, :100]), inv), (append, dict(out=x.bfloat16()), uns),
            (append, dict(pos=slots), inv), (append, dict(slots=i32), inv), (append, dict(slots=slots[:2]), inv),
            (append, dict(cos=None), inv), (append, dict(cos=half.double()), inv), (append, dict(sin=half[:4]), inv),
            (append, dict(cos=torch.rand(5, 64, **cuda), sin=torch.rand(5, 64, **cuda)), inv), (append, dict(kg=g[:1]), inv),
            (append, dict(vg=g.double()), inv), (append, dict(page=32), inv), (append, dict(page=0), inv),
            (append, dict(cache=cache[:, :-1]), inv), (append, dict(cache=cache.view(-1)), inv), (append, dict(slots=None), inv),
            (append, dict(slots=[1, 2, 3]), inv), (append, dict(page="16"), inv), (append, dict(k=x.cpu()), inv),
            (gather, dict(k=x[:, :64]), inv), (gather, dict(v=x.bfloat16()), uns), (gather, dict(slots=slots[:1]), inv),
            (gather, dict(k=x[:2], v=x[:2]), inv), (gather, dict(cache=cache.float()), inv),
            (attend, dict(o=x[:2]), inv), (attend, dict(o=x.bfloat16()), uns), (attend, dict(table=slots[:, None]), uns),
            (attend, dict(table=i32), inv), (attend, dict(kv_len=i32[:2]), inv), (attend, dict(kv_len=slots), inv),
            (attend, dict(table=i32[:2, None], kv_len=i32[:2]), inv), (attend, dict(cu_q=i32), inv),
            (attend, dict(cu_q=cu.long()), inv), (attend, dict(lse=torch.zeros(3, 3, **cuda)), inv),
            (attend, dict(lse=torch.zeros(3, 2, dtype=torch.float64, **cuda)), inv), (attend, dict(scale=float("nan")), inv),
            (attend, dict(scale="big"), inv), (attend, dict(window=-1), inv), (attend, dict(window=1 << 40), inv),
            (attend, dict(most=-1), inv), (attend, dict(max_q_len=0), inv), (attend, dict(most=100000), inv),
            (attend, dict(most=100000, ws=torch.empty(16, dtype=torch.uint8, **cuda)), inv)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call(**bad)
        assert e.value.status == status, (bad, str(e.value))


# ----------------------------------------------------------------------------- attention

class Problem:
    """A cache holding sequences of the given lengths in shuffled pages, with bytes that
    decode to NaN wherever no token is, and table entries out of range past each end."""

    def __init__(self, nv, kv, m, Hq, Hkv, D, page, dtype, seed, q_gain=1.0, extra_pages=2):
        rng = np.random.default_rng(seed)
        self.kv, self.m, self.Hq, self.Hkv, self.D, self.page, self.dtype = kv, m, Hq, Hkv, D, page, dtype
        self.kg, self.vg = _gscales(rng, Hkv)
        need = [-(-n // page) for n in kv]
        n_pages = sum(need) + extra_pages
        order = rng.permutation(n_pages)
        self.width = max(need + [1]) + 1
        table = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, n_pages], (len(kv), self.width))
        at, slots = 0, []
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            slots += [int(table[b, t // page]) * page + t % page for t in range(kv[b])]
            at += n
        total = sum(kv)
        self.slots = np.array(slots, dtype=np.int64)
        x = _draw(rng, (2, total, Hkv, D), "f32")
        self.cache = nv.empty_kv_cache(n_pages, Hkv, page, D)
        self.cache.fill_(0x7F)                                # an E4M3 NaN in every scale byte
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
        self.dkg, self.dvg = dev(self.kg), dev(self.vg)
        if total:
            k, v = dev(x[0].reshape(total, -1)), dev(x[1].reshape(total, -1))
            nv.nvfp4_rope_append_kv(None, k, v, None, None, torch.zeros(total, dtype=torch.int32, device="cuda"),
                                    dev(self.slots), self.cache, self.dkg, self.dvg, page, None)
        self.k, self.v = KV.gather(self.cache.cpu().numpy().reshape(-1), self.slots, Hkv, D, self.kg, self.vg, page) \
            if total else np.zeros((2, 0, Hkv, D))
        self.T = sum(m)
        self.q = torch.from_numpy(_draw(rng, (self.T, Hq, D), dtype) * np.float32(q_gain)).to(DT[dtype])
        self.table, self.kv_len = dev(table.astype(np.int32)), dev(np.array(kv, dtype=np.int32))
        self.cu = dev(np.concatenate([[0], np.cumsum(m)]).astype(np.int32))

    def run(self, nv, window=0, scale=None, hints=None, use_cu=True, pad=0, table=None):
        wide = torch.full((self.T, self.Hq * self.D + pad), float("nan"), dtype=DT[self.dtype], device="cuda")
        q = wide[:, :self.Hq * self.D]
        q.copy_(self.q.reshape(self.T, -1))
        o = torch.full_like(wide, 3.0)
        lse = torch.full((self.T, self.Hq), 3.0, device="cuda")
        mq, mk = hints or (max(self.m), max(self.kv))
        ws = torch.empty(nv.nvfp4_kv_attention_workspace(self.T, len(self.kv), self.Hq, self.Hkv, self.D, mq, mk, q.dtype),
                         dtype=torch.uint8, device="cuda")
        nv.nvfp4_kv_attention(q, self.cache, self.table if table is None else table, self.kv_len, self.dkg, self.dvg,
                              self.page, o[:, :self.Hq * self.D], mk, ws, cu_q=self.cu if use_cu else None, max_q_len=mq,
                              scale=scale, window=window, lse=lse)
        torch.cuda.synchronize()
        if pad:
            assert torch.all(o[:, self.Hq * self.D:] == 3.0)
        return o[:, :self.Hq * self.D].float().cpu().numpy().reshape(self.T, self.Hq, self.D).astype(np.float64), \
            lse.cpu().numpy().astype(np.float64)

    def check(self, got, window=0, scale=None, rows=None):
        """rows: query rows per sequence to check (None: all)."""
        scale = self.D ** -0.5 if scale is None else scale
        o, lse = got
        qa, ka = 0, 0
        for n, m in zip(self.kv, self.m):
            k, v = self.k[ka:ka + n], self.v[ka:ka + n]
            for i in (range(m) if rows is None else [r for r in rows if r < m]):
                if rows is None and i:
                    break
                sl = slice(0, m) if rows is None else slice(i, i + 1)
                # the rows alone, with the keys up to the last of them
                end = n if rows is None else max(0, n - m + i + 1)
                q = self.q[qa:qa + m][sl].float().numpy()
                wo, wl, w = KV.attention(q, k[:end], v[:end], scale, window)
                if rows is not None and n - m + i < 0:
                    wo, wl, w = np.zeros_like(wo), np.full_like(wl, -np.inf), np.zeros((1, self.Hq, end))
                bo, bl = KV.attention_bounds(q, k[:end], v[:end], w, scale, self.dtype)
                go, gl = o[qa:qa + m][sl], lse[qa:qa + m][sl]
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
                fin = np.isfinite(wl)
                assert np.all(np.abs(go - wo) <= bo + O.ulp(wo, self.dtype)), np.max(np.abs(go - wo))
                assert np.all(np.abs(gl - wl)[fin] <= (bl + 4 * 2.0 ** -24 * np.abs(wl))[fin])
                assert np.all(go[~fin] == 0)
            qa, ka = qa + m, ka + n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv,m,Hq,Hkv,D,page,window", [
    ([1], [1], 1, 1, 64, 16, 0),                                   # one token, one head
    ([0, 3, 17], [1, 1, 1], 4, 2, 64, 16, 0),                      # an empty sequence
    ([15, 16, 17, 63, 64, 65, 129], [1] * 7, 8, 2, 128, 16, 0),    # ends around granules, pages and steps
    ([200, 31], [1, 1], 6, 2, 256, 32, 0),
    ([300, 40, 5], [1, 1, 1], 5, 5, 128, 64, 33),                  # a window that starts inside a page
    ([100, 70], [1, 1], 20, 1, 64, 128, 0),                        # more query heads than one column block
    ([90, 20, 64], [4, 1, 7], 4, 2, 128, 16, 0),                   # several tokens each
    ([3, 50], [8, 2], 2, 1, 64, 16, 0),                            # more query tokens than keys: rows see nothing
    ([40, 100, 7], [0, 100, 7], 3, 3, 128, 32, 9),                 # a sequence without queries, whole prompts, a window
    ([150], [150], 4, 1, 256, 16, 0),
    ([120, 30], [57, 30], 7, 7, 64, 64, 1),                        # each token sees itself alone
])
def test_attention_matches_oracle(nv, dtype, kv, m, Hq, Hkv, D, page, window):
    p = Problem(nv, kv, m, Hq, Hkv, D, page, dtype, seed=sum(kv) + D)
    p.check(p.run(nv, window), window)
    if all(x == 1 for x in m):
        p.check(p.run(nv, window, use_cu=False), window)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,n,m", [
    ("bf16", 128, 8, 2, 5000, 1), ("f32", 64, 4, 4, 3333, 1), ("bf16", 256, 6, 1, 2600, 2), ("f32", 256, 2, 1, 2111, 3),
    ("bf16", 64, 9, 3, 4097, 5)])
def test_long_keys_are_split_and_joined(nv, dtype, D, Hq, Hkv, n, m):
    p = Problem(nv, [n, 130], [m, m], Hq, Hkv, D, 16, dtype, seed=n)
    assert nv.nvfp4_kv_attention_workspace(p.T, 2, Hq, Hkv, D, m, n, p.q.dtype) > 0
    p.check(p.run(nv))
    p.check(p.run(nv, window=1500), window=1500)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,n,m", [
    ("bf16", 128, 8, 2, 1500, 1500), ("bf16", 256, 4, 1, 900, 300), ("bf16", 64, 6, 6, 700, 650),
    ("bf16", 128, 5, 1, 2000, 333), ("f32", 128, 4, 2, 600, 500)])
@pytest.mark.parametrize("window", [0, 257])
def test_long_queries(nv, dtype, D, Hq, Hkv, n, m, window):
    # ragged beside a short and an empty sequence; a sample of rows against the oracle
    p = Problem(nv, [n, 65, 0], [m, 33, 2], Hq, Hkv, D, 32, dtype, seed=n + m)
    rows = sorted({0, 1, 15, 16, 31, 32, 63, 64, 127, 128, 255, 256, 257, m // 2, m - 2, m - 1})
    p.check(p.run(nv, window), window, rows=rows)


@pytest.mark.parametrize("D,Hq,Hkv,kv,m", [
    (64, 56, 56, [400, 65, 0], [300, 65, 7]), (128, 64, 32, [333, 150, 1], [140, 150, 1]),
    (256, 56, 28, [290, 129, 40], [150, 3, 0]), (128, 4, 2, [300] + [5] * 89, [129] + [1] * 89)])
@pytest.mark.parametrize("window", [0, 70])
def test_prompts_of_many_items(nv, D, Hq, Hkv, kv, m, window):
    # more (sequence, head, 256 query columns) than are cut along the keys
    p = Problem(nv, kv, m, Hq, Hkv, D, 16, "bf16", seed=D + len(kv))
    rows = sorted({0, 1, 31, 32, 127, 128, m[0] - 1, m[0], m[0] + 1})
    p.check(p.run(nv, window), window, rows=rows)


@pytest.mark.parametrize("D,Hq,Hkv,kv,m", [
    (64, 56, 56, [400, 65, 0], [300, 65, 7]), (128, 64, 32, [1333, 150, 1], [140, 150, 1]),
    (256, 56, 28, [290, 129, 40], [150, 3, 0])])
def test_prompts_of_unlike_lengths(nv, D, Hq, Hkv, kv, m):
    # as many items, cut all the same: new tokens of unlike numbers under a bound of many keys
    p = Problem(nv, kv, m, Hq, Hkv, D, 16, "bf16", seed=D + 1)
    assert nv.nvfp4_kv_attention_workspace(p.T, 3, Hq, Hkv, D, max(m), 20000, p.q.dtype) > 0
    assert nv.nvfp4_kv_attention_workspace(p.T, 3, Hq, Hkv, D, max(m), max(kv), p.q.dtype) == 0
    rows = sorted({0, 1, 31, 32, 127, 128, m[0] - 1, m[1] - 1})
    p.check(p.run(nv, hints=(max(m), 20000)), rows=rows)
    p.check(p.run(nv, 70, hints=(max(m), 20000)), 70, rows=rows)


def test_prompt_hints_that_are_too_low(nv):
    # the tiles of columns that were not planned for, whole and cut along the keys
    for kv, m, Hq, Hkv, hint in (([900, 4, 300], [600, 1, 9], 4, 1, 64), ([300, 290], [280, 290], 192, 96, 128)):
        p = Problem(nv, kv, m, Hq, Hkv, 64, 16, "bf16", seed=8)
        p.check(p.run(nv, hints=(hint, 10)), rows=[0, 1, 63, 64, 129, 255, 256, 279, 280, 281])


def test_hints_that_are_too_low(nv):
    p = Problem(nv, [900, 4, 300], [40, 1, 9], 4, 2, 128, 16, "bf16", seed=5)
    for hints in ((1, 1), (3, 500), (1, 5000), (40, 0)):
        p.check(p.run(nv, hints=hints))


def test_strided_rows_tables_and_scale(nv):
    p = Problem(nv, [77, 40], [1, 1], 4, 2, 128, 32, "bf16", seed=6)
    p.check(p.run(nv, scale=0.3, pad=24), scale=0.3)
    wide = torch.full((2, 2 * p.width + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :p.width] = p.table
    p.check(p.run(nv, table=wide[:, :p.width]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gain", [0.0, 1e-35, 1e-6, 30.0])
def test_query_magnitudes(nv, dtype, gain):
    # zero and tiny queries average the values, large ones single out a key
    p = Problem(nv, [130, 700], [2, 1], 4, 2, 128, 16, dtype, seed=7, q_gain=gain)
    p.check(p.run(nv))


@pytest.mark.parametrize("dtype,D,Hq,Hkv,kv,m,hint", [
    ("bf16", 64, 6, 2, [70, 33], [1, 1], 70),                      # whole items
    ("f32", 128, 4, 2, [3000, 40], [2, 1], 3000),                  # joined pieces, many and few
    ("bf16", 128, 8, 4, [2500] * 6, [3] * 6, 2500),
    ("bf16", 128, 4, 1, [400, 100], [200, 70], 400),               # prompts, joined pieces
    ("bf16", 64, 56, 56, [300, 65, 7], [290, 65, 7], 300)])        # and whole items
def test_a_nan_stays_in_its_row(nv, dtype, D, Hq, Hkv, kv, m, hint):
    p = Problem(nv, kv, m, Hq, Hkv, D, 16, dtype, seed=11)
    clean = p.run(nv, hints=(max(m), hint))
    at, q = (m[0] // 2, Hq - 1), p.q
    p.q = q.clone()
    p.q[at[0], at[1], 5] = float("nan")
    o, lse = p.run(nv, hints=(max(m), hint))
    p.q = q
    assert np.all(np.isnan(o[at])) and np.isnan(lse[at])
    o[at], lse[at] = clean[0][at], clean[1][at]
    p.check((o, lse), rows=sorted({0, m[0] // 2, m[0] - 1, max(0, m[0] // 2 - 1)}))


def test_rising_scores_move_the_reference(nv):
    # keys that grow along the sequence: the maximum keeps rising, tile after tile
    D, n = 64, 1024
    g = torch.full((1,), 40.0 / 2688, device="cuda")
    ramp = torch.linspace(0.01, 6.0, n, device="cuda")[:, None].expand(n, D).contiguous()
    v = torch.randn(n, D, device="cuda")
    cache = nv.empty_kv_cache(n // 16, 1, 16, D)
    slots = torch.arange(n, device="cuda")
    nv.nvfp4_rope_append_kv(None, ramp, v, None, None, torch.zeros(n, dtype=torch.int32, device="cuda"), slots, cache, g,
                            g, 16, None)
    kk, vv = KV.gather(cache.cpu().numpy().reshape(-1), slots.cpu().numpy(), 1, D, g.cpu().numpy(), g.cpu().numpy(), 16)
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    for sign in (1.0, -1.0):
        q = torch.full((1, D), 2.0 * sign, device="cuda")
        o = torch.empty_like(q)
        nv.nvfp4_kv_attention(q, cache, table, kv_len, g, g, 16, o, 1)
        qn = q.cpu().numpy().reshape(1, 1, D)
        wo, _, w = KV.attention(qn, kk, vv, D ** -0.5)
        bo, _ = KV.attention_bounds(qn, kk, vv, w, D ** -0.5, "f32")
        assert np.all(np.abs(o.cpu().numpy().reshape(1, 1, D) - wo) <= bo + O.ulp(wo, "f32"))


def test_cache_beyond_4_gib(nv):
    # a page whose byte offset passes 2^32, and slots behind it
    H, D, page = 8, 128, 256
    n_pages = (5 << 30) // nv.nvfp4_kv_page_bytes(H, page, D)
    cache = nv.empty_kv_cache(n_pages, H, page, D)
    rng = np.random.default_rng(8)
    T = 300
    x = _draw(rng, (2, T, H, D), "f32")
    kg, vg = _gscales(rng, H)
    pages = [n_pages - 1, 3]
    slots = np.array([pages[t // page] * page + t % page for t in range(T)], dtype=np.int64)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()       # noqa: E731
    nv.nvfp4_rope_append_kv(None, dev(x[0].reshape(T, -1)), dev(x[1].reshape(T, -1)), None, None,
                            torch.zeros(T, dtype=torch.int32, device="cuda"), dev(slots), cache, dev(kg), dev(vg), page, None)
    k_out, v_out = torch.empty(2, T, H * D, device="cuda")
    nv.nvfp4_kv_gather(cache, dev(slots), dev(kg), dev(vg), page, k_out, v_out)
    want = []
    for a, g in ((x[0], kg), (x[1], vg)):
        c, s = KV.quantize_heads(a, g)
        want.append(O.dequantize_rows(c.reshape(T * H, -1), s.reshape(T * H, -1), np.tile(g, T)).reshape(T, H, D))
    assert np.array_equal(k_out.cpu().numpy().reshape(T, H, D), want[0].astype(np.float32))
    assert np.array_equal(v_out.cpu().numpy().reshape(T, H, D), want[1].astype(np.float32))
    q = _draw(rng, (1, H, D), "f32")
    o = torch.empty(1, H * D, device="cuda")
    ws = torch.empty(nv.nvfp4_kv_attention_workspace(1, 1, H, H, D, 1, T), dtype=torch.uint8, device="cuda")
    nv.nvfp4_kv_attention(dev(q.reshape(1, -1)), cache, dev(np.array([pages], dtype=np.int32)),
                          dev(np.array([T], dtype=np.int32)), dev(kg), dev(vg), page, o, T, ws)
    wo, _, w = KV.attention(q, want[0], want[1], D ** -0.5)
    bo, _ = KV.attention_bounds(q, want[0], want[1], w, D ** -0.5, "f32")
    assert np.all(np.abs(o.cpu().numpy().reshape(1, H, D) - wo) <= bo + O.ulp(wo, "f32"))


def test_results_repeat_and_follow_the_stream(nv):
    p = Problem(nv, [3000, 100], [1, 1], 8, 2, 128, 16, "bf16", seed=9)
    first = p.run(nv)
    again = p.run(nv)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = p.run(nv)
    assert np.array_equal(first[0], other[0])


def test_graph_replays(nv):
    # append and attend in a captured graph: every replay against the eager result
    H, D, page, n_pages = 2, 128, 16, 80
    rng = torch.Generator(device="cuda")
    rng.manual_seed(1)
    x = torch.randn(1, 8 * D, generator=rng, device="cuda")
    q_out, o = torch.empty(1, 4 * D, device="cuda"), torch.empty(1, 4 * D, device="cuda")
    g = torch.full((H,), 0.002, device="cuda")
    cos, sin = torch.rand(2, 2000, D // 2, generator=rng, device="cuda")
    pos, slots = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    kv_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = nv.empty_kv_cache(n_pages, H, page, D).zero_()
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    need = nv.nvfp4_kv_attention_workspace(1, 1, 4, H, D, 1, n_pages * page)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        q, k, v = x.split([4 * D, H * D, H * D], 1)
        nv.nvfp4_rope_append_kv(q, k, v, cos, sin, pos, slots, cache, g, g, page, q_out)
        nv.nvfp4_kv_attention(q_out, cache, table, kv_len, g, g, page, o, n_pages * page, ws)

    def at(t):
        pos.fill_(t)
        slots.fill_(t)
        kv_len.fill_(t + 1)
        x.copy_(torch.randn(1, 8 * D, generator=torch.Generator(device="cuda").manual_seed(t), device="cuda"))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    eager = []
    for t in range(0, 600, 7):
        at(t)
        step()
        eager.append((o.clone(), q_out.clone()))
    cache.zero_()
    for i, t in enumerate(range(0, 600, 7)):
        at(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[i][0]) and torch.equal(q_out, eager[i][1]), t
