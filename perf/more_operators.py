"""Timed cases of drafted trees over the paged NVFP4 key/value cache and of eviction from
it: attention of a tree of drafted tokens, moving the accepted path's rows to their places,
the attention weight that cached tokens receive, and evicting the tokens of least weight.
`run` computes them with the framework's kernels where `own` is true, and in plain fp32
torch operations otherwise; `exact` gives the results in 64 bits.

Cache layout: pages [n_pages][Hkv][page/16] of granules of 16 tokens; a granule holds, for
head dimension D,
    K codes   [16 tokens][D/2]                    two E2M1 codes a byte, low nibble first
    K scales  [16 tokens][D/16]                   E4M3
    V codes   [4 quads][16][4 tokens][D/32]       the D/2 code bytes of a token in 16 parts
    V scales  [4 quads][D/16][4 tokens]           E4M3
A value is e2m1 * s * g[head], g one fp32 scale per kv head for keys and one for values.
Weights of cached tokens are fp32 [n_pages][Hkv][page].
"""

import math
import random

import torch

own = False

DEV = "cuda"
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)          # between consecutive magnitudes


# ------------------------------------------------------------------------ the cases

def _tree(name, dtype, batch, kv_min, kv_max, q_min, q_max, hq, hkv, d, page, window=0):
    c = {"op": "tree", "dtype": dtype, "batch": batch, "kv_min": kv_min, "kv_max": kv_max, "q_min": q_min,
         "q_max": q_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window}
    return dict(c, name=name) if name else c


def _accept(name, batch, kv_max, q_min, q_max, path, hkv, d, page):
    c = {"op": "accept", "batch": batch, "kv_min": q_max, "kv_max": kv_max, "q_min": q_min, "q_max": q_max, "path": path,
         "hkv": hkv, "d": d, "page": page}
    return dict(c, name=name) if name else c


def _weights(name, dtype, batch, kv_min, kv_max, q_min, q_max, hq, hkv, d, page, window=0, decay=1.0):
    c = {"op": "weights", "dtype": dtype, "batch": batch, "kv_min": kv_min, "kv_max": kv_max, "q_min": q_min,
         "q_max": q_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window, "decay": decay}
    return dict(c, name=name) if name else c


def _evict(name, batch, kv_min, kv_max, budget, first, last, hkv, d, page):
    c = {"op": "evict", "batch": batch, "kv_min": kv_min, "kv_max": kv_max, "budget": budget, "first": first,
         "last": last, "hkv": hkv, "d": d, "page": page}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one chat, a small tree: latency counts
        _tree("tree_short", "bf16", 1, 300, 300, 8, 8, 32, 8, 128, 64),
        # 16 sequences being served, trees of up to 60 nodes
        _tree("tree_16x60", "bf16", 16, 1000, 8192, 25, 60, 32, 8, 128, 64),
        # long documents, few sequences: the key axis has to be split
        _tree("tree_long", "bf16", 2, 100000, 131072, 13, 32, 32, 8, 128, 128),
        # fp32 with a sliding window, odd head counts, small pages
        _tree("tree_f32_window", "f32", 5, 20, 3001, 1, 17, 15, 5, 64, 16, 700),
        # wide heads, large trees, many query heads per key head
        _tree("tree_d256", "bf16", 8, 9000, 16384, 64, 128, 16, 2, 256, 64),
        # one chat accepts a part of its tree
        _accept("accept_1", 1, 300, 8, 8, 4, 8, 128, 64),
        # a batch of large trees
        _accept("accept_64_d256", 64, 2000, 40, 64, 9, 4, 256, 32),
        # a decode step of a full batch, older weights fading
        _weights("weights_32x8k", "bf16", 32, 1024, 8192, 1, 1, 32, 8, 128, 64, 0, 0.97),
        # fp32 chunks with a window, odd head counts, small pages
        _weights("weights_f32_chunk", "f32", 3, 700, 2049, 37, 300, 15, 5, 64, 16, 1000),
        # the weights of an 8K prompt
        _weights("weights_prompt_8k", "bf16", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 64),
        # a batch that goes over its budget every hundred tokens or so; some sequences are not there yet
        _evict("evict_step", 32, 4060, 4201, 4096, 4, 256, 8, 128, 64),
        # long documents cut to an eighth after their prompt
        _evict("evict_prompt", 2, 100001, 131072, 16384, 16, 1000, 8, 128, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        d = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 5, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
        page = rng.choice([16, 32, 64, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        kind = rng.choice(["tree", "tree", "accept", "weights", "weights", "prompt", "evict", "evict"])
        window = rng.choice([0, 0, _log_int(rng, 100, 5000)])
        if kind == "tree":
            batch, kv, q = _log_int(rng, 1, 48), _log_int(rng, 150, 131072), _log_int(rng, 2, 128)
            q = min(q, kv)
            c = _tree(None, dtype, batch, max(q, int(kv * rng.random())), kv, max(1, int(q * rng.random())), q, hq, hkv, d,
                      page, window)
            cost = batch * max(kv * hkv * d / (2 * 131072 * 8 * 128), q * kv * hq * d / (8 * 128 * 16384 * 16 * 256))
        elif kind == "accept":
            batch, q = _log_int(rng, 1, 64), _log_int(rng, 2, 128)
            c = _accept(None, batch, q + _log_int(rng, 1, 1900), max(1, int(q * rng.random())), q, rng.randint(1, min(q, 17)),
                        hkv, d, page)
            cost = batch * c["kv_max"] * hkv * d / (64 * 2000 * 8 * 256)
        elif kind == "evict":
            batch, kv = _log_int(rng, 1, 48), _log_int(rng, 200, 131072)
            budget = rng.choice([_log_int(rng, 64, kv - 1), kv - _log_int(rng, 1, 128)])
            first, last = rng.choice([0, 1, 4, 16]), rng.choice([0, 8, 64, 300, 1024])
            first, last = min(first, budget // 4), min(last, budget // 2)
            c = _evict(None, batch, int(kv * (1 - 0.5 * rng.random())), kv, budget, first, last, hkv, d, page)
            cost = batch * kv * hkv * d / (2 * 131072 * 8 * 128)
        else:
            if kind == "weights":
                batch, kv, q = _log_int(rng, 1, 48), _log_int(rng, 50, 131072), rng.choice([1, 1, rng.randint(2, 64)])
            else:
                batch, kv = rng.randint(1, 4), _log_int(rng, 64, 8192)
                q = rng.randint(kv // 4, kv)
            c = _weights(None, dtype, batch, int(kv * rng.random()), kv, max(1, int(q * rng.random())), q, hq, hkv, d, page,
                         window, rng.choice([1.0, 1.0, 0.9]))
            cost = batch * max(kv * hkv * d / (2 * 131072 * 8 * 128), q * kv * hq * d / (8192 * 8192 * 32 * 128),
                               q * kv * hq / (8192 * 8192 * 32))
        if cost <= 1:
            return c


def _spread(lo, hi, n, step):
    """n whole numbers spread over [lo, hi], the last of them hi."""
    v = [lo + int((hi - lo) * ((i * step) % 1.0) + 0.5) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(case):
    kv = _spread(case["kv_min"], case["kv_max"], case["batch"], 0.6180339887)
    q = _spread(case.get("q_min", 0), case.get("q_max", 0), case["batch"], 0.7548776662)
    return kv, q


def work(case):
    kv, q = _lengths(case)
    d, hkv = case["d"], case["hkv"]
    row = d * 9 // 8                                         # bytes of a token's key and value, one head
    if case["op"] == "accept":
        moved = sum(min(case["path"], m) for m in q) * hkv
        return {"bytes": 2 * moved * row + 4 * (moved // hkv + 2 * case["batch"]), "flops": 0.0}
    if case["op"] == "evict":
        over = [n for n in kv if n > case["budget"]]
        spare = case["budget"] - case["first"] - case["last"]
        # of the heaviest tokens, the share that stands behind the places
        moved = sum(case["last"] + spare * (n - case["budget"]) / (n - case["first"] - case["last"]) for n in over) * hkv
        places = sum(min(n, case["budget"]) for n in kv)
        return {"bytes": 4 * hkv * sum(kv) + 2 * moved * row + 8 * hkv * places, "flops": 0.0}
    hq = case["hq"]
    size = 2 if case["dtype"] == "bf16" else 4
    window = case["window"] or (1 << 40)
    keys = pairs = 0
    for n, m in zip(kv, q):
        if case["op"] == "tree":                             # a path is taken to be a quarter of the nodes
            path = (m + 3) // 4
            keys += min(n, m + window)
            pairs += m * min(n - m + path, window)
        else:
            first = max(0, n - m)
            keys += n - max(0, min(n, first - window + 1))
            pairs += sum(min(p + 1, window) for p in range(first, n))
    rows = sum(q)
    if case["op"] == "tree":
        return {"bytes": keys * hkv * row + rows * (hq * (2 * d * size + 4) + 8 * -(-case["q_max"] // 64)),
                "flops": 4.0 * d * hq * pairs}
    return {"bytes": keys * hkv * (row // 2) + 8 * hkv * (keys if case["decay"] == 1 else sum(kv)) + rows * hq * (d * size + 4),
            "flops": 2.0 * d * hq * pairs}


# ------------------------------------------------------------------------ the inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tables():
    """The formats' values on the device, kept by the program: the two values of each byte
    of codes, the value of each E4M3 byte."""
    mags = torch.tensor(MAGS, device=DEV)
    signed = torch.cat([mags, -mags])
    byte = torch.arange(256, device=DEV)
    e, m = (byte >> 3) & 15, (byte & 7).float()
    v = torch.where(e > 0, torch.ldexp(1.0 + m / 8, e - 7), m / 512)
    return {"pairs": torch.stack([signed[byte & 15], signed[byte >> 4]], -1), "e4m3": torch.where(byte >= 128, -v, v)}


def _quantize(x, g):
    """NVFP4 of the last dimension of x (fp32) under g: code bytes and scale bytes."""
    blocks = x.unflatten(-1, (-1, 16))
    scale = (blocks.abs().amax(-1) / (6 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = (scale.float() * g).clamp(min=1e-30)
    code = torch.bucketize(blocks.abs() / unit[..., None], torch.tensor(MIDS, device=DEV))
    code = (code + 8 * (blocks < 0)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _fill_pages(s, gen):
    """Pages of keys with a few large channels, and of values."""
    case = s["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    gain = torch.rand(hkv, d, generator=gen, device=DEV) + 0.5
    gain = torch.where(torch.rand(hkv, d, generator=gen, device=DEV) < 0.03, gain * 4, gain)
    some = max(1, (1 << 23) // (hkv * page * d))             # pages filled at a time
    for p in range(0, s["cache"].shape[0], some):
        n = min(some, s["cache"].shape[0] - p)
        k = torch.randn(n, page, hkv, d, generator=gen, device=DEV) * gain
        v = torch.randn(n, page, hkv, d, generator=gen, device=DEV)
        kc, ks = _quantize(k, s["k_gscale"][:, None])
        vc, vs = _quantize(v, s["v_gscale"][:, None])
        rows = lambda x: x.transpose(1, 2).reshape(n, hkv, page // 16, 16, -1)   # noqa: E731
        vc = rows(vc).unflatten(-1, (16, -1)).unflatten(3, (4, 4)).transpose(4, 5)
        vs = rows(vs).unflatten(3, (4, 4)).transpose(4, 5)
        parts = [rows(kc), rows(ks), vc, vs]
        s["cache"][p:p + n] = torch.cat([x.reshape(n, hkv, page // 16, -1) for x in parts], -1).view(n, -1)


def _draw_trees(q, seed):
    """The paths of trees of q nodes each: for each node the numbers of its ancestors and
    its own; every parent is one of the eight nodes before."""
    rng = random.Random(seed)
    trees = []
    for m in q:
        paths = [1]
        for j in range(1, m):
            paths.append(paths[rng.randrange(max(0, j - 8), j)] | 1 << j)
        trees.append(paths)
    return trees


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    d, hkv, page, batch = case["d"], case["hkv"], case["page"], case["batch"]
    kv, q = _lengths(case)
    need = [-(-n // page) for n in kv]
    n_pages, n_max = sum(need) + 1, -(-case["kv_max"] // page)
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((batch, n_max), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = {"case": case, "table": table, "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV),
         "cu_q": torch.tensor([0] + q, device=DEV).cumsum(0).to(torch.int32)}
    size = hkv * page * d * 9 // 8
    if case["op"] in ("accept", "evict"):                    # rows are moved, whatever they hold
        s["cache"] = torch.randint(0, 256, (n_pages, size), generator=gen, device=DEV, dtype=torch.uint8)
        s["kv_len_out"] = torch.empty_like(s["kv_len"])
    else:
        s["cache"] = torch.empty(n_pages, size, dtype=torch.uint8, device=DEV)
        s["tables"] = _tables()
        s["k_gscale"] = (14.0 + torch.rand(hkv, generator=gen, device=DEV)) / 2688.0
        s["v_gscale"] = (5.0 + torch.rand(hkv, generator=gen, device=DEV)) / 2688.0
        _fill_pages(s, gen)
        rows, hq = sum(q), case["hq"]
        s["q"] = (torch.randn(rows, hq * d, generator=gen, device=DEV) * 0.7).to(_dtype(case))
    if case["op"] == "tree":
        words = -(-case["q_max"] // 64)
        bits = [[(p >> 64 * w) & (1 << 64) - 1 for w in range(words)] for t in _draw_trees(q, seed) for p in t]
        s["mask"] = torch.tensor([[x - (x >> 63 << 64) for x in row] for row in bits], dtype=torch.int64, device=DEV)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
    elif case["op"] == "accept":
        # an accepted path: nodes of increasing numbers, from the root on
        paths = []
        for t in _draw_trees(q, seed):
            path = [j for j in range(len(t)) if t[-1] >> j & 1][:case["path"]]
            paths.append(path + [-1] * (case["path"] - len(path)))
        s["accepted"] = torch.tensor(paths, dtype=torch.int32, device=DEV)
        s["n_accepted"] = (s["accepted"] >= 0).sum(1).to(torch.int32)
    else:
        # what tokens have received in the steps so far: a few of them most of it, some nothing at all
        w = torch.exp(2.0 * torch.randn(n_pages, hkv, page, generator=gen, device=DEV) - 7.0)
        s["key_weights"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.04, 0.0, w)
        if case["op"] == "weights":
            s["lse"] = _plain_tops(s, *_plain_scores(s))
        else:
            s["weights_out"] = torch.zeros_like(s["key_weights"])
            s["kept"] = torch.empty(batch, hkv, case["budget"], dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------ plain forms

def _plain_granules(s):
    case = s["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    pages = s["cache"].view(-1, hkv, page // 16, 18 * d)[s["table"].clamp(min=0).long()]
    pages = pages.permute(0, 2, 1, 3, 4)                           # [B, Hkv, pages, granules, bytes]
    return pages.reshape(case["batch"], hkv, -1, 18 * d)


def _plain_look(table, x, shape):
    return table.index_select(0, x.reshape(-1).int()).view(shape)


def _plain_keys(s, pages):
    """Keys [B, Hkv, S, D] of the sequences' pages in fp32, without the global scales."""
    d, lead = s["case"]["d"], pages.shape[:3]
    k = _plain_look(s["tables"]["pairs"], pages[..., :8 * d], lead + (16, d // 16, 16))
    k = k * _plain_look(s["tables"]["e4m3"], pages[..., 8 * d:9 * d], lead + (16, d // 16, 1))
    return k.reshape(lead[:2] + (-1, d))


def _plain_values(s, pages):
    d, lead = s["case"]["d"], pages.shape[:3]
    vc = _plain_look(s["tables"]["pairs"], pages[..., 9 * d:17 * d], lead + (4, 16, 4, d // 16))
    vs = _plain_look(s["tables"]["e4m3"], pages[..., 17 * d:], lead + (4, d // 16, 4))
    v = vc.transpose(4, 5).reshape(lead + (4, 4, d // 16, 16)) * vs.transpose(4, 5)[..., None]
    return v.reshape(lead[:2] + (-1, d))


def _plain_places(s):
    """The place of each query row among [B, the most query tokens]."""
    row = torch.arange(s["q"].shape[0], device=DEV)
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu[1:], row, right=True)
    return seq * s["case"]["q_max"] + row - cu[seq]


def _plain_rows(s, x, fill=0.0):
    """Query rows x [T, ...] at their places [B, the most query tokens, ...]."""
    case = s["case"]
    y = torch.full((case["batch"] * case["q_max"],) + x.shape[1:], fill, dtype=x.dtype, device=DEV)
    y[_plain_places(s)] = x
    return y.view((case["batch"], case["q_max"]) + x.shape[1:])


def _plain_scores(s, pages=None):
    """Scores [B, Hkv, group, the most query tokens, S] in fp32, -inf where a row does not
    attend, and the keys that each row [B, the most query tokens, S] attends to."""
    case = s["case"]
    d, hq, hkv, batch, most = case["d"], case["hq"], case["hkv"], case["batch"], case["q_max"]
    k = _plain_keys(s, _plain_granules(s) if pages is None else pages)
    q = _plain_rows(s, s["q"].float()).view(batch, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(batch, hkv, -1, d), k.transpose(2, 3).contiguous())
    score *= (s["k_gscale"] / math.sqrt(d))[:, None, None]
    n, m = s["kv_len"].long()[:, None, None], (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None, None]
    t = torch.arange(k.shape[2], device=DEV)
    i = torch.arange(most, device=DEV)[:, None]
    window = case["window"] or (1 << 40)
    if case["op"] == "tree":
        words = s["mask"].shape[1]
        bit = s["mask"][:, torch.arange(64 * words, device=DEV) // 64] >> (torch.arange(64 * words, device=DEV) % 64) & 1
        upto = bit.cumsum(1)
        bit = (bit > 0) & (upto[:, -1:] - upto < window)     # the last `window` nodes of the path
        bit, length = _plain_rows(s, bit, False), _plain_rows(s, upto[:, -1:])
        node = (t - (n - m)).clamp(0, 64 * words - 1).expand(batch, most, -1)
        allowed = torch.where(t < n - m, t >= n - m + length - window, bit.gather(2, node))
    else:
        allowed = (t <= n - m + i) & (t > n - m + i - window)
    allowed = allowed & (t < n) & (i < m)
    score = score.view(batch, hkv, hq // hkv, most, -1).masked_fill_(~allowed[:, None, None], -math.inf)
    return score, allowed


def _plain_tops(s, score, allowed):
    """The log of each row's softmax denominator [T, Hq]."""
    top = score.amax(-1, keepdim=True)
    total = torch.exp_(score.sub_(torch.where(top > -math.inf, top, 0))).sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return lse.permute(0, 3, 1, 2).flatten(0, 1).flatten(1)[_plain_places(s)]


def _plain_tree(s):
    case = s["case"]
    d, hq, hkv, batch, most = case["d"], case["hq"], case["hkv"], case["batch"], case["q_max"]
    pages = _plain_granules(s)
    score, _ = _plain_scores(s, pages)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(torch.where(top > -math.inf, top, 0)))
    total = p.sum(-1, keepdim=True)
    v = _plain_values(s, pages)
    live = torch.arange(v.shape[2], device=DEV) < s["kv_len"][:, None]
    v = torch.where(live[:, None, :, None], v, 0)             # places past the end hold anything
    o = torch.matmul(p.view(batch, hkv, -1, p.shape[-1]), v) * s["v_gscale"][:, None, None]
    o = o.view(batch, hkv, hq // hkv, most, d) / torch.where(total > 0, total, 1)
    lse = (top + total.log()).squeeze(-1)
    place = _plain_places(s)
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(batch * most, hq * d)[place].to(_dtype(case)),
            "lse": lse.permute(0, 3, 1, 2).reshape(batch * most, hq)[place]}


def _plain_slots(s, t):
    """Slots of tokens t [B, ...] of each sequence."""
    page = s["case"]["page"]
    pg = (t // page).clamp(0, s["table"].shape[1] - 1)
    return s["table"].long().gather(1, pg.flatten(1)).view(pg.shape) * page + t % page


def _plain_weights(s):
    case = s["case"]
    batch, hkv, page = case["batch"], case["hkv"], case["page"]
    score, _ = _plain_scores(s)
    lse = _plain_rows(s, s["lse"]).view(batch, case["q_max"], hkv, -1).permute(0, 2, 3, 1)
    p = torch.exp_(score.sub_(torch.where(lse > -math.inf, lse, 0)[..., None]))
    got = p.sum((2, 3))                                       # [B, Hkv, S]
    n, m = s["kv_len"].long()[:, None], (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None]
    t = torch.arange(got.shape[2], device=DEV).expand(batch, -1)
    slot = _plain_slots(s, t)[:, None] // page * (hkv * page) + (t % page)[:, None]
    slot = slot + (torch.arange(hkv, device=DEV) * page)[:, None]
    flat = s["key_weights"].view(-1)
    old = torch.where((t < n - m)[:, None], flat[slot.clamp(min=0)] * case["decay"], 0)
    live = ((t < n) & (m > 0))[:, None].expand(slot.shape)
    flat[slot[live]] = (old + got)[live]
    return s["key_weights"]


def _plain_bytes(s, slot, head):
    """The places of the bytes [..., 9 D / 8] of a token's key and value in the flat cache."""
    case = s["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    base = ((slot // page * hkv + head) * (page // 16) + slot % page // 16)[..., None] * (18 * d)
    r = (slot % 16)[..., None]
    quad, e = r // 4, r % 4
    j, b, part = torch.arange(d // 2, device=DEV), torch.arange(d // 16, device=DEV), d // 32
    return torch.cat([base + r * (d // 2) + j, base + 8 * d + r * (d // 16) + b,
                      base + 9 * d + ((quad * 16 + j // part) * 4 + e) * part + j % part,
                      base + 17 * d + (quad * (d // 16) + b) * 4 + e], -1)


def _plain_move(s, old, new, live):
    """Rows old -> new (tokens [B, Hkv, moves] of each sequence) where live, all read before
    any is written."""
    head = torch.arange(s["case"]["hkv"], device=DEV)[:, None].expand(live.shape[1:])
    head = head.expand(live.shape)[live]
    flat = s["cache"].view(-1)
    rows = flat[_plain_bytes(s, _plain_slots(s, torch.where(live, old, 0))[live], head)]
    flat[_plain_bytes(s, _plain_slots(s, torch.where(live, new, 0))[live], head)] = rows


def _plain_accept(s):
    case = s["case"]
    m = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    count = torch.minimum(s["n_accepted"].long(), m)
    first = (s["kv_len"].long() - m)[:, None, None]
    i = torch.arange(case["path"], device=DEV)
    live = (i < count[:, None])[:, None].expand(-1, case["hkv"], -1)
    old = first + s["accepted"].long()[:, None].expand(live.shape)
    _plain_move(s, old, (first + i).expand(live.shape), live)
    s["kv_len_out"].copy_(first.view(-1) + count)
    return {"cache": s["cache"], "kv_len": s["kv_len_out"]}


def _plain_evict(s):
    case = s["case"]
    batch, hkv, page = case["batch"], case["hkv"], case["page"]
    budget, first, last = case["budget"], case["first"], case["last"]
    n = s["kv_len"].long()[:, None, None]
    over = n > budget
    t = torch.arange(max(case["kv_max"], budget), device=DEV).expand(batch, hkv, -1)
    head = (torch.arange(hkv, device=DEV) * page)[:, None]
    slot = _plain_slots(s, t).clamp(min=0)
    at = slot // page * (hkv * page) + head + slot % page
    w = s["key_weights"].view(-1)[at]
    # the heaviest tokens between the first and the last ones: ties to the lowest index
    rated = (t >= first) & (t < n - last)
    order = torch.where(rated, torch.nan_to_num(w, -math.inf, math.inf, -math.inf), -math.inf)
    order = torch.argsort(torch.where(rated, -order, math.inf), dim=-1, stable=True)
    # tokens that are not rated stand behind the rated ones of no weight
    behind = (~rated).gather(2, order).to(torch.int8)
    order = order.gather(2, torch.argsort(behind, dim=-1, stable=True))
    rank = torch.empty_like(order).scatter_(2, order, t)
    stays = rated & (rank < budget - first - last)
    # those that stand past the places of the heaviest fill the free ones
    moves = stays & (t >= budget - last)
    free = rated & ~stays & (t < budget - last)
    most = max(1, min(budget - first - last, case["kv_max"] - budget))
    i = torch.arange(most, device=DEV).expand(batch, hkv, -1)

    def places(which):
        at = torch.where(which, which.cumsum(-1) - 1, most)
        return torch.zeros(batch, hkv, most + 1, dtype=torch.int64, device=DEV).scatter_(2, at.clamp(max=most), t)[..., :-1]

    count = moves.sum(-1, keepdim=True)
    old, new = places(moves), places(free)
    j = torch.arange(last, device=DEV).expand(batch, hkv, -1)
    old, new = torch.cat([old, n - last + j], -1), torch.cat([new, budget - last + j], -1)
    live = torch.cat([(i < count) & over, over.expand(j.shape)], -1)
    _plain_move(s, old, new, live)
    place = torch.arange(budget + 1, device=DEV).expand(batch, hkv, -1)
    kept = torch.where(place < n, place, -1).scatter(2, torch.where(live, new, budget), torch.where(live, old, -1))
    s["kept"].copy_(kept[..., :-1])
    kept = kept[..., :-1]
    live = kept >= 0
    s["weights_out"].view(-1)[at[..., :budget][live]] = w.gather(2, kept.clamp(min=0))[live]
    s["kv_len_out"].copy_(s["kv_len"].clamp(max=budget))
    return {"cache": s["cache"], "key_weights": s["weights_out"], "kept": s["kept"], "kv_len": s["kv_len_out"]}


# ------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        plain = {"tree": _plain_tree, "accept": _plain_accept, "weights": _plain_weights, "evict": _plain_evict}
        return plain[case["op"]](s)
    import nvfp4_w4a4_quantized_amd as nv
    hkv, page = case["hkv"], case["page"]
    if case["op"] == "accept":
        nv.nvfp4_kv_accept(s["cache"], s["table"], s["kv_len"], s["cu_q"], s["accepted"], s["n_accepted"], hkv, page,
                           s["kv_len_out"])
        return {"cache": s["cache"], "kv_len": s["kv_len_out"]}
    if case["op"] == "evict":
        if "workspace" not in s:                             # kept by the program between its calls
            need = nv.nvfp4_kv_evict_workspace(case["batch"], hkv, case["budget"], case["kv_max"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        nv.nvfp4_kv_evict(s["cache"], s["key_weights"], s["table"], s["kv_len"], page, case["budget"], s["kv_len_out"],
                          case["kv_max"], s["workspace"], keep_first=case["first"], keep_last=case["last"],
                          weights_out=s["weights_out"], kept=s["kept"])
        return {"cache": s["cache"], "key_weights": s["weights_out"], "kept": s["kept"], "kv_len": s["kv_len_out"]}
    cu_q = None if case["q_max"] == 1 else s["cu_q"]
    if case["op"] == "weights":
        nv.nvfp4_kv_attention_weights(s["q"], s["cache"], s["table"], s["kv_len"], s["k_gscale"], page, s["lse"],
                                      s["key_weights"], case["kv_max"], cu_q=cu_q, max_q_len=case["q_max"],
                                      window=case["window"], decay=case["decay"])
        return s["key_weights"]
    if "workspace" not in s:
        need = nv.nvfp4_kv_attention_workspace(s["q"].shape[0], case["batch"], case["hq"], hkv, case["d"], case["q_max"],
                                               case["kv_max"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_tree_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["k_gscale"], s["v_gscale"], page, s["o"],
                               case["kv_max"], s["mask"], s["workspace"], cu_q=cu_q, max_q_len=case["q_max"],
                               window=case["window"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------------ in 64 bits

def _exact_scale(byte):
    byte = byte.to(torch.float64)
    sign, byte = torch.where(byte >= 128, -1.0, 1.0), byte % 128
    e, m = torch.floor(byte / 8), byte % 8
    return sign * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(torch.full_like(e, 2.0), e - 10))


def _exact_code(nibble):
    nibble = nibble.to(torch.float64)
    sign, c = torch.where(nibble >= 8, -1.0, 1.0), nibble % 8
    e, m = torch.floor(c / 2), c % 2
    return sign * torch.where(e == 0, m * 0.5, (2 + m) * torch.pow(torch.full_like(e, 2.0), e - 2))


def _exact_rows(granules, d, n, g, values):
    """The first n keys or values [n, D] held by granules [G, 18 D]."""
    parts = d // 16
    nib = lambda x: torch.stack([x % 16, x // 16], -1).flatten(-2)   # noqa: E731
    if not values:
        x = _exact_code(nib(granules[:, :8 * d])).view(-1, 16, parts, 16)
        x = x * _exact_scale(granules[:, 8 * d:9 * d]).view(-1, 16, parts, 1)
    else:
        x = _exact_code(nib(granules[:, 9 * d:17 * d])).view(-1, 4, 16, 4, parts).permute(0, 1, 3, 2, 4)
        x = x.reshape(-1, 16, parts, 16)
        x = x * _exact_scale(granules[:, 17 * d:]).view(-1, 4, parts, 4).permute(0, 1, 3, 2).reshape(-1, 16, parts, 1)
    return x.reshape(-1, d)[:n] * g.double()


def _exact_evicted(w, n, case):
    """The tokens that a head of n tokens of weights w [n] keeps, in their new places."""
    budget, first, last = case["budget"], case["first"], case["last"]
    if n <= budget:
        return list(range(n))
    heavy = sorted(range(first, n - last), key=lambda t: (-w[t], t))[:budget - first - last]
    further = sorted(t for t in heavy if t >= budget - last)
    near = {t for t in heavy if t < budget - last}
    kept = list(range(first))
    for place in range(first, budget - last):
        kept.append(place if place in near else further.pop(0))
    return kept + list(range(n - last, n))


def exact(case, seed):
    if case["op"] == "accept":
        return None                                          # bytes moved, nothing computed
    s = prepare(case, seed)
    hkv, page = case["hkv"], case["page"]
    kv, q = _lengths(case)
    if case["op"] == "evict":
        old = s["key_weights"].cpu().double()
        new = torch.zeros_like(old)
        for n, table in zip(kv, s["table"].cpu().long()):
            at, place = table[torch.arange(n) // page], torch.arange(n) % page
            for h in range(hkv):
                w = old[at, h, place]
                kept = torch.tensor(_exact_evicted(w.tolist(), n, case))
                new[at[:len(kept)], h, place[:len(kept)]] = w[kept]
        return {"cache": None, "key_weights": new.to(DEV), "kept": None, "kv_len": None}
    d, hq = case["d"], case["hq"]
    group, rows = hq // hkv, s["q"].shape[0]
    o = torch.zeros(rows, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["key_weights"].double() if case["op"] == "weights" else None
    trees = _draw_trees(q, seed) if case["op"] == "tree" else [[]] * len(kv)
    start = 0
    for n, m, table, tree in zip(kv, q, s["table"].long(), trees):
        pages = s["cache"].view(-1, hkv, page // 16, 18 * d)[table[:-(-n // page)]]
        t = torch.arange(n, device=DEV)
        where, window = table[t // page], case["window"] or (1 << 40)
        for h in range(hkv if n else 0):
            k = _exact_rows(pages[:, h].reshape(-1, 18 * d), d, n, s["k_gscale"][h], False)
            if weights is None:
                v = _exact_rows(pages[:, h].reshape(-1, 18 * d), d, n, s["v_gscale"][h], True)
            else:
                sums = torch.where(t < n - m, case["decay"] * weights[where, h, t % page], 0.0)
            heads = slice(h * group, (h + 1) * group)
            step = max(1, min(1024, (1 << 28) // (n * group)))
            for i in range(0, m, step):
                mm = min(step, m - i)
                at = slice(start + i, start + i + mm)
                x = s["q"][at].double().view(mm, hq, d)[:, heads].reshape(mm * group, d)
                score = (x @ k.t() / math.sqrt(d)).view(mm, group, n)
                if weights is None:
                    sees = torch.zeros(mm, n, dtype=torch.bool, device=DEV)
                    for r in range(mm):
                        path = [j for j in range(m) if tree[i + r] >> j & 1]
                        sees[r, max(0, n - m - max(0, window - len(path))):n - m] = True
                        sees[r, torch.tensor([n - m + j for j in path[-window:]], device=DEV)] = True
                else:
                    pos = n - m + i + torch.arange(mm, device=DEV)[:, None]
                    sees = (t <= pos) & (t > pos - window)
                score = score.masked_fill(~sees[:, None], -math.inf)
                if weights is None:
                    weight = torch.softmax(score, -1).nan_to_num(0.0)
                    o[at, heads] = (weight.reshape(mm * group, n) @ v).view(mm, group, d)
                    lse[at, heads] = torch.logsumexp(score, -1)
                else:
                    sums += torch.exp(score - s["lse"][at, heads].double()[..., None]).nan_to_num(0.0).sum((0, 1))
            if weights is not None and m:
                weights[where, h, t % page] = sums
        start += m
    return {"o": o.reshape(rows, -1), "lse": lse} if weights is None else weights
