"""Timed cases of the paged NVFP4 key/value cache: rotating, quantizing and appending
keys and values (with the appended rows read back as values), and attention over the
cache.  `run` computes them with the framework's kernels where `own` is true, and in
plain fp32 torch operations otherwise; `exact` gives the results in 64 bits.

Cache layout (both forms read and write the same bytes): pages [n_pages][Hkv][page/16]
of granules of 16 tokens; a granule holds, for head dimension D,
    K codes   [16 tokens][D/2]                    two E2M1 codes a byte, low nibble first
    K scales  [16 tokens][D/16]                   E4M3
    V codes   [4 quads][16][4 tokens][D/32]       the D/2 code bytes of a token in 16 parts
    V scales  [4 quads][D/16][4 tokens]           E4M3
A value is e2m1 * s * g[head], g one fp32 scale per kv head for keys and one for values.
"""

import math
import random

import torch

own = False

DEV = "cuda"
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)          # between consecutive magnitudes
TIE_UP = (False, True, False, True, False, True, False)  # a tie goes to the even code
THETA = 10000.0


# ------------------------------------------------------------------------ the cases

def _append(name, dtype, tokens, hq, hkv, d, page, rot, interleaved=False, skipped=0):
    c = {"op": "append", "dtype": dtype, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "page": page, "rot": rot,
         "interleaved": interleaved, "skipped": skipped}
    return dict(c, name=name) if name else c


def _attention(name, dtype, batch, kv_min, kv_max, q_min, q_max, hq, hkv, d, page, window=0):
    c = {"op": "attention", "dtype": dtype, "batch": batch, "kv_min": kv_min, "kv_max": kv_max, "q_min": q_min,
         "q_max": q_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence decoding: a single token is rotated and appended
        _append("append_1", "bf16", 1, 32, 8, 128, 64, 128),
        # a decode step of a full batch, a quarter of a wide head rotated
        _append("append_96_d256", "bf16", 96, 16, 2, 256, 32, 64),
        # a prefill chunk that also holds padding tokens (no slot), fp32, interleaved pairs, odd head counts
        _append("append_ragged_f32", "f32", 1543, 15, 5, 64, 16, 32, True, 37),
        # an 8K prompt
        _append("append_8k", "bf16", 8192, 32, 8, 128, 64, 128),
        # the first steps of one chat
        _attention("decode_short", "bf16", 1, 257, 257, 1, 1, 32, 8, 128, 64),
        # 32 sequences being served, contexts up to 8K
        _attention("decode_32x8k", "bf16", 32, 1024, 8192, 1, 1, 32, 8, 128, 64),
        # long documents, few sequences: the key axis has to be split
        _attention("decode_long", "bf16", 2, 100000, 131072, 1, 1, 32, 8, 128, 128),
        # wide heads, many query heads per key head
        _attention("decode_d256", "bf16", 16, 16384, 32768, 1, 1, 16, 2, 256, 32),
        # fp32 with a sliding window, odd head counts, small pages, a sequence still empty
        _attention("decode_f32_window", "f32", 9, 0, 4097, 1, 1, 15, 5, 64, 16, 1000),
        # several drafted tokens per sequence checked at once, ragged
        _attention("verify_24", "bf16", 24, 700, 6001, 1, 6, 48, 8, 128, 64),
        # chunked prefill: new tokens of several sequences over longer contexts
        _attention("chunk_d256", "bf16", 3, 5000, 16384, 300, 2048, 16, 2, 256, 64),
        # an 8K prompt
        _attention("prefill_8k", "bf16", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 64),
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
        kind = rng.choice(["append", "decode", "decode", "several", "prefill"])
        if kind == "append":
            tokens = _log_int(rng, 1, 8192)
            c = _append(None, dtype, tokens, hq, hkv, d, page, rng.choice([r for r in (32, 64, 128, 256) if r <= d]),
                        rng.random() < 0.3, tokens // rng.choice([7, 20, 10 ** 6]))
            cost = tokens * (hq + 2 * hkv) * d / (8192 * 48 * 128)
        else:
            window = rng.choice([0, 0, _log_int(rng, 100, 5000)])
            if kind == "decode":
                batch, kv, q = _log_int(rng, 1, 64), _log_int(rng, 50, 131072), 1
            elif kind == "several":
                batch, kv, q = _log_int(rng, 1, 32), _log_int(rng, 50, 16384), rng.randint(2, 17)
            else:
                batch, kv = rng.randint(1, 4), _log_int(rng, 64, 8192)
                q = rng.randint(kv // 4, kv)
            c = _attention(None, dtype, batch, int(kv * rng.random()), kv, max(1, int(q * rng.random())), q, hq, hkv, d,
                           page, window)
            cost = batch * max(kv * hkv * d / (2 * 131072 * 8 * 128), q * kv * hq * d / (8192 * 8192 * 32 * 128 / 2),
                               q * kv * hq / (8192 * 8192 * 32))
        sizes = [v for v in c.values() if isinstance(v, int)] + [hq * d, hkv * d, (hq + 2 * hkv) * d]
        if cost <= 1 and 3072 not in sizes:
            return c


def _spread(lo, hi, n, step):
    """n whole numbers spread over [lo, hi], both ends among them where n > 1."""
    v = [lo + int((hi - lo) * ((i * step) % 1.0) + 0.5) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(case):
    kv = _spread(case["kv_min"], case["kv_max"], case["batch"], 0.6180339887)
    q = _spread(case["q_min"], case["q_max"], case["batch"], 0.7548776662)
    return kv, q


def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        t, rows = case["tokens"], case["tokens"] - case["skipped"]
        moved = t * (2 * hq + 2 * hkv) * d * size + t * case["rot"] * 4 + 2 * rows * hkv * d * 9 // 8 + 2 * t * hkv * d * size
        return {"bytes": moved, "flops": 3.0 * t * (hq + hkv) * case["rot"] + 4.0 * rows * hkv * d}
    kv, q = _lengths(case)
    window = case["window"] or (1 << 40)
    keys = pairs = 0
    for n, m in zip(kv, q):
        first = max(0, n - m)                                # positions of the queries: n - m .. n - 1
        keys += n - max(0, min(n, first - window + 1))
        for_all = sum(min(p + 1, window) for p in range(first, n))
        pairs += for_all
    rows = sum(q)
    moved = keys * hkv * d * 9 // 8 + rows * hq * (2 * d * size + 4)
    return {"bytes": moved, "flops": 4.0 * d * hq * pairs}


# ------------------------------------------------------------------------ the inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _channels(gen, heads, d):
    """Per-channel gains of keys: most near 1, a few channels several times larger."""
    gain = torch.rand(heads, d, generator=gen, device=DEV) + 0.5
    big = torch.rand(heads, d, generator=gen, device=DEV) < 0.03
    return torch.where(big, gain * 4, gain)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)   # noqa: E731
    gain = _channels(gen, hkv, d)
    s = {"case": case, "tables": _tables(),
         "k_gscale": (14.0 + torch.rand(hkv, generator=gen, device=DEV)) / 2688.0,
         "v_gscale": (5.0 + torch.rand(hkv, generator=gen, device=DEV)) / 2688.0}
    if case["op"] == "append":
        t = case["tokens"]
        qkv = torch.cat([normal(t, hq * d), (normal(t, hkv, d) * gain).view(t, hkv * d), normal(t, hkv * d)], 1)
        s["qkv"] = qkv.to(_dtype(case))                      # one fused projection's output
        n_pages = -(-t // page) + 2
        slots = torch.randperm(n_pages, generator=gen, device=DEV)[torch.arange(t, device=DEV) // page] * page
        s["slots"] = slots + torch.arange(t, device=DEV) % page
        if case["skipped"]:
            s["slots"][torch.randperm(t, generator=gen, device=DEV)[:case["skipped"]]] = -1
        n_pos = 32768
        s["positions"] = ((torch.randint(0, n_pos, (1,), generator=gen, device=DEV) + torch.arange(t, device=DEV))
                          % n_pos).to(torch.int32)
        inv = THETA ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        angle = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["cache"] = torch.zeros(n_pages, hkv * page * d * 9 // 8, dtype=torch.uint8, device=DEV)
        s["q_out"] = torch.empty(t, hq * d, dtype=_dtype(case), device=DEV)
        s["k_rows"] = torch.empty(t, hkv * d, dtype=_dtype(case), device=DEV)
        s["v_rows"] = torch.empty(t, hkv * d, dtype=_dtype(case), device=DEV)
        return s
    kv, q = _lengths(case)
    rows, n_max = sum(q), -(-case["kv_max"] // page)
    need = [-(-n // page) for n in kv]
    n_pages = sum(need) + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((case["batch"], n_max), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["cache"] = torch.empty(n_pages, hkv * page * d * 9 // 8, dtype=torch.uint8, device=DEV)
    some = max(1, (1 << 23) // (hkv * page * d))             # pages filled at a time
    for p in range(0, n_pages, some):
        n = min(some, n_pages - p)
        k = normal(n, page, hkv, d) * gain
        s["cache"][p:p + n] = _pages_of(k, normal(n, page, hkv, d), s["k_gscale"], s["v_gscale"], s["tables"])
    s["q"] = (normal(rows, hq, d) * 0.7).view(rows, hq * d).to(_dtype(case))
    s["table"] = table
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu_q"] = torch.tensor([0] + q, device=DEV).cumsum(0).to(torch.int32)
    s["o"] = torch.empty(rows, hq * d, dtype=_dtype(case), device=DEV)
    s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------ plain forms

def _side(a, m, g):
    """Sign of a - m g in fp32 operations, exactly, for a >= 0 and m of at most 7
    significant bits: g is split so that both partial products are exact."""
    high = (g.view(torch.int32) & -4096).view(torch.float32)
    low = g - high
    return (a - m * high) - m * low


def _tables():
    """The formats' values on the device, kept by the program: E2M1 magnitudes, the
    midpoints between them and which ties go up, the two values of each byte of codes,
    the value of each E4M3 byte."""
    mags = torch.tensor(MAGS, device=DEV)
    signed = torch.cat([mags, -mags])
    byte = torch.arange(256, device=DEV)
    e, m = (byte >> 3) & 15, (byte & 7).float()
    v = torch.where(e > 0, torch.ldexp(1.0 + m / 8, e - 7), m / 512)
    return {"mags": mags, "mids": torch.tensor(MIDS, device=DEV), "tie_up": torch.tensor(TIE_UP, device=DEV),
            "pairs": torch.stack([signed[byte & 15], signed[byte >> 4]], -1), "e4m3": torch.where(byte >= 128, -v, v)}


def _quantize(x, g, tables):
    """NVFP4 of the last dimension of x (fp32) under g (broadcast over it): codes
    [..., D] and scales [..., D/16] as whole numbers in uint8."""
    blocks = x.unflatten(-1, (-1, 16))
    g = g.expand(x.shape[:-1] + (1,)).contiguous()
    amax = blocks.abs().amax(-1)
    t = (amax / (6.0 * g)).clamp(max=448.0)
    e = torch.frexp(t).exponent.clamp(min=-5) - 1                  # t in [2^e, 2^(e+1)), at least 2^-6
    step = torch.ldexp(torch.ones_like(t), e - 3)
    n = torch.floor(t / step)
    r = _side(amax, 6.0 * (n + 0.5) * step, g)
    n = n + ((r > 0) | ((r == 0) & (n % 2 == 1)))
    s = (n * step).clamp(max=448.0)
    r = _side(blocks.abs().unsqueeze(-1), (s[..., None] * tables["mids"]).unsqueeze(-2), g[..., None, None])
    code = ((r > 0) | ((r == 0) & tables["tie_up"])).sum(-1)
    code = torch.where(s[..., None] > 0, code, 0) + 8 * torch.signbit(blocks)
    e = torch.frexp(s).exponent - 1
    byte = torch.where(e < -6, s * 512.0, (e + 7) * 8 + (torch.ldexp(s, -e) - 1) * 8)
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def _pairs(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _pages_of(k, v, kg, vg, tables):
    """Pages [n, bytes] of k and v [n, page, Hkv, D]."""
    n, page, hkv, d = k.shape
    kc, ks = _quantize(k, kg[:, None], tables)
    vc, vs = _quantize(v, vg[:, None], tables)
    rows = lambda x: x.transpose(1, 2).reshape(n, hkv, page // 16, 16, -1)   # noqa: E731
    vc = rows(_pairs(vc)).unflatten(-1, (16, -1)).unflatten(3, (4, 4)).transpose(4, 5)
    vs = rows(vs).unflatten(3, (4, 4)).transpose(4, 5)
    parts = [rows(_pairs(kc)), rows(ks), vc, vs]
    return torch.cat([p.reshape(n, hkv, page // 16, -1) for p in parts], -1).view(n, -1)


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] fp32; cos and sin [T, rot/2]."""
    c, s = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def _plain_append(s):
    case = s["case"]
    t, d, hq, hkv, page = case["tokens"], case["d"], case["hq"], case["hkv"], case["page"]
    x = s["qkv"].float()
    pos = s["positions"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(x[:, :hq * d].view(t, hq, d), cos, sin, case["rot"], case["interleaved"])
    k = _rotate(x[:, hq * d:(hq + hkv) * d].view(t, hkv, d), cos, sin, case["rot"], case["interleaved"])
    v = x[:, (hq + hkv) * d:].view(t, hkv, d)
    kc, ks = _quantize(k, s["k_gscale"][:, None], s["tables"])
    vc, vs = _quantize(v, s["v_gscale"][:, None], s["tables"])

    # the bytes' places in the cache
    live = s["slots"] >= 0
    slot = s["slots"].clamp(min=0)
    token = slot % page
    size = 18 * d
    base = ((slot // page)[:, None] * hkv + torch.arange(hkv, device=DEV)) * (page // 16) + (token // 16)[:, None]
    base = base[..., None] * size
    r = (token % 16)[:, None, None]
    quad, e = r // 4, r % 4
    j, b = torch.arange(d // 2, device=DEV), torch.arange(d // 16, device=DEV)
    part = d // 32
    places = [base + r * (d // 2) + j, base + 8 * d + r * (d // 16) + b,
              base + 9 * d + ((quad * 16 + j // part) * 4 + e) * part + j % part,
              base + 17 * d + (quad * (d // 16) + b) * 4 + e]
    at = torch.cat([p.expand(t, hkv, -1) for p in places], -1)
    new = torch.cat([_pairs(kc), ks, _pairs(vc), vs], -1)
    # tokens without a slot write to one byte past the cache
    flat = torch.cat([s["cache"].view(-1), s["cache"].new_zeros(1)])
    flat[torch.where(live[:, None, None], at, flat.numel() - 1)] = new
    s["cache"].view(-1).copy_(flat[:-1])

    def rows(code, scale, g):
        code = code.long()
        mags = s["tables"]["mags"][code & 7]
        value = torch.where(code >= 8, -mags, mags) * s["tables"]["e4m3"][scale.long()].repeat_interleave(16, -1) * g[:, None]
        return torch.where(live[:, None, None], value, 0).reshape(t, -1).to(_dtype(case))

    return {"q": q.reshape(t, -1).to(_dtype(case)), "k": rows(kc, ks, s["k_gscale"]), "v": rows(vc, vs, s["v_gscale"])}


def _plain_values(s):
    """Keys and values [B, Hkv, S, D] of the sequences' pages in fp32, without the
    global scales."""
    case = s["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    b, n = s["table"].shape
    pages = s["cache"].view(-1, hkv, page // 16, 18 * d)[s["table"].clamp(min=0).long()]
    pages = pages.permute(0, 2, 1, 3, 4)                           # [B, Hkv, pages, granules, bytes]
    pair, e4m3 = s["tables"]["pairs"], s["tables"]["e4m3"]
    lead = (b, hkv, n * (page // 16))

    def codes(x):
        return pair.index_select(0, x.reshape(-1).int()).view(lead + (-1,))

    def scales(x):
        return e4m3.index_select(0, x.reshape(-1).int()).view(lead + (-1,))

    kc = codes(pages[..., :8 * d]).view(lead + (16, d // 16, 16))
    k = kc * scales(pages[..., 8 * d:9 * d]).view(lead + (16, d // 16, 1))
    vc = codes(pages[..., 9 * d:17 * d]).view(lead + (4, 16, 4, d // 16))
    vs = scales(pages[..., 17 * d:]).view(lead + (4, d // 16, 4))
    v = vc.transpose(4, 5).reshape(lead + (4, 4, d // 16, 16)) * vs.transpose(4, 5)[..., None]
    return k.reshape(b, hkv, -1, d), v.reshape(b, hkv, -1, d)


def _plain_attention(s):
    case = s["case"]
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    group, batch, most = hq // hkv, case["batch"], case["q_max"]
    rows = s["q"].shape[0]
    k, v = _plain_values(s)
    row = torch.arange(rows, device=DEV)
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu[1:], row, right=True)
    place = seq * most + row - cu[seq]
    q = torch.zeros(batch * most, hq * d, device=DEV)
    q[place] = s["q"].float()
    q = q.view(batch, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * most, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (s["k_gscale"] / math.sqrt(d))[:, None, None]
    n, m = s["kv_len"].long(), cu[1:] - cu[:-1]
    pos = (n - m)[:, None] + torch.arange(most, device=DEV)
    t = torch.arange(k.shape[2], device=DEV)
    allowed = (t <= pos[..., None]) & (t < n[:, None, None])
    if case["window"]:
        allowed &= t > pos[..., None] - case["window"]
    score = score.view(batch, hkv, group, most, -1).masked_fill_(~allowed[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(torch.where(top > -math.inf, top, 0)))
    total = p.sum(-1, keepdim=True)
    # tokens past the end hold whatever the pages hold: never multiplied in
    live = t < n[:, None]
    v = torch.where(live[:, None, :, None], v, 0)
    o = torch.matmul(p.view(batch, hkv, group * most, -1), v) * s["v_gscale"][:, None, None]
    o = o.view(batch, hkv, group, most, d) / torch.where(total > 0, total, 1)
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch * most, hq * d)[place]
    lse = lse.permute(0, 3, 1, 2).reshape(batch * most, hq)[place]
    return {"o": o.to(_dtype(case)), "lse": lse}


# ------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return _plain_append(s) if case["op"] == "append" else _plain_attention(s)
    import nvfp4_w4a4_quantized_amd as nv
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    if case["op"] == "append":
        q, k, v = s["qkv"].split([hq * d, hkv * d, hkv * d], 1)
        nv.nvfp4_rope_append_kv(q, k, v, s["cos"], s["sin"], s["positions"], s["slots"], s["cache"], s["k_gscale"],
                                s["v_gscale"], page, s["q_out"], interleaved=case["interleaved"])
        nv.nvfp4_kv_gather(s["cache"], s["slots"], s["k_gscale"], s["v_gscale"], page, s["k_rows"], s["v_rows"])
        return {"q": s["q_out"], "k": s["k_rows"], "v": s["v_rows"]}
    if "workspace" not in s:                                 # kept by the program between its calls
        need = nv.nvfp4_kv_attention_workspace(s["q"].shape[0], case["batch"], hq, hkv, d, case["q_max"], case["kv_max"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_attention(s["q"], s["cache"], s["table"], s["kv_len"], s["k_gscale"], s["v_gscale"], page, s["o"],
                          case["kv_max"], s["workspace"], cu_q=None if case["q_max"] == 1 else s["cu_q"],
                          max_q_len=case["q_max"], window=case["window"], lse=s["lse"])
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


def _exact_grid(q, values):
    """q >= 0 rounded to the nearest of the increasing values (ties to an even place)."""
    values = torch.tensor(values, dtype=torch.float64, device=q.device)
    hi = torch.searchsorted(values, q).clamp(1, len(values) - 1)
    lo = hi - 1
    below, above = q - values[lo], values[hi] - q
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return values[torch.where(up, hi, lo)]


def _exact_quantized(x, g):
    """The values that NVFP4 holds for x [T, H, D] under g [H], in 64 bits."""
    g = g.double()[:, None, None]
    blocks = x.unflatten(-1, (-1, 16))
    grid = [m / 512 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    s = _exact_grid(blocks.abs().amax(-1, keepdim=True) / (6 * g), grid)
    unit = torch.where(s > 0, s * g, 1)
    value = torch.sign(blocks) * _exact_grid(blocks.abs() / unit, [0, 0.5, 1, 1.5, 2, 3, 4, 6]) * s * g
    return value.flatten(-2)


def _exact_append(s):
    case = s["case"]
    t, d, hq, hkv, rot = case["tokens"], case["d"], case["hq"], case["hkv"], case["rot"]
    x = s["qkv"].double().view(t, -1, d)
    pos = s["positions"].long()
    turn = torch.complex(s["cos"].double()[pos], s["sin"].double()[pos])[:, None]
    head = x[:, :hq + hkv, :rot]
    pair = head.unflatten(-1, (-1, 2)) if case["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.complex(pair[..., 0], pair[..., 1]) * turn)
    turned = turned.flatten(-2) if case["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    y = torch.cat([turned, x[:, :hq + hkv, rot:]], -1)
    live = (s["slots"] >= 0)[:, None, None]
    k = torch.where(live, _exact_quantized(y[:, hq:], s["k_gscale"]), 0)
    v = torch.where(live, _exact_quantized(x[:, hq + hkv:], s["v_gscale"]), 0)
    return {"q": y[:, :hq].reshape(t, -1), "k": k.reshape(t, -1), "v": v.reshape(t, -1)}


def _exact_rows(granules, d, n):
    """The first n keys and values [n, D] held by granules [G, 18 D], without global scales."""
    parts = d // 16
    nib = lambda x: torch.stack([x % 16, x // 16], -1).flatten(-2)   # noqa: E731
    kc = _exact_code(nib(granules[:, :8 * d])).view(-1, 16, parts, 16)
    k = kc * _exact_scale(granules[:, 8 * d:9 * d]).view(-1, 16, parts, 1)
    vc = _exact_code(nib(granules[:, 9 * d:17 * d])).view(-1, 4, 16, 4, parts).permute(0, 1, 3, 2, 4)
    vs = _exact_scale(granules[:, 17 * d:]).view(-1, 4, parts, 4).permute(0, 1, 3, 2)
    v = vc.reshape(-1, 16, parts, 16) * vs.reshape(-1, 16, parts, 1)
    return k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    group = hq // hkv
    kv, q = _lengths(case)
    rows = s["q"].shape[0]
    o = torch.zeros(rows, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)
    start = 0
    for n, m, table in zip(kv, q, s["table"]):
        pages = s["cache"].view(-1, hkv, page // 16, 18 * d)[table[:-(-n // page)].long()]
        for h in range(hkv if n else 0):
            k, v = _exact_rows(pages[:, h].reshape(-1, 18 * d), d, n)
            k, v = k * s["k_gscale"][h].double(), v * s["v_gscale"][h].double()
            heads = slice(h * group, (h + 1) * group)
            for i in range(0, m, 1024):
                mm = min(1024, m - i)
                at = slice(start + i, start + i + mm)
                x = s["q"][at].double().view(mm, hq, d)[:, heads].reshape(mm * group, d)
                score = (x @ k.t() / math.sqrt(d)).view(mm, group, n)
                pos = n - m + i + torch.arange(mm, device=DEV)[:, None, None]
                t = torch.arange(n, device=DEV)
                score = score.masked_fill((t > pos) | (t <= pos - (case["window"] or 1 << 40)), -math.inf)
                weight = torch.softmax(score, -1).nan_to_num(0.0)
                o[at, heads] = (weight.reshape(mm * group, n) @ v).view(mm, group, d)
                lse[at, heads] = torch.logsumexp(score, -1)
        start += m
    return {"o": o.reshape(rows, -1), "lse": lse}
