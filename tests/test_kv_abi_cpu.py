"""Host-side validation of the key/value cache entry points: every refusal happens before
the GPU is touched.  CPU only."""

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(1 << 20)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def nv():
    if not os.path.exists(os.path.join(ROOT, "nvfp4_w4a4_quantized_amd", "libnvfp4.so")):
        import __graft_entry__
        __graft_entry__.build()
    import nvfp4_w4a4_quantized_amd as nvmod
    return nvmod


def test_page_bytes(nv):
    assert nv.nvfp4_kv_page_bytes(8, 64, 128) == 8 * 64 * 128 * 9 // 8
    for bad in ((0, 64, 128), (8, 64, 96), (8, 48, 128), (8, 8, 128), (8, 8192, 128)):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_kv_page_bytes(*bad)
    assert nv.lib.nvfp4_kv_page_bytes(8, 64, 128, None) == nv.NVFP4_ERR_INVALID_ARG


def _append(nv, q=FAKE, ldq=512, k=FAKE, ldk=256, v=FAKE, ldv=256, dt=1, T=4, hq=4, hkv=2, d=128, cos=FAKE, sin=FAKE,
            n_pos=100, rot=64, pos=FAKE, slots=FAKE, cache=FAKE, pages=4, page=16, kg=FAKE, vg=FAKE, qo=FAKE, ldqo=512):
    return nv.lib.nvfp4_rope_append_kv(q, ldq, k, ldk, v, ldv, dt, T, hq, hkv, d, cos, sin, n_pos, rot, 0, pos, slots, cache,
                                       pages, page, kg, vg, qo, ldqo, None)


def test_append_validation(nv):
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("k", "v", "pos", "slots", "cache", "kg", "vg", "cos", "sin"):
        assert _append(nv, **{name: None}) == inv, name
    assert _append(nv, q=None) == inv and _append(nv, qo=None) == inv and _append(nv, hq=0) == inv
    assert _append(nv, hq=-1) == inv and _append(nv, hkv=0) == inv and _append(nv, T=0) == inv
    assert _append(nv, ldk=128) == inv and _append(nv, ldqo=256) == inv
    assert _append(nv, d=96) == uns and _append(nv, page=24) == uns and _append(nv, dt=5) == uns
    assert _append(nv, pages=0) == inv and _append(nv, n_pos=0) == inv
    assert _append(nv, rot=160) == inv and _append(nv, rot=-32) == inv
    assert _append(nv, rot=48) == uns and "multiple of 32" in nv.nvfp4_last_error()
    assert _append(nv, cache=ODD) == uns and _append(nv, k=ODD) == uns and _append(nv, cos=ODD) == uns
    assert _append(nv, ldv=260) == uns
    assert _append(nv, T=1 << 30) == uns


def _gather(nv, cache=FAKE, pages=4, page=16, hkv=2, d=128, kg=FAKE, vg=FAKE, slots=FAKE, T=4, ko=FAKE, ldk=256, vo=FAKE,
            ldv=256, dt=1):
    return nv.lib.nvfp4_kv_gather(cache, pages, page, hkv, d, kg, vg, slots, T, ko, ldk, vo, ldv, dt, None)


def test_gather_validation(nv):
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("cache", "kg", "vg", "slots", "ko", "vo"):
        assert _gather(nv, **{name: None}) == inv, name
    assert _gather(nv, T=0) == inv and _gather(nv, ldk=128) == inv and _gather(nv, pages=-1) == inv
    assert _gather(nv, d=80) == uns and _gather(nv, page=20) == uns and _gather(nv, dt=2) == uns and _gather(nv, vo=ODD) == uns


def _attn(nv, q=FAKE, dt=1, ldq=512, T=2, hq=4, hkv=2, d=128, batch=2, cu=None, mq=1, kv=FAKE, mk=10, table=FAKE, mp=4, ldt=4,
          cache=FAKE, pages=4, page=16, kg=FAKE, vg=FAKE, scale=0.1, window=0, o=FAKE, ldo=512, lse=None, ws=None, wsb=0):
    return nv.lib.nvfp4_kv_attention(q, dt, ldq, T, hq, hkv, d, batch, cu, mq, kv, mk, table, mp, ldt, cache, pages, page, kg,
                                     vg, ctypes.c_float(scale), window, o, ldo, lse, ws, wsb, None)


def test_attention_validation(nv):
    inv, uns = nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED
    for name in ("q", "o", "kv", "table", "cache", "kg", "vg"):
        assert _attn(nv, **{name: None}) == inv, name
    assert _attn(nv, T=3) == inv and "one token" in nv.nvfp4_last_error()
    assert _attn(nv, T=0) == inv and _attn(nv, batch=0) == inv and _attn(nv, hq=3) == inv and _attn(nv, hkv=0) == inv
    assert _attn(nv, mq=0) == inv and _attn(nv, mk=-1) == inv and _attn(nv, window=-1) == inv
    assert _attn(nv, scale=float("nan")) == inv and _attn(nv, scale=float("inf")) == inv
    assert _attn(nv, mp=0) == inv and _attn(nv, ldt=3) == inv and _attn(nv, mp=1 << 28, ldt=1 << 28) == inv
    assert _attn(nv, ldq=256) == inv and _attn(nv, ldo=256) == inv
    assert _attn(nv, d=32) == uns and _attn(nv, page=17) == uns and _attn(nv, dt=9) == uns
    assert _attn(nv, q=ODD) == uns and _attn(nv, o=ODD) == uns and _attn(nv, cache=ODD) == uns
    assert _attn(nv, batch=1 << 22, T=1 << 22) == uns
    # a split call needs its workspace
    need = nv.nvfp4_kv_attention_workspace(2, 2, 4, 2, 128, 1, 100000, torch.bfloat16)
    assert need > 0
    assert _attn(nv, mk=100000) == inv and "workspace" in nv.nvfp4_last_error()
    assert _attn(nv, mk=100000, ws=FAKE, wsb=need - 1) == inv
    assert _attn(nv, mk=100000, ws=ODD, wsb=need) == uns


def test_workspace_covers_both_types(nv):
    for args in ((1, 1, 8, 1, 128, 1, 1), (64, 2, 6, 2, 64, 32, 70000), (8192, 1, 32, 8, 128, 8192, 8192)):
        both = nv.nvfp4_kv_attention_workspace(*args)
        assert both == max(nv.nvfp4_kv_attention_workspace(*args, dtype=t) for t in (torch.float32, torch.bfloat16))
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_kv_attention_workspace(1, 1, 8, 1, 128, 1, 1, dtype=torch.float16)


def test_binding_refuses_host_memory(nv):
    cache = torch.empty(4, nv.nvfp4_kv_page_bytes(2, 16, 64), dtype=torch.uint8)
    g, x, i32 = torch.ones(2), torch.zeros(3, 128), torch.zeros(3, dtype=torch.int32)
    slots = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: nv.nvfp4_kv_gather(cache, slots, g, g, 16, x, x.clone()),
                 lambda: nv.nvfp4_rope_append_kv(None, x, x, None, None, i32, slots, cache, g, g, 16, None),
                 lambda: nv.nvfp4_kv_attention(x, cache, i32[:, None], i32, g, g, 16, x.clone(), 10)):
        with pytest.raises(nv.Nvfp4Error, match="device memory") as e:
            call()
        assert e.value.status == nv.NVFP4_ERR_INVALID_ARG
