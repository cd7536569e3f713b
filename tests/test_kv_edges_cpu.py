"""Host-side rules of the key/value cache at the edges of their ranges.  CPU only."""

import ctypes
import importlib.util
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import kv as KV
from tests.test_kv_abi_cpu import _append, _gather, nv  # noqa: F401  (the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_w4a4_quantized_amd", "csrc")

RULES = """
#include "kv_layout.hpp"
extern "C" int planned_tiles(long long tiles, long long pairs, int threads) {
  return nvfp4::kv_planned_tiles(tiles, pairs, threads);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    """The host rules of kv_layout.hpp as a library."""
    at = tmp_path_factory.mktemp("rules")
    (at / "rules.cpp").write_text(RULES)
    subprocess.run(["g++", "-std=c++20", "-shared", "-fPIC", "-I", CSRC, "-o", str(at / "rules.so"), str(at / "rules.cpp")],
                   check=True)
    return ctypes.CDLL(str(at / "rules.so"))


@pytest.mark.parametrize("threads", [256, 512])
def test_planned_grids_stay_within_a_launch(rules, threads):
    plan = lambda tiles, pairs: rules.planned_tiles(ctypes.c_longlong(tiles), ctypes.c_longlong(pairs), threads)   # noqa: E731
    for pairs in (1, 7, 8192, 65536, (1 << 22) - 1, 1 << 22):
        for tiles in (1, 2, 127, 1024, 16384, 1 << 23, (1 << 31) // 16):
            got = plan(tiles, pairs)
            assert 1 <= got <= tiles and got * pairs * threads < 1 << 32
            assert got == tiles or (got + 1) * pairs * threads >= 1 << 32     # no fewer than need be


def test_rows_beyond_a_launch_are_refused(nv):   # noqa: F811
    # 2^36 elements are 2^32 threads, one more than a launch takes; just below, the missing slots are refused
    uns, inv = nv.NVFP4_ERR_UNSUPPORTED, nv.NVFP4_ERR_INVALID_ARG
    for d, tokens in ((64, 1 << 27), (128, 1 << 26), (256, 1 << 25)):
        heads = dict(d=d, hkv=2, ldk=2 * d, ldv=2 * d, slots=None)
        q = dict(hq=4, ldq=4 * d, ldqo=4 * d)
        assert _append(nv, T=tokens, **q, **heads) == uns and "2^36" in nv.nvfp4_last_error(), d
        assert _append(nv, T=tokens - 64, **q, **heads) == inv and "slots" in nv.nvfp4_last_error()
        assert _gather(nv, T=2 * tokens, **heads) == uns and "2^36" in nv.nvfp4_last_error(), d
        assert _gather(nv, T=2 * tokens - 64, **heads) == inv and "slots" in nv.nvfp4_last_error()


def test_prompts_leave_the_workspace_of_captured_steps_alone(nv, monkeypatch):   # noqa: F811
    """examples/attention_layer.py with the device's calls left out: the workspace that a captured
    step got is still the layer's after prompts that need more than any call before them."""
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    used = []
    for name in ("nvfp4_pack_weight", "nvfp4_w4a4_linear", "nvfp4_rope_append_kv"):
        monkeypatch.setattr(example.nv, name, lambda *a, **k: None)
    monkeypatch.setattr(example.nv, "nvfp4_kv_attention", lambda *a, **k: used.append(a[9]))
    layer = example.AttentionLayer(256, 8, 2, 64, 3, 5000, 3000, page=16, device="cpu")
    x, y = torch.zeros(3000, 256, dtype=torch.bfloat16), torch.zeros(3000, 256, dtype=torch.bfloat16)
    layer.prompt(x[:33], [30, 2, 1], y[:33])
    layer.decode(x[:3], y[:3])
    need = nv.nvfp4_kv_attention_workspace(3, 3, 8, 2, 64, 1, 5000, torch.bfloat16)
    captured = used[-1].data_ptr()
    assert need > 0 and used[-1].numel() >= need
    for lens in ([100, 200, 300], [2000, 10, 900], [1, 1, 1]):
        layer.prompt(x[:sum(lens)], lens, y[:sum(lens)])
        now = nv.nvfp4_kv_attention_workspace(sum(lens), 3, 8, 2, 64, max(lens), 5000, torch.bfloat16)
        assert used[-1].numel() >= now and used[-1].data_ptr() != captured
        layer.decode(x[:3], y[:3])
        assert used[-1].data_ptr() == captured


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py with its results under tmp_path and its commands recorded instead of run."""
    spec = importlib.util.spec_from_file_location("nvfp4_build", os.path.join(ROOT, "nvfp4_w4a4_quantized_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name, at in (("OBJDIR", "objects"), ("LIB", "libnvfp4.so"), ("BINDING", "_torch_binding.so")):
        monkeypatch.setattr(mod, name, str(tmp_path / at))
    mod.refuse = ()

    def run(cmd, verbose):
        if os.path.basename(cmd[0]) in mod.refuse:
            raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
    monkeypatch.setattr(mod, "_run", run)
    return mod


def test_the_library_is_built_without_torch_and_without_a_host_compiler(build, tmp_path, monkeypatch, capsys):
    library, binding = tmp_path / "libnvfp4.so", tmp_path / "_torch_binding.so"
    build.build()
    assert library.exists() and binding.exists()
    library.unlink()
    binding.unlink()
    build.refuse = ("g++",)
    with pytest.raises(FileNotFoundError):            # said, with the library in place
        build.build()
    assert library.exists() and not binding.exists()
    library.unlink()
    build.refuse = ()
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == str(library) and library.exists() and not binding.exists()
    assert "torch" in capsys.readouterr().err


def test_a_failed_runtime_is_reported_as_such(nv, monkeypatch):   # noqa: F811
    cache = torch.empty(4, nv.nvfp4_kv_page_bytes(2, 16, 64), dtype=torch.uint8)
    g, x, slots = torch.ones(2), torch.zeros(3, 128), torch.zeros(3, dtype=torch.int64)

    def call():
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.nvfp4_kv_gather(cache, slots, g, g, 16, x, x.clone())
        return e.value

    def failed():
        raise RuntimeError("HIP error: an earlier launch failed")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", failed)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    got = call()
    assert got.status == nv.NVFP4_ERR_HIP and "an earlier launch failed" in str(got)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)   # no GPU
    got = call()
    assert got.status == nv.NVFP4_ERR_INVALID_ARG and "device memory" in str(got)


def test_bounds_of_negative_scales():
    """A negative scale's bounds are those of the negated queries under the positive one."""
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((50, 2, 64)), rng.standard_normal((50, 2, 64))
    for dtype in ("bf16", "f32"):
        o, lse, w = KV.attention(q, k, v, -0.2)
        o2, lse2, w2 = KV.attention(-q, k, v, 0.2)
        assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2)
        for a, b in zip(KV.attention_bounds(q, k, v, w, -0.2, dtype), KV.attention_bounds(-q, k, v, w2, 0.2, dtype)):
            assert np.all(a > 0) and np.allclose(a, b, rtol=1e-9)
