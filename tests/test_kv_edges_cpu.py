"""Host-side rules of the key/value cache at the edges of their ranges.  CPU only."""

import ctypes
import os
import subprocess

import pytest

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
