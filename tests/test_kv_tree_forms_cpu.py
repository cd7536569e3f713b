"""Which kernel a drafted tree's attention is planned for, by the workspace that the call asks for: sizes
for every form of the prompts' kernel (tests/test_gpu_kv_tree_forms.py runs them), so that a change of the rule
that chooses between the kernels is seen here."""

import ctypes
import re
from typing import NamedTuple

import numpy as np
import pytest
import torch

from tests.test_kv_abi_cpu import FAKE, nv  # noqa: F401  (the fixture)


class Form(NamedTuple):
    """Trees of up to `most_q` announced nodes (m: the real ones) of sequences of kv tokens, under an announced
    length far above them, which is what sends such short ones to the prompts' kernel.  tile: columns of an
    item (128: two groups of waves share its tiles); cut: whether items are cut along the keys."""
    D: int
    group: int
    Hkv: int
    kv: tuple
    m: tuple
    most_q: int
    window: int
    tile: int
    cut: bool
    most_kv: int = 100000

    @property
    def words(self):
        return -(-max(self.m) // 64)


def _batch(kv, m, size):
    """Further sequences of few tokens and nodes, down to none."""
    rng = np.random.default_rng(size)
    more = size - len(kv)
    n = rng.integers(0, 60, more)
    return tuple(kv) + tuple(n.tolist()), tuple(m) + tuple(np.minimum(rng.integers(0, 10, more), n + 2).tolist())


def _forms():
    out = []
    for D in (64, 128, 256):
        for tile in (128, 256) if D < 256 else (256,):
            g = 2 if tile == 128 else 4
            # cut, then whole (more than 64 sequences); a window that ends inside the longest ones
            out.append(Form(D, g, 2, (700, 64, 300), (64, 33, 40), 64, 0, tile, True))
            out.append(Form(D, g, 3, *_batch((2600, 2075, 64), (64, 40, 64), 33), 64, 2000, tile, True))
            wide = 4 * g
            heads = 256 // tile
            out.append(Form(D, wide, heads, *_batch((400, 130), (9, 9), 66), 9, 0, tile, False))
            out.append(Form(D, wide, heads, *_batch((5400, 5010), (9, 7), 66), 9, 5000, tile, False))
            # more nodes than announced: tiles past the planned ones
            out.append(Form(D, g, 2, (500, 160), (150, 70), 40, 0, tile, True, 1000000))
            out.append(Form(D, wide, heads, *_batch((300, 90), (40, 9), 66), 9, 0, tile, False))
        # words that do not fit a tile's place in LDS
        out.append(Form(D, 1, 1, (700,), (600,), 600, 0, 256, True, 1000000))
        out.append(Form(D, 1, 1, *_batch((3900,), (600,), 33), 600, 3000, 256, True))
    return out


FORMS = _forms()


def form_id(f):
    return f"{f.D}-{f.tile}-{'cut' if f.cut else 'whole'}-{len(f.kv)}x{max(f.kv)}-{max(f.m)}of{f.most_q}-w{f.window}"


@pytest.mark.skipif(torch.cuda.is_available(), reason="its buffers are not real: where there is a GPU the calls would be launched")
@pytest.mark.parametrize("f", FORMS, ids=form_id)
def test_form(nv, f):  # noqa: F811
    T, batch, hq = sum(f.m), len(f.kv), f.group * f.Hkv
    st = nv.lib.nvfp4_kv_tree_attention(FAKE, 1, hq * f.D, T, hq, f.Hkv, f.D, batch, FAKE, f.most_q, FAKE, f.most_kv, FAKE, 1000,
                                        1000, FAKE, 1 << 20, 16, FAKE, FAKE, ctypes.c_float(0.1), f.window, FAKE, f.words, f.words,
                                        FAKE, hq * f.D, None, None, 0, None)
    cols = min(f.most_q, T) * f.group
    items = batch * f.Hkv * -(-cols // f.tile)
    if f.cut:
        # a workgroup a piece, a piece a result of D + 4 floats a column, and 32 bytes: with 16 or 64 columns an
        # item, as in the other kernel, the sizes are others
        assert items <= 160 and batch <= 64
        blocks = 256 - items // 2 + items
        assert st == nv.NVFP4_ERR_INVALID_ARG
        need = int(re.search(r"too small: (\d+) needed", nv.nvfp4_last_error()).group(1))
        assert need == blocks * (f.tile * (f.D + 4) * 4 + 32)
    else:
        # no workspace: the call goes on to look for a device.  The other kernel, whose items of 16 columns are
        # fewer than 1024 and have more than 64 steps, would ask for one.
        assert st in (nv.NVFP4_ERR_HIP, nv.NVFP4_ERR_DEVICE), nv.nvfp4_last_error()
        span = min(f.window + f.most_q, f.most_kv) if f.window else f.most_kv
        assert batch * f.Hkv * -(-cols // 16) < 1024 and span > 64 * 64
