"""The calls with packed arguments (include/a4w4_binding.h) are those of the same name: every word in its place (no GPU needed)."""

import os
import re

import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from mxfp4_a4w4_gemm_gb300 import _native
from mxfp4_a4w4_gemm_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

GOOD = {   # arguments that only the missing device refuses, in the order of include/a4w4.h
    "a4w4_gemm_w8a8": [16, 2, 256, 16, 16, 256, 16, 0, 0, 0, 0],
    "a4w4_kv_read": [16, 4, 16, 16, 2, 2, 128, 16, 16, 0],
    "a4w4_moe_route": [16, 0, 64, 16, 2, 64, 1, 16, 8, 2, 4, 8, 1, 2.5, 16, 16, 0],
    "a4w4_qk_norm_rope": [16, 512, 16, 256, 16, 2, 4, 2, 128, 16, 16, 1e-6, 16, 128, 0, 16, 512, 16, 256, 0],
    "a4w4_kv_append_rope": [16, 512, 16, 256, 16, 256, 16, 16, 2, 4, 2, 128, 16, 16, 1e-6, 16, 128, 0, 16, 512, 16, 4, 16, 0],
}
WRONG = (-1, 1, 3, 1 << 20, 0)     # values that some of the arguments must not have


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return a4w4.lib()


def test_every_declared_symbol_is_exported_and_packed(L):
    src = open(os.path.join(ROOT, "include", "a4w4_binding.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(a4w4_\w+)\s*\(", src)))
    assert names == sorted(_native.PACKED)
    for n in names:
        plain = n.replace("packed_", "")
        assert _native.PACKED[n].size == 8 * len(a4w4.SIGNATURES[plain][1]) == 8 * len(GOOD[plain])
        assert getattr(L, n)(None) == a4w4.A4W4_ERR_ARG


@pytest.mark.parametrize("name", sorted(GOOD))
def test_refusals_are_the_same_whichever_argument_is_wrong(L, name):
    plain, packed = getattr(L, name), getattr(L, name.replace("a4w4_", "a4w4_packed_"))
    pack = _native.PACKED[name.replace("a4w4_", "a4w4_packed_")].pack
    seen = set()
    for i in range(len(GOOD[name])):
        for v in WRONG:
            args = list(GOOD[name])
            args[i] = float(v) if isinstance(args[i], float) else v
            if plain(*args) == a4w4.A4W4_ERR_ARG:       # (nothing that a GPU would run)
                assert packed(pack(*args)) == a4w4.A4W4_ERR_ARG
                seen.add(i)
    # every argument but flags of two values, optional pointers that 0 leaves out, and the stream can be wrong
    assert len(seen) >= len(GOOD[name]) - 3
