"""Registers and scratch of built kernels, as the compiler states them in the
library: what one form of a kernel carries must not cost the others their
waves.  Reads only the gfx950 code objects that this repository's build made."""
import os

import pytest

import fp4_block_scaled_quantize_amd as fq
from tests.helpers import kernel_resources as kr


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(fq.LIB_PATH) or not kr.available():
        pytest.skip("no built library, or no tools to read it")
    return kr.kernels(fq.LIB_PATH, tmp_path_factory.mktemp("code"))


def _of(kernels, name):
    return {n: v for n, v in kernels.items() if f"fp4::{name}<" in n}


# Waves of a SIMD in the plain weight-only product's forms before it could take
# adapters (E2M1, block 16, binary E4M3 scales): waves a workgroup, slots, row
# groups, X rows / 4, runs a chunk.
PLAIN = {"4, 4, 1, 0, 16, false, false, 0, 1": 8, "8, 4, 1, 0, 16, false, false, 0, 1": 8,
         "4, 4, 2, 1, 16, false, false, 0, 1": 4, "4, 4, 1, 1, 16, false, false, 0, 1": 8,
         "4, 4, 2, 2, 16, false, false, 0, 1": 4, "4, 4, 1, 2, 16, false, false, 0, 2": 5,
         "4, 2, 2, 4, 16, false, false, 0, 1": 4}


def test_plain_weight_only_product_keeps_its_waves(kernels):
    wo = _of(kernels, "k_wo_gemm")
    assert wo and not any(v["scratch"] for v in wo.values())
    for form, waves in PLAIN.items():
        plain = [v for n, v in wo.items() if f"k_wo_gemm<{form}>" in n or f"k_wo_gemm<{form}, false>" in n]
        assert len(plain) == 1, form
        assert kr.waves(plain[0]["vgpr"]) >= waves, (form, plain[0])
