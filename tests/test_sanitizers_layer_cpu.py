"""The host code of the epilogue, mixture-of-experts and distillation calls
under AddressSanitizer and UndefinedBehaviorSanitizer, without a GPU: their
argument checks, workspaces, size products, K ranges and launch shapes over
the sizes that they take (tests/helpers/abi_layer_host.cpp, which stands in for
the HIP runtime and looks at every launch)."""
import concurrent.futures as cf
import os
import shutil

import pytest

from tests.conftest import ROOT
from tests.test_sanitizers_train_cpu import CLANG, CSRC, ENV, _run


def test_layer_abi_host_code_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc) or not os.path.exists(CLANG):
        pytest.skip("no ROCm toolchain")
    # the host pass alone: no device code is made, and none is needed
    flags = ["--offload-host-only", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    srcs = [*(os.path.join(CSRC, f) for f in ("api_layer.cpp", "gemm.hip", "gemm_epilogue.hip", "moe.hip", "epilogue.hip", "distill.hip")),
            os.path.join(ROOT, "tests", "helpers", "abi_layer_host.cpp")]

    def build(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([hipcc, *flags, "-x", "hip", "-c", src, "-o", obj])
        return obj
    with cf.ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(build, srcs))
    exe = str(tmp_path / "abi_layer_san")
    # the device code's images, which a registration would name, do not exist
    _run([CLANG, "-fsanitize=address,undefined", *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe])
    r = _run([exe], env={**os.environ, **ENV}, timeout=300)
    assert r.stdout.strip() == "ok"
