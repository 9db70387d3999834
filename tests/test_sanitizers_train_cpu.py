"""The host code of the adapter, token-probability and residual-norm calls
under AddressSanitizer and UndefinedBehaviorSanitizer, without a GPU: their
argument checks, workspace offsets, size products and launch shapes over the
sizes that they take (tests/helpers/abi_train_host.cpp, which stands in for the
HIP runtime and looks at every launch)."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "fp4_block_scaled_quantize_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"
ENV = {"ASAN_OPTIONS": "detect_leaks=1:abort_on_error=1", "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1"}


def _run(cmd, **kw):
    r = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert r.returncode == 0, f"{' '.join(cmd)}\n{r.stdout[-4000:]}\n{r.stderr[-4000:]}"
    return r


def test_train_abi_host_code_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc) or not os.path.exists(CLANG):
        pytest.skip("no ROCm toolchain")
    # the host pass alone: no device code is made, and none is needed
    flags = ["--offload-host-only", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in [*(os.path.join(CSRC, f) for f in ("api_train.cpp", "lora.hip", "logprobs.hip", "norm.hip")),
                os.path.join(ROOT, "tests", "helpers", "abi_train_host.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run([hipcc, *flags, "-x", "hip", "-c", src, "-o", objs[-1]])
    exe = str(tmp_path / "abi_train_san")
    # the device code's images, which a registration would name, do not exist
    _run([CLANG, "-fsanitize=address,undefined", *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe])
    r = _run([exe], env={**os.environ, **ENV}, timeout=300)
    assert r.stdout.strip() == "ok"
