"""The layers' host code built with AddressSanitizer and UndefinedBehavior-
Sanitizer (host pass only) and driven by tests/abi_sanitize_layers.cpp on the
CPU, any report failing the test."""

import importlib.util
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.conftest import ROOT

HIPCC = "/opt/rocm/bin/hipcc"
SANITIZE = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_layers_host_code_under_sanitizers(tmp_path):
    spec = importlib.util.spec_from_file_location(
        "taco_build", os.path.join(ROOT, "quantized_compression_tensor_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        lang = ["-x", "hip"] if src.endswith(".cpp") else []
        b = subprocess.run([HIPCC, *build.FLAGS, "-O1", "-g", *SANITIZE, "-Xarch_host", "-fno-sanitize-recover=undefined",
                            "-Xarch_host", "-fno-omit-frame-pointer", *lang, "-c", src, "-o", obj],
                           capture_output=True, text=True, timeout=600)
        return obj, b

    sources = [os.path.join(build.CSRC, s) for s in build.SOURCES] + [os.path.join(ROOT, "tests", "abi_sanitize_layers.cpp")]
    with ThreadPoolExecutor(len(sources)) as ex:
        built = list(ex.map(compile_one, sources))
    for _, b in built:
        assert b.returncode == 0, b.stdout[-3000:] + b.stderr[-3000:]
    exe = str(tmp_path / "abi_sanitize_layers")
    b = subprocess.run([HIPCC, "--offload-arch=gfx950", *SANITIZE, *[o for o, _ in built], "-o", exe],
                       capture_output=True, text=True, timeout=600)
    assert b.returncode == 0, b.stdout[-3000:] + b.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "all checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
