"""Host-side sanitizer run of the entry points between token ids and the expert layer: their host layer built
with AddressSanitizer and UndefinedBehaviorSanitizer (host code only), driven by an
argument fuzzer; the device code is linked as it was built.  No GPU is used."""
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_gram_amd", "csrc")
OBJS = os.path.join(ROOT, "newton_schulz_gram_amd", "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANG = "/opt/rocm/llvm/bin/clang++"
HOST_SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
            "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]


def _run(cmd, **kw):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
    assert r.returncode == 0, " ".join(cmd) + "\n" + r.stdout[-4000:]
    return r.stdout


@pytest.mark.skipif(not (os.path.exists(HIPCC) and shutil.which(CLANG)), reason="ROCm compilers not found")
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch kernels on addresses that are none")
def test_layer_host_code_under_asan_ubsan(tmp_path):
    kernels = [os.path.join(OBJS, f + ".o") for f in ("nsg_embed.hip", "nsg_norm.hip", "nsg_route.hip")]
    if not all(os.path.exists(k) for k in kernels):
        pytest.skip("device objects not built (run __graft_entry__.build() first)")
    api = str(tmp_path / "nsg_layer_api_san.o")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", *HOST_SAN,
          "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-x", "hip", "-c", os.path.join(CSRC, "nsg_layer_api.cpp"),
          "-o", api])
    lib = str(tmp_path / "libnsg_layer_san.so")
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *HOST_SAN, api, *kernels, "-o", lib])
    exe = str(tmp_path / "layer_host_fuzz")
    _run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
          "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "layer_host_fuzz.cpp"), lib, "-Wl,-rpath," + str(tmp_path), "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    out = _run([exe, "20000"], env=env, timeout=600)
    assert "ok 20000 iterations" in out
