"""Host code of the entry points over 4-bit integer weights and over inputs saved in 8
bits (argument checks, workspace queries, the plans of the products) under
AddressSanitizer and UndefinedBehaviorSanitizer, built on the host pass only; no kernel
is launched.  Any report aborts the driver."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import BUILD, CLANGXX, CSRC, HERE, HIPCC, ROOT, SAN_HOST, run

CHECKED = ["api.cpp", "mxfp4_api.cpp", "int4_api.cpp", "mxint8_api.cpp", "mxfp4_gemm.hip", "int4_gemm.hip", "int4_gemm_t.hip"]
PLAIN = ["lowrank_kernels.hip", "gemm_kernels.hip", "dora_kernels.hip", "mxfp4_kernels.hip", "mxfp4_gemm_t.hip",
         "mxfp4_join.hip", "int4_kernels.hip", "int4_finish.hip", "mxint8_kernels.hip"]


def test_packed_host_code_under_sanitizers(tmp_path):
    kernels = [os.path.join(BUILD, f + ".o") for f in PLAIN]
    if not (os.path.exists(HIPCC) and os.path.exists(CLANGXX) and all(map(os.path.exists, kernels))):
        pytest.skip("hipcc / clang++ or the built kernel objects are missing")
    includes = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    flags = ["-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", *includes,
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]

    def build(src):
        obj = str(tmp_path / (src + ".o"))
        run([HIPCC] + flags + SAN_HOST + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    with ThreadPoolExecutor(4) as pool:
        objs = list(pool.map(build, CHECKED))
    drv = str(tmp_path / "packed_driver.o")
    run([CLANGXX, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         "-D__HIP_PLATFORM_AMD__", *includes, "-I", "/opt/rocm/include",
         "-c", os.path.join(HERE, "packed_driver.cpp"), "-o", drv])
    exe = str(tmp_path / "packed_san")
    run([CLANGXX, "-fsanitize=address,undefined", drv] + objs + kernels +
        ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    assert "all checks passed" in run([exe]).stdout
