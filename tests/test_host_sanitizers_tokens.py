"""Host AddressSanitizer + UndefinedBehaviorSanitizer build of the whole C ABI
(api.cpp and api_tokens.cpp), with the ABI tests and the host tests of the
token-level calls run under it in a child process (no GPU)."""
import glob
import os
import sys

import pytest
import torch

from test_host_sanitizers import BUILD, CSRC, HIPCC, ROOT, _child, _run

DEVICE = ("quantize", "dequantize", "repack", "gemm", "selfcheck", "route", "tables", "combine", "logprobs")
TESTS = ["tests/test_%s.py" % n for n in ("abi", "tokens_api", "tokens_overlap", "tokens_strides", "tokens_sizes")]


def test_token_calls_under_asan_ubsan(tmp_path):
    rts = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    objs = [os.path.join(BUILD, n + ".o") for n in DEVICE]
    if not os.path.exists(HIPCC) or not rts or not all(os.path.exists(o) for o in objs):
        pytest.skip("hipcc, the clang sanitizer runtime or the built device objects are missing")
    so = str(tmp_path / "libmxfp8_san.so")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    host = []
    for n in ("api", "api_tokens"):
        host.append(str(tmp_path / (n + "_san.o")))
        _run([HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "-fno-omit-frame-pointer", *san,
              "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, n + ".cpp"), "-o", host[-1]])
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *san, *objs, *host, "-o", so])
    code = (
        "import sys; sys.path[:0] = ['tests', '.']\n"
        "import mxfp8_block_scaled_05_amd as m\n"
        "m.LIB_PATH = %r\n"
        "import pytest\n"
        "rc = pytest.main(['-q', '-x', '-p', 'no:cacheprovider', '-m', 'not gpu'] + %r)\n"
        "assert m.lib()._name == m.LIB_PATH\n"
        "print('RC', int(rc), flush=True)\n"
        "sys.exit(int(rc))\n") % (so, TESTS)
    out = _child(rts[-1], code, str(tmp_path))
    assert "RC 0" in out and ("skipped" not in out or torch.cuda.is_available())
