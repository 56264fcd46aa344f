"""Build libpkv's host code, the context operators' included, with
AddressSanitizer and UndefinedBehaviorSanitizer.

    python tests/sanitize/build_sanitized_context.py -> _build/libpkv_san_context.so

As build_sanitized.py, with csrc/context/context_api.cpp and its stub
launchers added.
"""
from __future__ import annotations

import os
import subprocess
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import build_sanitized as base  # noqa: E402

LIB = os.path.join(base.OUT_DIR, "libpkv_san_context.so")
SOURCES = base.SOURCES + [os.path.join(base.CSRC, "context", "context_api.cpp"),
                          os.path.join(base.HERE, "stub_context_launchers.cpp")]


def build() -> str:
    os.makedirs(base.OUT_DIR, exist_ok=True)
    cmd = ["g++", *base.FLAGS, *SOURCES, f"-L{base.ROCM}/lib", "-lamdhip64",
           f"-Wl,-rpath,{base.ROCM}/lib", "-o", LIB]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"sanitizer build failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return LIB


if __name__ == "__main__":
    print(build())
    sys.exit(0)
