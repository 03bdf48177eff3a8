"""The host side of the calls around the product under AddressSanitizer and UndefinedBehaviorSanitizer
(tests/sanitize/layer_host_checks.cpp; the sources' host side only, as in tests/test_sanitize.py)."""

import os
import re

import pytest

# the sources that decide sizes, plans and launches of these calls on the host
SOURCES = ["dg_host.hip", "norm_fp8.hip", "epilogue_bwd.hip"]


def test_layer_host_logic_under_asan_ubsan(tmp_path):
    from tests.test_sanitize import CLANG, HERE, HIPCC, PKG, ROOT, SAN_FLAGS, _env, _run

    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("ROCm toolchain not installed")
    lib = os.path.join(PKG, "libdg.so")
    if not os.path.exists(lib):
        pytest.skip("libdg.so not built (run __graft_entry__.build())")
    host_san = [x for f in SAN_FLAGS for x in ("-Xarch_host", f)]
    objs, no_code = [], []
    for src in SOURCES:
        objs.append(str(tmp_path / (src + ".o")))
        rc, out = _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", "--offload-host-only"] + host_san + ["-c", os.path.join(PKG, "csrc", src), "-o", objs[-1]])
        assert rc == 0, out
        # the device code that is not compiled: a symbol of the program's own in its place, registered nowhere
        rc, syms = _run(["nm", objs[-1]])
        assert rc == 0, syms
        no_code += ["-Wl,--defsym=%s=layer_checks_no_device_code" % x for x in sorted(set(re.findall(r" U (__hip_fatbin_\w+)", syms)))]
    exe = str(tmp_path / "layer_host_checks")
    rc, out = _run([CLANG, "-O1", "-g", "-std=c++17"] + SAN_FLAGS + ["-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "layer_host_checks.cpp")] +
                   objs + no_code + ["-L" + PKG, "-l:libdg.so", "-Wl,-rpath," + PKG, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=_env(False))
    assert rc == 0 and "layer host checks passed" in out, out
    assert "Sanitizer" not in out and "runtime error" not in out, out
