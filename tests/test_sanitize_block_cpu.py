"""The host logic of the row, routing and epilogue operators under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): the library's
translation units compiled for the host, linked with
tests/sanitize/block_checks.cpp and the stand-in HIP runtime without a device
(tests/sanitize/hip_stub.cpp)."""
import glob
import os
import re
import subprocess

import pytest

from test_sanitize_cpu import CLANG, CSRC, ENV, HIPCC, ROOT, SAN_DIR, _run


def test_block_host_logic_under_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("ROCm compilers not available")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    san = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer"]
    san_host = [x for f in san for x in ("-Xarch_host", f)]
    objs, procs = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        procs.append(subprocess.Popen(
            [HIPCC, "--offload-host-only", "-O1", "-g", "-std=c++17"] + san_host + inc
            + ["-c", src, "-o", objs[-1]], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
            text=True))
    for p in procs:
        out, _ = p.communicate()
        assert p.returncode == 0, out[-4000:]
    # empty device code bundles, which the stand-in runtime never reads
    names = set()
    for obj in objs:
        names |= set(re.findall(r"\b(__hip_fatbin_[0-9a-f]+)\b", _run(["nm", "-u", obj])))
    fat = tmp_path / "fatbins.cpp"
    fat.write_text("".join('extern "C" { extern const unsigned char %s[16]; '
                           'const unsigned char %s[16] = {0}; }\n' % (n, n) for n in sorted(names)))
    for src, obj in ((os.path.join(SAN_DIR, "block_checks.cpp"), "block_checks.o"),
                     (os.path.join(SAN_DIR, "hip_stub.cpp"), "hip_stub.o"),
                     (str(fat), "fatbins.o")):
        objs.append(str(tmp_path / obj))
        _run([CLANG, "-O1", "-g", "-std=c++17"] + san + inc + ["-c", src, "-o", objs[-1]])
    exe = str(tmp_path / "block_checks")
    _run([CLANG] + san + objs + ["-o", exe])
    assert "block checks passed" in _run([exe], env=ENV, timeout=300)
