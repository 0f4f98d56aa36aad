"""The host code of the short convolution, the selective scan and the norm with
the residual's addition under AddressSanitizer and UndefinedBehaviorSanitizer (CPU):
tests/sanitize/layer_driver.cpp with the library's sources, as
test_linattn_host_sanitizer.py does for the linear attention."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_host_sanitizer import CSRC, ENV, HIPCC, ROOT, SAN_HOST, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_layer_host_code_under_asan_ubsan(tmp_path):
    base = [HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", *SAN_HOST,
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]
    srcs = [os.path.join(CSRC, s) for s in ("ckda_api.cpp", "layer_api.cpp", "short_conv.hip", "selective_scan.hip", "add_norm.hip",
                                            "part_sums.hip")]
    srcs.append(os.path.join(ROOT, "tests", "sanitize", "layer_driver.cpp"))

    def compile_one(path):
        obj = str(tmp_path / (os.path.basename(path) + ".o"))
        return run(base + ["-c", path, "-o", obj]), obj

    with ThreadPoolExecutor(max_workers=7) as ex:
        results = list(ex.map(compile_one, srcs))
    for (rc, out), _ in results:
        assert rc == 0, out[-2000:]
    exe = str(tmp_path / "layer_driver")
    rc, out = run([HIPCC, "--offload-arch=gfx950", *SAN_HOST[:4], *[o for _, o in results],
                   "-Wl,--unresolved-symbols=ignore-in-object-files", "-o", exe])
    assert rc == 0, out[-2000:]
    rc, out = run([exe], env=dict(ENV, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"))
    assert rc == 0 and " 0 failures" in out, out[-3000:]
