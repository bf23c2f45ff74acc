"""The host code of the gated recurrence, the group norm and the moves under AddressSanitizer and
UndefinedBehaviorSanitizer, every report fatal: argument checks, plans, workspaces.  Nothing here touches a GPU."""
import glob
import os
import subprocess
import sys

import pytest

from tests.test_sanitized import ROOT, _hip_objects


def test_host_tests_pass_with_the_host_side_sanitized(tmp_path):
    if os.environ.get("LD_PRELOAD"):
        pytest.skip("a library is already preloaded; the sanitizer runtime has to come first")
    found = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not found:
        pytest.skip("no clang AddressSanitizer runtime here")
    libbuild, objs = _hip_objects(tmp_path)
    own = ["ssq_api.cpp", "ssq_gated.hip", "ssq_norm.hip", "ssq_move.hip"]
    objs = [o for o in objs if not any(n.rsplit(".", 1)[0] in os.path.basename(o) for n in own)]
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = [f for f in libbuild.FLAGS if not f.startswith("-O")] + ["-O1", "-g"]
    jobs = []
    for src in own:
        objs.append(str(tmp_path / (src + "_san.o")))
        jobs.append(subprocess.Popen([libbuild.HIPCC, *flags, *host_san, "-c", os.path.join(libbuild.CSRC, src), "-o", objs[-1]],
                                     stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL))
    assert [j.wait() for j in jobs] == [0] * len(own)
    so = str(tmp_path / "libssq_san.so")
    subprocess.check_call([libbuild.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", so])
    env = dict(os.environ, SSQ_LIBRARY=so, LD_PRELOAD=found[0], ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "not gpu", "-p", "no:cacheprovider", "--capture=sys",
                        os.path.join(ROOT, "tests", "test_recurrent_layer_abi.py")], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
    assert " passed" in out
