"""Host: a move of states takes little of its caller's stack, whatever number of states it may name: 16 KiB at most, as a
thread of a server may have 64 KiB and less."""
import os
import subprocess

from mamba_decode_amd import build as libbuild


def test_frame_of_a_move(tmp_path):
    r = subprocess.run([libbuild.HIPCC, *libbuild.FLAGS, "--offload-host-only", "-Wframe-larger-than=16384", "-c",
                        os.path.join(libbuild.CSRC, "ssq_api.cpp"), "-o", str(tmp_path / "api.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "in 'ssq_state_move'" not in r.stderr, r.stderr[-2000:]
