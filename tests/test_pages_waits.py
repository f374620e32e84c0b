"""The bounded waits of the paged kernels: one that runs out is recorded, and every
warp leaves with its own copies landed."""
import ctypes
import os
import subprocess

import pytest
import torch

from bit_quantized_kv_02_gb300 import build

gpu = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
WARPS, STAGES, STEPS = 4, 3, 9


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("wait") / "libwait_probe.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-shared", os.path.join(HERE, "wait_probe.cu"), "-o", out],
                   check=True, capture_output=True)
    f = ctypes.CDLL(out).wait_probe
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return f


def test_probe_compiles(probe):
    assert probe


@gpu
@pytest.mark.parametrize("lost", [None, (0, 0), (1, 2), (2, 4), (3, 5), (0, 8)])
def test_a_wait_that_runs_out(probe, lost):
    """`lost` = (warp, step) of the copy that never comes: that warp stops there, the
    others have read all of theirs by then or stop as well; copies further on, which
    stand a phase further where the ring begins anew, have landed."""
    src = torch.arange(STEPS * 256, dtype=torch.int32, device="cuda")
    out = torch.zeros(1 + 3 * WARPS, dtype=torch.int32, device="cuda")
    assert probe(src.data_ptr(), *(lost or (-1, -1)), out.data_ptr()) == 0
    err, *rest = out.tolist()
    done, landed, sums = rest[:WARPS], rest[WARPS:2 * WARPS], rest[2 * WARPS:]
    assert err == (2 if lost else 0)
    for w in range(WARPS):
        if lost and w == lost[0]:
            ahead = min(STAGES, STEPS - lost[1])
            assert done[w] == lost[1] and landed[w] == (1 << ahead) - 2
        else:
            assert done[w] == STEPS and landed[w] == 0
        n = done[w] * 256
        assert sums[w] == n * (n - 1) // 2
    # the next call finds everything in order
    out.zero_()
    assert probe(src.data_ptr(), -1, -1, out.data_ptr()) == 0
    assert out.tolist()[:1 + WARPS] == [0] + [STEPS] * WARPS
