"""The bounded wait between the segments of a long sequence whose tokens are kept."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

from bit_quantized_kv_02_gb300 import build

gpu = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
SEGMENT = 128


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("keep") / "libkeep_probe.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-shared", os.path.join(HERE, "keep_probe.cu"), "-o", out],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.keep_probe_bytes.restype = ctypes.c_size_t
    lib.keep_probe.argtypes = [P, I, P, P, P, I, P, I, ctypes.c_ulonglong, P, P, P]
    return lib


def test_probe_compiles(probe):
    assert probe.keep_probe_bytes() > 0


@gpu
@pytest.mark.parametrize("skip", [0, 1, 2])
def test_a_wait_for_a_segment_that_is_not_read_runs_out(probe, skip):
    """600 tokens of which the first goes, so that each segment's tokens move down by one, into the segment before.
    The first `skip` segments are drawn by nobody: the next one waits 30 ms for the last of them, is recorded and
    stays; those behind it find what they wait for and move."""
    n, pages = 600, 38
    number = torch.arange(pages * 16, dtype=torch.int16).view(pages, 1, 16, 1)  # a token's rows hold its number
    pool = torch.cat([number, 1000 + number], dim=1).expand(pages, 2, 16, 64).contiguous().cuda()
    keep = torch.ones(n, dtype=torch.uint8, device="cuda")
    keep[0] = 0
    q_start, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")
    lens_out, err = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.zeros(probe.keep_probe_bytes(), dtype=torch.uint8, device="cuda")

    def run(skip):
        torch.cuda.synchronize()
        t = time.perf_counter()
        assert probe.keep_probe(pool.data_ptr(), pages, q_start.data_ptr(), lens.data_ptr(), table.data_ptr(), n,
                                keep.data_ptr(), skip, 30_000_000, lens_out.data_ptr(), work.data_ptr(), err.data_ptr()) == 0
        assert time.perf_counter() - t < 2.0
        rows = pool.cpu().permute(1, 0, 2, 3).reshape(2, -1, 64)
        assert (rows == rows[:, :, :1]).all() and (rows[1, :, 0] == rows[0, :, 0] + 1000).all()
        return rows[0, :, 0].tolist()

    was = list(range(pages * 16))
    stays = SEGMENT * (skip + 1) - 1 if skip else 0  # places that nothing is written to
    want = was[:stays] + was[stays + 1:n] + was[n - 1:]
    assert run(skip) == want
    assert lens_out.item() == n - 1 and err.item() == (2 if skip else 0)
    # the next call finds everything in order
    err.zero_()
    assert run(0) == want[1:n] + want[n - 1:]
    assert lens_out.item() == n - 1 and err.item() == 0
