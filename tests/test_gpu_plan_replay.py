"""Device time-outs of a plan's captured runs: every replay reports its own, once,
and a replay after a time-out that has been read runs like the first."""
import pytest
import torch

from all_mxfp8_block_gb300 import inputs, mxa2a
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


def test_time_out_of_a_replay_is_reported():
    w = inputs.Workload("replayfault", 2, 512, 256, 512, 64, 2, 53)
    x = inputs.make_inputs(w)
    d = gu.to_device(x)
    with mxa2a.Plan(w.R, w.M, w.kPerRank, w.N, w.commMSize, w.buffer_num) as p:
        p.set_option(mxa2a.MXA2A_OPT_SPLIT_K, 1)
        gu.run_gpu(p, d, w.M, w.N)                                     # (kernels are loaded before the capture)
        torch.cuda.synchronize()
        p.set_option(mxa2a.MXA2A_OPT_TIMEOUT_NS, 100_000_000)
        p.set_option(mxa2a.MXA2A_OPT_FAULT_SKIP_STEP, 3)
        C = torch.full((w.M, w.N), -1, dtype=torch.int16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            p.run(d["A_seg"], d["A_scale_seg"], d["B"], d["B_scale"], C, side)
        assert p.status()["code"] == 0                                 # nothing has run yet, and the status has been read
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            st = p.status()
            assert st["code"] == mxa2a.MXA2A_ERR_TIMEOUT and st["launch"] == 2, st
            assert p.status()["code"] == 0
        p.set_option(mxa2a.MXA2A_OPT_FAULT_SKIP_STEP, -1)
        C = gu.run_gpu(p, d, w.M, w.N)
        torch.cuda.synchronize()
        assert p.status()["code"] == 0
        got = gu.host_bits(C)
    gu.assert_parity(got, gu.oracle_full(x), "after the replays")
