"""Time-outs of the linear layer's bounded waits, without a fault: a contraction
of 2^20 takes a tile longer than the shortest limit that a layer takes (1 ms), so
the epilogue's wait for its first sums runs out while loads and MMAs go on.

How long a tile takes at least: 8192 blocks of 128 on a CTA pair are 2 x 256 x 256
x 2^20 operations, 2.7 ms at 25 TFLOP/s an SM; 152 tiles of 32 columns, two CTAs to
each, read 20.4 GB of weights, 2.5 ms at 8 TB/s.
"""
import pytest
import torch

from all_mxfp8_block_gb300 import mxa2a
from tests.test_gpu_linear import check_layer, layer_inputs

pytestmark = pytest.mark.gpu

LONG = 1 << 20
MS = 1_000_000
# rows, N: the CTA-pair kernel (40 tiles), and single CTAs that share a tile's contraction
SHAPES = {"pairs": (1024, 2560), "shared": (1, 152 * 128)}


class Case:
    def __init__(self, rows, N):
        zeros = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.rows, self.N = rows, N
        self.layer = mxa2a.Linear(1, rows, N, LONG)
        self.x, self.x_s = zeros(rows, LONG), zeros(LONG // 128, -(-rows // 128), 512)
        self.w, self.w_s = zeros(N, LONG), zeros(LONG // 128, -(-N // 128), 512)
        self.out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()

    def run(self):
        self.layer.run(self.rows, self.x, self.x_s, self.w, self.w_s, self.out, mxa2a.MXA2A_TYPE_BF16)

    def limit(self, ns):
        self.layer.set_option(mxa2a.MXA2A_OPT_TIMEOUT_NS, ns)


@pytest.fixture(params=list(SHAPES))
def case(request):
    c = Case(*SHAPES[request.param])
    yield c
    c.layer.destroy()
    del c.x, c.w
    torch.cuda.empty_cache()


def timed_out(st):
    return st["code"] == mxa2a.MXA2A_ERR_TIMEOUT and st["role"] in (2, 3, 4, 7) and 0 <= st["block"] < 304


def test_time_out_stores_nothing_and_leaves_the_layer_usable(case):
    case.limit(MS)
    case.run()
    torch.cuda.synchronize()
    assert timed_out(case.layer.status())
    # every tile takes longer than the limit: no CTA has sums to store
    assert (case.out == 7.0).all()
    assert case.layer.status()["code"] == 0      # reported once
    case.limit(2000 * MS)
    case.run()
    torch.cuda.synchronize()
    assert case.layer.status()["code"] == 0
    assert (case.out == 0).all()
    check_layer(layer_inputs([300], 256, 256, 1, dense=True))


def test_time_out_of_a_replay_is_reported():
    case = Case(*SHAPES["pairs"])
    case.run()                                   # (kernels are loaded before the capture)
    torch.cuda.synchronize()
    case.limit(MS)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.run()
    assert case.layer.status()["code"] == 0      # nothing has run yet, and the status has been read
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert timed_out(case.layer.status())    # every replay's own
        assert case.layer.status()["code"] == 0  # and once
    # a run of the layer itself between two replays does not hide the second one's
    case.limit(2000 * MS)
    case.run()
    torch.cuda.synchronize()
    assert case.layer.status()["code"] == 0
    g.replay()
    torch.cuda.synchronize()
    assert timed_out(case.layer.status())
