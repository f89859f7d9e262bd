"""moe_reader_status around captured and replayed decodes: it waits for a
replay on a stream of its own and clears exactly what it has reported."""

import pytest

from calibration_free_sparse_gb300 import reader as RD
from tests import gpu_common as C

pytestmark = pytest.mark.gpu

H, E, TOPK, I, CC, RANK, K = 256, 16, 2, 128, 80, 8, 32


def test_status_waits_for_a_replay_on_another_stream():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pair = C.Pair(H, E, TOPK, I, CC, RANK, max_batch=4, seed=0)
    x, ids, w = (torch.from_numpy(a).cuda() for a in pair.tokens(2, 5))
    y = torch.empty_like(x)
    good, wrong = ids.clone(), ids.clone()
    wrong[1, 0] = E + 3
    pair.reader.decode(x, ids, w, K, y)
    assert pair.reader.status() == (RD.OK, 0)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pair.reader.decode(x, ids, w, K, y)
    side = torch.cuda.Stream()
    for bad in (True, False, True, False):
        ids.copy_(wrong if bad else good)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)             # some 50 ms
            graph.replay()
        code, bits = pair.reader.status()
        assert (code, bits) == ((RD.EDEVICE, RD.ERR_EXPERT_RANGE) if bad else (RD.OK, 0))
    torch.cuda.synchronize()
    assert pair.reader.status() == (RD.OK, 0)
    assert (y - first).abs().max() <= 1e-4 * first.abs().max()
