"""A released request's place in DecodeAttention is as it was at the start, its adapter too."""
import pytest
import torch

from tests.test_decode_step_gpu import i32, tokens
from tests.test_decode_step_serving_gpu import layer

pytestmark = pytest.mark.gpu


def test_no_adapter_is_inherited(cuda_lib):
    """A request admitted where one with an adapter was released runs without one; the others keep theirs."""
    bs = cuda_lib
    (a, gen), (b, _) = layer(bs), layer(bs)
    x, y = tokens(9, gen), tokens(6, gen)
    for s in (a, b):
        s.which.copy_(i32([1, 0, 1]))
        s.step(x, i32([3, 4, 2]), 4)
    a.release(i32([0, 1, 0]))
    assert a.which.tolist() == [1, -1, 1] and a.lens.tolist() == [3, 0, 2]
    b.release(i32([0, 5, 0]))
    b.which.copy_(i32([1, -1, 1]))
    assert torch.equal(a.step(y, i32([1, 4, 1]), 4), b.step(y, i32([1, 4, 1]), 4))
    assert bs.device_status()[0] == bs.BS_OK


def test_released_in_a_graph(cuda_lib):
    bs = cuda_lib
    a, gen = layer(bs)
    done = i32([0, 0, 0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.release(done)
    for now, which in (([1, 0, 0], [-1, 0, 1]), ([0, 1, 1], [1, -1, -1]), ([0, 0, 0], [1, 0, 1])):
        a.which.copy_(i32([1, 0, 1]))
        done.copy_(i32(now))
        g.replay()
        assert a.which.tolist() == which
    assert bs.device_status()[0] == bs.BS_OK
