"""One-shot calls of the speculative step on a side stream while a graph is
captured: their tensors' memory must not be given out again before the side
stream has joined."""
import pytest
import torch

from gated_deltanet_recurrent_sigmoid_b200 import speculative as spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return spec.load()


def test_tensors_freed_in_a_capture_outlive_the_side_streams_call():
    rows, vocab = 64, 20011
    source = torch.randn(rows, vocab, device="cuda")
    p, side, graph = torch.zeros_like(source), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    spec.token_probs(source, p)
    want = p.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        x = source.clone()
        side.wait_stream(current)
        spec.token_probs(x, p, stream=side)
        at = x.data_ptr()
        del x
        y = torch.empty_like(source)
        again = y.data_ptr() == at
        y.fill_(0)
        current.wait_stream(side)
    assert not again, "memory that the side stream still reads was given out"
    for _ in range(3):
        p.zero_()
        graph.replay()
        assert torch.equal(p, want)
