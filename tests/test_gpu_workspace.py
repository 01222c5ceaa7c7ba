"""The binding's workspace where a stream is being captured."""
import pytest
import torch

from paged_kv_cache_480_b200 import binding

pytestmark = pytest.mark.gpu


def test_a_workspace_of_a_graph_zeroes_the_counters_alone(monkeypatch):
    """The first 256 bytes at each replay; the rest holds partial results."""
    monkeypatch.setattr(binding, "_workspaces", {})
    dev = torch.device("cuda", torch.cuda.current_device())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ws = binding.default_workspace(dev, 1 << 20)
    assert ws.numel() == 1 << 20 and binding._workspaces == {}
    for _ in range(2):
        ws.fill_(255)
        graph.replay()
        assert (ws[:256] == 0).all() and (ws[256:] == 255).all()


def test_a_workspace_for_a_captured_side_stream(monkeypatch):
    """The stream that a call names is the captured one, not the current one."""
    monkeypatch.setattr(binding, "_workspaces", {})
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        ws = binding.default_workspace(dev, 1 << 20, side)
        torch.cuda.current_stream().wait_stream(side)
    ws.fill_(255)
    graph.replay()
    assert (ws[:256] == 0).all() and binding._workspaces == {}
    torch.cuda.synchronize()
