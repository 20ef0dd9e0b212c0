"""The training example's weights change after a step has been captured."""
import pytest
import torch

import mx_gemm_gb300 as fg
from tests import train_ref as ref
from tests.test_gpu_streams import same
from tests.test_gpu_train_layer import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ref.MODES)
def test_a_captured_step_takes_the_new_weights(mode):
    layer, x, dy = make(mode, 300, seed=5)

    def step():
        y, kept = layer.forward(x)
        return (y, kept.balance.loss.view(1), *layer.backward(dy, kept))

    old = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    g = torch.Generator(device="cuda").manual_seed(6)
    for _ in range(2):
        for w in (layer.gate_up, layer.down):
            w += 0.1 * w.std() * torch.randn(w.shape, generator=g, device="cuda")
        layer.update()
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert same(got, step()) and not same(got, old)
    assert fg.get_error() == fg.FG_OK
