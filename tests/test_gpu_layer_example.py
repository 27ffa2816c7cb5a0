"""The example layer (examples/gated_delta_layer.py) runs its operators together:
training lowers the loss, the gradient is that of differences, and decoding from
prefilled states gives what the whole sequence gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_rnn_state_gb300 import _build

    _build.build()
    spec = importlib.util.spec_from_file_location("gated_delta_layer", os.path.join(ROOT, "examples", "gated_delta_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_training_lowers_the_loss(example, dtype):
    torch.manual_seed(0)
    model = example.Model(dtype=dtype).cuda()
    losses = example.train(model, 60)
    assert all(l == l for l in losses)
    assert losses[-1] < 0.8 * losses[0], (losses[0], losses[-1])


def test_gradient_against_differences(example):
    """The loss's slope along a random direction of all parameters, by central
    differences: fp32 losses of order 3 (rounding about 1e-6) over steps of 1e-2
    give the slope to about 1e-4, and the curvature term is of order 1e-4 too."""
    torch.manual_seed(1)
    model = example.Model(dtype=torch.float32, layers=1).cuda()
    tokens = torch.randint(0, 32, (4, 70), device="cuda")

    def loss():
        logits, states = model(tokens)
        return torch.nn.functional.cross_entropy(logits[:, 1:].flatten(0, 1), tokens[:, :-1].flatten()) + 1e-2 * states[0].square().mean()

    loss().backward()
    params = [p for p in model.parameters() if p.grad is not None]
    way = [torch.randn_like(p) for p in params]
    size = sum(w.square().sum() for w in way).sqrt()
    slope = sum((p.grad * w).sum() for p, w in zip(params, way)) / size
    at = []
    with torch.no_grad():
        for s in (1e-2, -1e-2):
            for p, w in zip(params, way):
                p += s * w / size
            at.append(float(loss()))
            for p, w in zip(params, way):
                p -= s * w / size
    measured = (at[0] - at[1]) / 2e-2
    assert abs(measured - float(slope)) <= 5e-4 + 1e-2 * abs(float(slope)), (measured, float(slope))


@pytest.mark.parametrize("dtype,bar", [(torch.float32, 2e-4), (torch.bfloat16, 0.3)], ids=["f32", "bf16"])
def test_decoding_is_the_whole_sequence(example, dtype, bar):
    """Logits of order 3; in bfloat16 each of some ten roundings of 2^-8 moves them."""
    torch.manual_seed(2)
    model = example.Model(dtype=dtype).cuda()
    assert example.serve(model) <= bar
