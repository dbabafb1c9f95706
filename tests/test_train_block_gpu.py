"""The bf16 training step of the example block: dropout and layer norm, the gated
projection, and their backward passes together (GPU).

Bounds, relative to a result's norm.  Every tensor that passes from one operator to
the next is rounded to bf16, off by at most 2^-8 of each value (half a step), some
2^-8 / sqrt(3) of a norm at the most.  out depends on four such roundings in a chain
(h, y, a, out), the gradients on up to nine (those, gate and up, d_a, d_gu, d_y and
themselves), through maps that are near-isometries here but for the activation's
product, which passes two factors' errors on: at most 2 * 9 * 2^-8 / sqrt(3) < 0.041.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"
BOUND = 18 * 2.0**-8 / 3**0.5


@pytest.fixture(scope="module")
def block():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(T, D, H, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *shape, std=1.0: (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()
    return (rand(T, D), rand(T, D), (1 + rand(D, std=0.1).float()).bfloat16(), rand(D, std=0.1), rand(2 * H, D, std=D**-0.5),
            rand(D, H, std=H**-0.5), rand(T, D, std=0.01), rand(T, D, std=0.01))


def rng(*v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("T,D,H", [(512, 1024, 1408), (100, 256, 384), (1, 128, 256), (333, 520, 264)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_step(block, T, D, H, p):
    args = inputs(T, D, H, T + D) + (p, rng(5, T))
    for name, a, b in zip("out d_x d_residual d_w d_b d_Wgu d_Wd".split(), block.train_bf16(*args), block.reference_bf16(*args)):
        err = float((a.float() - b).norm() / b.norm())
        print(T, D, H, p, name, err, flush=True)
        assert err < BOUND, name


def test_captured_steps_draw_new_masks(block):
    # one capture, replayed with the step's number changed on the device, against eager steps
    T, D, H = 96, 256, 384
    args, state = inputs(T, D, H, 3), rng(11, 0)
    eager = []
    for step in (0, 1, 2):
        state.copy_(torch.tensor([11, step]))
        eager.append([t.clone() for t in block.train_bf16(*args, 0.2, state)])
    assert not torch.equal(eager[0][0], eager[1][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # torch's products set themselves up outside a capture
        block.train_bf16(*args, 0.2, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.train_bf16(*args, 0.2, state)
    # torch's own products may add in another order inside the capture: what the library made is compared bit for
    # bit where nothing of torch's comes in front of it, the rest within the bounds
    for step in (0, 1, 2, 1):
        state.copy_(torch.tensor([11, step]))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager[step]):
            assert float((a.float() - b.float()).norm()) <= BOUND * float(b.float().norm())
        eager_again = block.train_bf16(*args, 0.2, state)
        assert all(torch.equal(a, b) for a, b in zip(eager_again, eager[step]))
