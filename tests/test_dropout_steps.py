"""The masks that the example's training step asks for: the same in the forward and
the backward pass, and no two alike among the dropouts of all steps (CPU only: the
library's calls are recorded, and the oracle makes the masks)."""

import importlib.util
import os

import pytest
import torch

import ln64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, D, H, P = 64, 96, 128, 0.25


class Recorder:
    """Takes the library's place: keeps each call's offset, and drops as the library does."""

    def __init__(self):
        self.offsets = []

    def layer_norm_quant(self, *args, offset=0, **named):
        self.offsets.append(("norm", offset))

    def layer_norm_bwd(self, *args, offset=0, **named):
        self.offsets.append(("norm", offset))

    def dropout_add(self, x, out, p, rng, residual=None, offset=0):
        self.offsets.append(("activation", offset))
        out.copy_(ln64.stream(x, residual, p, rng.tolist(), offset))

    def __getattr__(self, name):
        return lambda *args, **named: None


@pytest.fixture
def block(monkeypatch):
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    monkeypatch.setattr(module, "sq", Recorder())
    return module


def offsets(block):
    zeros = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    args = zeros(T, D), zeros(T, D), zeros(D), zeros(D), zeros(2 * H, D), zeros(D, H), zeros(T, D), zeros(T, D)
    block.train_bf16(*args, P, torch.tensor([5, 9]))
    forward, backward = block.sq.offsets[:2], block.sq.offsets[2:]
    assert [name for name, _ in forward] == ["norm", "activation"] and backward == forward[::-1]
    block.sq.offsets = []
    block.reference_bf16(*args, P, torch.tensor([5, 9]))
    assert [o for _, o in block.sq.offsets] == [o for _, o in forward]
    block.sq.offsets = []
    return [o for _, o in forward]


def test_no_two_dropouts_share_a_counter(block):
    steps = list(range(1000)) + list(range(2**32 - 1000, 2**32))
    both = offsets(block)
    used = [(step + o) % 2**64 for step in steps for o in both]
    assert len(set(used)) == len(used)


def test_masks_of_neighbouring_steps_are_independent(block):
    norm, activation = offsets(block)
    n = T * D
    for step in range(4):
        for later in range(1, 4):
            a = ~ln64.kept((7, step), T, D, P, activation)
            b = ~ln64.kept((7, step + later), T, D, P, norm)
            # both drop with probability p^2: five standard deviations
            assert abs(float((a & b).double().mean()) - P * P) <= 5 * (P * P * (1 - P * P) / n) ** 0.5, (step, later)
