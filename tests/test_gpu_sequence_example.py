"""The example over event sequences: lookup, block, backward, both updates and serving together.  Its
loss can only fall if what attention read reaches the score and every gradient its weight."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("more", [[], ["--q8"]], ids=["fp32_states", "8_bit_states"])
def test_training_steps_lower_the_loss_and_serving_agrees(more):
    spec = importlib.util.spec_from_file_location("sequence_step", os.path.join(ROOT, "examples", "sequence_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, worst = m.main(["--steps", "150"] + more)
    assert sum(losses[:5]) / 5 > 0.6        # about log 2 at first
    assert sum(losses[-5:]) / 5 < 0.5
    assert worst < 2.0 ** -8                # two roundings of values of about one


def test_gradients_of_the_whole_block_against_differences():
    """The block's hand-written backward, with 32-bit differences of the loss along random directions."""
    spec = importlib.util.spec_from_file_location("sequence_step", os.path.join(ROOT, "examples", "sequence_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    import numpy as np
    rng = np.random.default_rng(1)
    values = rng.standard_normal(50)
    model = m.SequenceModel(50, 16, False, seed=3)
    keys, off, labels = m.batch(rng, values, 16, n_seq=32)
    loss = lambda: torch.nn.functional.binary_cross_entropy_with_logits(  # noqa: E731
        model.forward(keys, off), labels, reduction="sum").item()
    logit = model.forward(keys, off)
    g, _ = model.backward(torch.sigmoid(logit) - labels, off)
    gen = torch.Generator().manual_seed(5)
    for name, w in model.w.items():
        d = (torch.randn(w.shape, generator=gen) * 0.02).to(w.device)
        keep, keep_c = w.clone(), model.c[name].clone()
        w.copy_(keep + d)
        model.c[name].copy_(w)
        up_w, up = (model.c[name].float() if name in ("qkv", "out", "head", "gate") else w.clone()), loss()
        w.copy_(keep - d)
        model.c[name].copy_(w)
        down_w, down = (model.c[name].float() if name in ("qkv", "out", "head", "gate") else w.clone()), loss()
        w.copy_(keep)
        model.c[name].copy_(keep_c)
        want = ((up_w - down_w) * g[name].view_as(w)).sum().item()
        # half-precision activations blur each loss by about 2^-11 of it, and the step is finite
        assert abs((up - down) - want) < 0.05 * abs(want) + 2 * 2.0 ** -11 * up, name
    model.table.close()
