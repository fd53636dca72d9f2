"""The example over event sequences with candidates that share a history: training on impressions, caches in 8 bits and
ranking."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402

from ad_recommendation_amd import dense  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sequence_step", os.path.join(ROOT, "examples", "sequence_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("more", [["--candidates", "12"], ["--candidates", "3", "--q8", "--window", "5"]])
def test_training_on_impressions_runs(example, more):
    losses, worst = example.main(["--steps", "4"] + more)
    assert len(losses) == 4 and all(np.isfinite(losses))
    assert worst < 2.0 ** -8  # two roundings of values of about one


@pytest.mark.parametrize("window,longest,most", [(16, 100, 12), (200, 150, 40)])
def test_gradients_against_differences(example, window, longest, most):
    """The hand-written backward of the block over candidates, with 32-bit differences of the loss along random directions
    of every weight, and of the rows of histories and of candidates."""
    m, rng = example, np.random.default_rng(1)
    values = rng.standard_normal(50)
    model = m.SequenceModel(50, window, False, seed=3)
    keys, off, labels, hist = m.candidate_batch(rng, values, window, n_seq=32, longest=longest, most=most)
    x = model.lookup(keys)
    model.lookup = lambda keys: x
    loss = lambda: torch.nn.functional.binary_cross_entropy_with_logits(  # noqa: E731
        model.forward_candidates(keys, off, hist), labels, reduction="sum").item()
    logit = model.forward_candidates(keys, off, hist)
    g, dx = model.backward_candidates(torch.sigmoid(logit) - labels, off, hist)
    gen = torch.Generator().manual_seed(5)

    def check(name, to, keep, grad, d):
        """`to` sets what the loss reads to a value and says what it became."""
        up_at, up = to(keep + d), loss()
        down_at, down = to(keep - d), loss()
        to(keep)
        want = ((up_at - down_at) * grad).sum().item()
        # half-precision activations blur each loss by about 2^-11 of it, and the step is finite
        assert abs((up - down) - want) < 0.05 * abs(want) + 2 * 2.0 ** -11 * up, name

    for name, w in model.w.items():
        def to(value):
            w.copy_(value)
            model.c[name].copy_(w)
            return model.c[name].float() if name in ("qkv", "out", "head", "gate") else w.clone()
        check(name, to, w.clone(), g[name].view_as(w), (torch.randn(w.shape, generator=gen) * 0.02).to(w.device))

    n_hist = int(hist[-1])
    for name, rows in (("histories", slice(0, n_hist)), ("candidates", slice(n_hist, None))):
        def to(value):
            x[rows] = value.half()
            return x[rows].float()
        # along the gradient's signs, where a history's small share of the loss stands above the blur
        keep = x[rows].float()
        check(name, to, keep, dx[rows].float(), dx[rows].float().sign() * 0.004)
    model.table.close()


def test_serving_from_8_bits_stays_near_the_whole_forward(example):
    m, rng = example, np.random.default_rng(2)
    model = m.SequenceModel(50, 40, False, seed=3)
    keys, off, _, hist = m.candidate_batch(rng, rng.standard_normal(50), 40, n_seq=20, longest=90, most=9)
    model.forward_candidates(keys, off, hist)
    _, _, q, k, v, kh, vh, o = model.saved[:8]
    lens = hist[1:] - hist[:-1]
    cache = m.new_cache(20, int(lens.max()))
    dense.cache_q8_write(kh, vh, hist, None, *cache)
    ranked = model.rank(cache, lens, q, k, v, off)
    # an element of a code is off by 2^-4 of itself: a score by delta, a weight by a factor of e^(2 delta)
    delta = 2.0 ** -4 * model.scale * (q.abs().float().amax(0) * kh.abs().float().amax(0)).sum(-1).max()
    most = torch.cat([vh, v]).abs().max().float()
    bound = (2 * torch.expm1(2 * delta) + 2.0 ** -4 + 2.0 ** -9) * most
    assert (ranked.float() - o.float()).abs().max() < bound
    # the newest event from its cache alone: a mean of values, nothing where there is no event
    some = lens > 0
    alone = model.serve_q8(cache, lens, q.new_ones(20, m.HEADS, m.HEAD))
    assert (alone[~some] == 0).all()
    assert alone[some].abs().max() <= (1 + 2.0 ** -4 + 2.0 ** -9) * vh.abs().max()
    model.table.close()
