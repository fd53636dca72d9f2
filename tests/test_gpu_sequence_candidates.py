"""The example over event sequences with candidates that share a history: training on impressions, caches in 8 bits and
ranking."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402

from ad_recommendation_amd import dense  # noqa: E402
from oracle import dense_oracle as O  # noqa: E402

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


def test_answers_from_8_bits_are_those_of_what_the_cache_holds(example):
    """The example's caches hold each key and value as the nearest code, and the newest events and candidates are answered
    from those values within the roundings of 16 bits."""
    m, rng = example, np.random.default_rng(4)
    model = m.SequenceModel(50, 40, False, seed=3)
    # queries that tell events apart: as they are drawn, all weights are nearly equal
    model.c["qkv"][:, :m.DIM] *= 32
    keys, off, _ = m.batch(rng, rng.standard_normal(50), 40, n_seq=20, longest=90)
    model.forward(keys, off)
    q, k, v = model.saved[2:5]
    lens, cache = off[1:] - off[:-1], m.history_cache(k, v, off)
    kb, vb = torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
    dense.cache_q8_read(*cache, off, None, kb, vb)
    for x, y in ((k, kb), (v, vb)):
        assert torch.equal(y, O.values_of(*O.quantise(x)).to(x.dtype))
    padded = [torch.zeros(20, cache[0].shape[1], m.HEADS, m.HEAD, dtype=k.dtype, device="cuda") for _ in range(2)]
    for s, (b, e) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        padded[0][s, :e - b], padded[1][s, :e - b] = kb[b:e], vb[b:e]
    newest = q[(off[1:] - 1).long()].contiguous()
    o, bound = O.attn_decode(newest, *padded, lens, 40, m.SINKS, model.scale)
    got = model.serve_q8(cache, lens, newest)
    assert ((got.double() - o).abs() <= bound).all()
    c_off = 8 * torch.arange(21, dtype=torch.int32, device="cuda")
    model.forward_candidates(torch.cat([keys, torch.from_numpy(rng.integers(1, 51, 160)).cuda()]), c_off, off)
    q, k, v = model.saved[2:5]
    o, _, bound, _ = O.attn_shared_fwd(q, k, v, kb, vb, c_off, None, off, 40, m.SINKS, model.scale)
    got = model.rank(cache, lens, q, k, v, c_off)
    assert ((got.double() - o).abs() <= bound).all()
    # a bound that binds: equal weights would not pass, nor a window one event longer
    flat = O.attn_shared_fwd(torch.zeros_like(q), k, v, kb, vb, c_off, None, off, 40, m.SINKS, model.scale)[0]
    wide = O.attn_shared_fwd(q, k, v, kb, vb, c_off, None, off, 41, m.SINKS, model.scale)[0]
    for other in (flat, wide):
        assert not ((other - o).abs() <= 2 * bound).all()
    model.table.close()
