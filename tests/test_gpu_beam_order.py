"""The order of beam_select where logits lie as near to one another as their type allows, over several chunks of a row."""
import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_beam import BF16, FP16, FP32, check

pytestmark = pytest.mark.gpu


def neighbours(vocab, dtype, level, n, rising=True, seed=0):
    """A row [vocab] far below `level`, but for n neighbouring numbers of the type from `level` on, at places all over the row: rising
    with the place, so that a chunk's best is always behind it, or in no order.  Every third one comes twice."""
    rng = np.random.default_rng(seed)
    words = torch.int32 if dtype == FP32 else torch.int16
    best = (torch.tensor([level], dtype=dtype).view(words) + torch.arange(n, dtype=words)).view(dtype)
    at = np.sort(rng.choice(vocab, n, replace=False))
    if not rising:
        at = rng.permutation(at)
    x = torch.tensor(-5.0 - 3.0 * rng.random(vocab), dtype=torch.float32).to(dtype)
    x[torch.tensor(at)] = best
    twice = np.setdiff1d(rng.choice(vocab, n // 3, replace=False), at)
    x[torch.tensor(twice)] = best[::3][:len(twice)]
    return x.cuda()


# Levels where a step of the type, 2^-37 and 2^-33 at most, is below 2^-35 of the total and above fp64's step at it: the oracle in 64 bits
# tells all totals apart, and orders them.
@pytest.mark.parametrize("dtype,level,score", [(FP32, 1e-4, -2.0), (FP32, 1e-3, -20.0), (FP32, 1e-3, -100.0), (FP32, 1e-3, -1e5), (FP32, 0.01, -1000.0),
                                               (FP32, 0.05, -1000.0), (FP32, 1.0, -1e5), (BF16, 1e-9, -2.0), (BF16, 1e-8, -100.0)])
@pytest.mark.parametrize("vocab", [40000, 100003])
def test_neighbouring_logits(dtype, level, score, vocab):
    """Counts below, equal to and above the number of neighbours."""
    s = torch.tensor([[score]], device="cuda")
    for rising in (True, False):
        x = neighbours(vocab, dtype, level, 48, rising)[None, None]
        for count in (5, 17, 48, 64):
            check(x, s, count)


@pytest.mark.parametrize("level,score", [(1e-4, -2.0), (1e-3, -20.0), (0.05, -1000.0)])
def test_neighbouring_logits_of_equal_beams(level, score):
    """Equal totals go to the lowest beam, nearly equal ones to the larger."""
    x = neighbours(50001, FP32, level, 12)
    for scores in ([score] * 4, [score, np.nextafter(np.float32(score), np.float32(0)), score, np.nextafter(np.float32(score), np.float32(2 * score))]):
        for count in (3, 16, 48, 64):
            check(x.expand(3, 4, 50001), torch.tensor(scores, device="cuda")[None].expand(3, 4).contiguous(), count)
    other = torch.stack([neighbours(50001, FP32, level, 12, False, i) for i in range(4)])
    for count in (3, 16, 48, 64):
        check(other[None], torch.full((1, 4), score, device="cuda"), count)


@pytest.mark.parametrize("dtype,level", [(FP32, 1e-6), (FP32, 1e-20), (FP32, 1e-40), (BF16, 1e-12), (BF16, 1e-30), (FP16, 1e-7)])
@pytest.mark.parametrize("score", [-1e5, -1e20, 0.0])
def test_logits_that_64_bits_do_not_tell_apart_once_summed(dtype, level, score):
    """Totals may be equal in 64 bits; within a beam the order is that of the logits all the same, then of the tokens."""
    for rising in (True, False):
        x = neighbours(70001, dtype, level, 48, rising)
        v = x.float().cpu().numpy().astype(np.float64)
        order = np.lexsort((np.arange(v.size), -v))
        for count in (5, 48, 64):
            best, beams, tokens = tkv.beam_select(x[None, None], torch.tensor([[score]], device="cuda"), count=count)
            assert np.array_equal(tokens[0].cpu().numpy(), order[:count]) and (beams == 0).all()
            assert (best[0, :-1] >= best[0, 1:]).all()


def test_many_equal_candidates():
    """Beams that are all alike, of logits that are all alike: the lowest beam's lowest tokens; and so behind a few that are better."""
    for beams, vocab in ((64, 50000), (8, 131072), (64, 300)):
        x, s = torch.zeros(2, beams, vocab, device="cuda"), torch.full((2, beams), -3.0, device="cuda")
        for count in (1, 8, 64):
            check(x, s, count)
        x[0, beams // 2, vocab // 3], x[1, beams - 1, vocab - 1] = 2.0, 2.0
        for count in (1, 8, 64):
            check(x, s, count)
    done = torch.zeros(1, 64, dtype=torch.bool, device="cuda")
    done[0, ::2] = True
    check(torch.zeros(1, 64, 1, device="cuda"), torch.zeros(1, 64, device="cuda"), 64, done, 0)      # every total is 0, of either kind
    check(torch.zeros(1, 64, 1, device="cuda"), torch.zeros(1, 64, device="cuda") * (1 - 2 * done.float()), 64, done, 0)   # or -0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scores", [[-3e38, 0.0, -1e30, -7.0], [3e38, -3e38, 3.4e38, 0.0], [-1e9, -1e9, 0.0, -1e9], [-3.4028234e38] * 4, [1e-40, -1e-40, 0.0, -0.0]])
def test_scores_of_any_size(dtype, scores):
    """Totals that 64 bits cannot tell apart go by beam, then logit, then token; one below the lowest fp32 number is none."""
    g = torch.Generator("cuda").manual_seed(2)
    x = (torch.randn(2, 4, 30011, generator=g, device="cuda") * 2.5).to(dtype)
    s = torch.tensor([scores] * 2, device="cuda")
    v, w = x.double().cpu().numpy(), s.double().cpu().numpy()
    log_p = v - v.max(-1, keepdims=True)
    total = w[..., None] + (log_p - np.log(np.exp(log_p).sum(-1, keepdims=True)))
    for count in (1, 8, 64):
        best, beams, tokens = (t.cpu().numpy() for t in tkv.beam_select(x, s, count=count))
        for b in range(2):
            beam, token = np.divmod(np.arange(4 * 30011), 30011)
            order = np.lexsort((token, -v[b].ravel(), beam, -total[b].ravel()))[:count]
            order = order[total[b].ravel()[order] > -(2.0 ** 128 - 2.0 ** 103)]
            n = len(order)
            assert np.array_equal(beams[b, :n], beam[order]) and np.array_equal(tokens[b, :n], token[order])
            assert (beams[b, n:] == -1).all() and (tokens[b, n:] == -1).all() and np.isneginf(best[b, n:]).all()
            # the logarithm's 2^-20, the sum's half a step
            assert np.all(np.abs(best[b, :n] - total[b].ravel()[order]) <= 2.0 ** -20 + 2.0 ** -24 * np.abs(total[b].ravel()[order]))
