"""Beam selection where candidates of different beams nearly tie.  A row's normaliser is a sum of 32-bit exponentials,
off by at most 2^-16:
  an exponential 2^-22 of itself; its argument y (log2, below the maximum) 2^-22.7 of itself (the subtraction, the
  product and the constant log2(e)), which over a row of V <= 2^20 logits comes to at most 20 ln 2 2^-22.7 of the sum (the
  mean of |y| under the weights is at most log2 V), 2^-18.9;
  a thread's sum, up to 43 rounds of 16: 6 + 2 x 43 roundings of 2^-24, and up to 43 rescales by an exponential of
  2^-22, 2^-16.6; the joins of warps and slices some 2^-21 more.
So candidates 2^-15 apart rank as in 64 bits, and those of one beam always."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi

pytestmark = pytest.mark.gpu

GAP = 2.0**-15


@pytest.fixture(scope="module")
def dev(cuda_device):
    abi.load()
    torch.cuda.set_device(cuda_device)
    return cuda_device


@pytest.fixture(autouse=True)
def status(dev):
    ch.clean_status()
    yield
    assert ch.clean_status() == 0


def rows(kind, V, seed):
    """Two rows whose normalisers come about differently."""
    rng = np.random.default_rng(seed)
    a, b = rng.standard_normal(V) * 2.5, rng.standard_normal(V) * 2.5
    if kind == "alike":  # every logit the same
        a[:], b[:] = 0.7, -3.3
    elif kind == "rising":  # a new maximum in every round of every thread
        a, b = np.linspace(-9, 3, V), np.linspace(4, -8, V)
    elif kind == "low":  # most of the sum lies far below the maximum
        a[:], b[:] = -13.0, -13.7
        a[V // 3], b[V // 5] = 0.0, 0.0
    elif kind == "shuffled":
        b = rng.permutation(a)
    a[V // 2], b[V // 7] = a.max() + 0.5, b.max() + 0.25  # one best candidate each
    return np.stack([a, b]).astype(np.float32)


def lse(x):
    x = x.astype(np.float64)
    return x.max(1) + np.log(np.exp(x - x.max(1, keepdims=True)).sum(1))


@pytest.mark.parametrize("kind", ["drawn", "alike", "rising", "low", "shuffled"])
@pytest.mark.parametrize("V,groups", [(50, 1), (5003, 1), (151936, 8), (1 << 20, 1), (1 << 20, 32)])
def test_candidates_of_two_beams_a_gap_apart(dev, kind, V, groups):
    x = rows(kind, V, V)
    best = x.max(1).astype(np.float64) - lse(x)
    d = torch.from_numpy(x).to(dev).repeat(groups, 1)
    pad = torch.zeros((2 * groups, -(-V // 4) * 4), device=dev)
    pad[:, :V] = d
    for sign in (1, -1):
        # the second beam's score puts its best candidate a gap above or below the first one's (rounded to 32 bits: a
        # score of below 32 is off by at most 2^-20)
        s = np.array([[0.0, best[0] - best[1] + sign * (GAP + 2.0**-19)]], np.float32)
        want = cache_ref.beam(x, s.astype(np.float64), None, -1)
        assert abs(s[0, 1] + best[1] - best[0]) >= GAP and abs(s[0, 1]) < 32
        assert want[1][0, 0] == (1 if sign > 0 else 0) and want[1][0, 1] == (0 if sign > 0 else 1)
        got = abi.beam_select(pad, torch.from_numpy(np.repeat(s, groups, 0)).to(dev), vocab=V)
        p, t, sc = got[1].cpu().numpy(), got[2].cpu().numpy(), got[0].cpu().numpy()
        assert (p - 2 * np.arange(groups)[:, None] == want[1]).all() and (t == want[2]).all()
        assert (np.abs(sc - want[0]) <= 2.0**-24 * np.abs(want[0]) + 2.0**-16).all()


@pytest.mark.parametrize("V", [1000, 151936])
def test_one_beam_ranks_by_its_logits(dev, V):
    """Neighbouring 32-bit logits of one beam, and two beams of the same row, whose normalisers are the same."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((1, V)) * 2).astype(np.float32)
    top = np.float32(9.0)
    places = rng.permutation(V)[:8]
    for i in places:
        x[0, i] = top
        top = np.nextafter(top, np.float32(10), dtype=np.float32)
    two = torch.from_numpy(np.repeat(x, 2, 0)).to(dev)
    pad = torch.zeros((2, -(-V // 4) * 4), device=dev)
    pad[:, :V] = two
    got = abi.beam_select(pad[:1], torch.zeros((1, 1), device=dev), vocab=V)
    assert got[2].item() == places[-1]
    got = abi.beam_select(torch.cat([pad] * 4), torch.zeros((1, 8), device=dev), vocab=V)
    # eight beams alike: the best logit of each, in their order
    assert got[1].tolist() == [list(range(8))] and got[2].tolist() == [[int(places[-1])] * 8]
    s = torch.full((1, 8), -float("inf"), device=dev)
    s[0, 3] = -1.0
    got = abi.beam_select(torch.cat([pad] * 4), s, vocab=V)
    assert got[1].tolist() == [[3] * 8] and got[2].tolist() == [[int(i) for i in places[::-1]]]
