"""GPU parity of beam selection with the 64-bit reference: parents and tokens
exactly; a score is one 32-bit rounding (2^-24 of itself) of a 64-bit sum whose
normaliser holds 32-bit exponentials (each within 2^-22 of itself)."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    abi.load()
    torch.cuda.set_device(cuda_device)
    return cuda_device


def check(dev, x, scores, finished=None, eos=2, pad=0, ws=None):
    groups, beams = scores.shape
    V = x.shape[1]
    ld = -(-(V + pad) // 4) * 4
    buf = torch.full((x.shape[0], ld), 1e30, device=dev)  # past V: never read as a logit
    buf[:, :V] = torch.from_numpy(x).to(dev)
    f = None if finished is None else torch.from_numpy(finished).to(dev)
    got = abi.beam_select(buf, torch.from_numpy(scores).to(dev), vocab=V, finished=f, eos=eos, workspace=ws)
    torch.cuda.synchronize()
    s, p, t, d = (g.cpu().numpy() for g in got)
    ws_, wp, wt, wd = cache_ref.beam(x, scores.astype(np.float64), finished, eos)
    assert np.array_equal(p, wp), (p, wp)
    assert np.array_equal(t, wt)
    assert np.array_equal(d, wd)
    with np.errstate(invalid="ignore"):
        assert ((np.abs(s - ws_) <= 2.0**-24 * np.abs(ws_) + 2.0**-22) | (s == ws_)).all()
    return s, p, t, d


def draw(seed, groups, beams, V):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((groups * beams, V)) * 2.5).astype(np.float32), \
        (-8 * rng.random((groups, beams))).astype(np.float32)


@pytest.mark.parametrize("groups,beams,V", [
    (1, 1, 1), (1, 1, 7), (1, 4, 3), (2, 3, 5), (1, 8, 1000), (3, 5, 1023), (2, 4, 1024), (2, 4, 1025), (1, 64, 64),
    (1, 64, 2048), (64, 1, 333), (8, 8, 32000), (1, 4, 8192), (1, 4, 8193), (2, 2, 65537), (1, 8, 151936),
    (8, 8, 151936), (1, 2, 1 << 20), (1, 40, 50021)])
def test_matches_reference(dev, groups, beams, V):
    x, s = draw(groups * 1000 + beams + V, groups, beams, V)
    check(dev, x, s, pad=V % 3)


@pytest.mark.parametrize("V", [5, 1000, 40000])
def test_finished_beams(dev, V):
    x, s = draw(V, 4, 4, V)
    f = np.array([[0, 1, 0, 1], [1, 1, 1, 1], [0, 0, 0, 0], [0, 255, 0, 0]], np.uint8)
    check(dev, x, s, f, eos=V - 1)


def test_first_step_from_one_live_beam(dev):
    x, s = draw(1, 2, 4, 500)
    s[:, 1:] = -np.inf
    x[1:4], x[5:] = x[0], x[4]
    got = check(dev, x, s)
    assert (got[1] == [[0] * 4, [4] * 4]).all()


@pytest.mark.parametrize("groups,beams,V", [(1, 4, 20000), (2, 8, 3000), (1, 64, 9000), (1, 1, 8192)])
def test_ties_take_the_lowest_place(dev, groups, beams, V):
    """Constant rows, and rows of a few levels: thousands tie."""
    s = np.zeros((groups, beams), np.float32)
    got = check(dev, np.full((groups * beams, V), 1.5, np.float32), s)
    assert (got[2] == np.arange(beams)).all() and (got[1] == np.arange(groups)[:, None] * beams).all()
    x = np.random.default_rng(0).integers(0, 3, (1, V)).astype(np.float32)
    check(dev, np.repeat(x, groups * beams, 0), s)


def test_masked_logits_and_dead_beams(dev):
    """-inf logits are never taken, a beam of score -inf or NaN neither; too few candidates leave empty places."""
    x = np.full((6, 3000), -np.inf, np.float32)
    x[0, 2999], x[1, 17], x[4, 5], x[4, 6] = 1.0, 2.0, 3.0, 3.0
    s = np.array([[0.0, -1.0, -np.inf], [-np.inf, -2.0, np.nan]], np.float32)
    x[2] = 0.0
    x[3] = 0.0
    x[5] = 0.0
    got = check(dev, x, s)
    assert (got[1][0] == [0, 1, -1]).all() and (got[1][1] == [4, 4, -1]).all() and np.isneginf(got[0][:, 2]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_rows_with_nan_or_inf_have_no_candidate(dev, bad):
    x, s = draw(3, 2, 3, 5000)
    x[1, 4321] = bad
    x[3, 0] = bad
    got = check(dev, x, s)
    assert not np.isin(got[1], [1, 3]).any()


def test_wide_and_low_logits(dev):
    """Rows far from zero, and rows over a wide range, keep their normaliser."""
    x, s = draw(4, 2, 4, 12000)
    x[0] -= 5000
    x[1] += 5000
    x[2] *= 40
    x[3] = -1e30
    x[4, 100] = 3e38
    x[5, 0] = -3e38
    check(dev, x, s)


def test_outputs_may_be_the_inputs_and_workspace_is_left_ready(dev):
    x, s = draw(5, 2, 4, 30000)
    f = np.array([[0, 1, 0, 0], [0, 0, 0, 1]], np.uint8)
    ws = abi.beam_select_workspace(2, 4, 30000, dev)
    a = check(dev, x, s, f, ws=ws)
    X, S, F = torch.from_numpy(x).to(dev), torch.from_numpy(s).to(dev), torch.from_numpy(f).to(dev)
    abi.beam_select(X, S, finished=F, eos=2, scores_out=S, finished_out=F, workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(S.cpu().numpy(), a[0]) and np.array_equal(F.cpu().numpy(), a[3])
    check(dev, *draw(6, 2, 4, 1000), ws=ws)
    check(dev, x, s, f, ws=ws)


def test_two_graphs_at_once(dev):
    """Two captured selections with a workspace each, replayed on two streams over changing logits."""
    sets, graphs = [], []
    for i in range(2):
        x, s = draw(20 + i, 2, 4, 20000 + i * 3001)
        ld = -(-x.shape[1] // 4) * 4
        buf = torch.zeros((8, ld), device=dev)
        S, ws, st = torch.zeros((2, 4), device=dev), abi.beam_select_workspace(2, 4, x.shape[1], dev), torch.cuda.Stream(dev)
        st.wait_stream(torch.cuda.current_stream(dev))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            got = abi.beam_select(buf, S, vocab=x.shape[1], workspace=ws)
        sets.append((x, s, buf, S, got, st))
        graphs.append(g)
    for rnd in range(4):
        for x, s, buf, S, _, _ in sets:
            buf[:, :x.shape[1]] = torch.from_numpy(np.roll(x, rnd, 0)).to(dev)
            S.copy_(torch.from_numpy(s))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, (*_, st) in zip(graphs, sets):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for x, s, _, _, got, _ in sets:
            _, p, t, _ = cache_ref.beam(np.roll(x, rnd, 0), s.astype(np.float64), None, -1)
            assert np.array_equal(got[1].cpu().numpy(), p) and np.array_equal(got[2].cpu().numpy(), t)


def test_helper_refuses(dev):
    x, s = torch.zeros((4, 100), device=dev), torch.zeros((1, 4), device=dev)
    with pytest.raises(abi.Nvfp4Error) as e:
        abi.beam_select(x, s, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    assert e.value.status == abi.NVFP4_ERR_SCRATCH
    for bad in (dict(logits=x.half()), dict(logits=x[:3]), dict(logits=x.t()), dict(scores=s.double()),
                dict(vocab=101), dict(finished=s)):
        kw = dict(logits=x, scores=s)
        kw.update(bad)
        with pytest.raises(ValueError):
            abi.beam_select(**kw)
