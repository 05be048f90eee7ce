"""The attention's range: values near bf16's largest and very small ones, under
scores that rise from tile to tile and under scores of any size.  Bounds as in
test_gpu_attn; where the scores are exact in 32 bits, without the scores' error."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi
from test_gpu_attn import compare

pytestmark = pytest.mark.gpu

# rows and query heads (one cached head): blocks of 16, of 128 and of 256 query rows (heads of 256: 16 and 128)
BLOCKS = [(3, 4), (32, 4), (40, 4)]


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


def lane(dev, rng, n, rows, dim, keys, values, q, scale):
    """One lane whose slot t has keys[t] and values[t]; (out, lse) checked, and finite."""
    c, r = ch.make(dev, 1, [n], [rows], hkv=1, page=16, dim=dim)
    t = np.arange(n + rows)
    p, o = r.table[0, t // r.page], t % r.page
    r.k[0, p, 0, o], r.v[0, p, 0, o] = cache_ref.bf16_bits(keys), cache_ref.bf16_bits(values)
    c = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    q = ch.dev_bf16(cache_ref.bf16_bits(q), dev)
    out, lse = abi.attn_tree(c, 0, q, scale, row_start=ch.ints([0, rows], dev), max_nodes=rows, want_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    compare(c, r, q, scale, [0, rows], None, out, lse)
    return r, q, out, lse


def large(rng, shape):
    """Up to 3e38, of one sign in the first half of a head and of either in the second."""
    v = rng.uniform(0.4, 1.0, shape) * 3e38
    v[..., shape[-1] // 2:] *= rng.choice([-1.0, 1.0], shape[:-1] + (shape[-1] - shape[-1] // 2,))
    return v


@pytest.mark.parametrize("rise", [0, 6, 20, 31, 90])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim", [(300, 64), (300, 128), (300, 256), (9000, 128), (9000, 256)])
def test_large_values_under_rising_scores(dev, n, dim, rows, hq, rise):
    """Half the slots' scores lie `rise` above the others' in log2: references that hold, and references that rise."""
    rng = np.random.default_rng(rise)
    top = np.where(np.arange(n + rows) >= n // 2, rise * np.log(2.0), 0.0) + 0.3 * rng.standard_normal(n + rows)
    keys = np.repeat(top[:, None], dim, 1)
    lane(dev, rng, n, rows, dim, keys, large(rng, (n + rows, dim)), np.ones((rows, hq, dim)), 1.0 / dim)


@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("dim", [64, 256])
def test_the_largest_values_alike(dev, dim, rows, hq):
    """All scores and all values alike, the largest of bf16: the result is that value."""
    n = 5000
    v = np.full((n + rows, dim), 2.0**127 * (2 - 2.0**-7))
    _, _, out, _ = lane(dev, None, n, rows, dim, np.zeros((n + rows, dim)), v, np.ones((rows, hq, dim)), 1.0)
    assert (out.float() >= 2.0**127 * (2 - 2.0**-6)).all()


@pytest.mark.parametrize("power", [20, 26, 33, 60])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim", [(0, 128), (300, 64), (300, 256), (9000, 128)])
def test_large_values_under_scores_of_any_size(dev, n, dim, rows, hq, power):
    """Scores of some 2^power for every second row."""
    rng = np.random.default_rng(power)
    q = rng.standard_normal((rows, hq, dim))
    q[::2] *= 2.0**power
    lane(dev, rng, n, rows, dim, rng.standard_normal((n + rows, dim)), large(rng, (n + rows, dim)), q, 0.1)


@pytest.mark.parametrize("small", [2.0**-90, 2.0**-60, 2.0**60])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("dim", [128, 256])
def test_small_and_middling_values(dev, dim, rows, hq, small):
    n = 700
    rng = np.random.default_rng(3)
    r, q, out, _ = lane(dev, rng, n, rows, dim, rng.standard_normal((n + rows, dim)),
                        rng.standard_normal((n + rows, dim)) * small, rng.standard_normal((rows, hq, dim)), dim**-0.5)
    # (compare allows 1e-38 in any case: of the size of none of these)
    assert out.float().abs().max() > small * 0.05


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("step", [2.0**-12, 0.5, 4.0, 64.0])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim,power", [(100, 64, 12), (1000, 128, 90), (9000, 128, -30), (600, 256, 12)])
def test_large_scores_that_are_exact(dev, n, dim, power, rows, hq, step, sign):
    """Products 2^power + 2^(power - 22) j, j up to 59, exact in 32 bits with every partial sum, times a scale that makes
    them 2^22 step + j step.  Two scores' difference is then known to 2^-23 of itself (the scale is rounded twice), and
    where differences of logarithms pass some 2^7 a weight is next to nothing; below 2^12 a score in log2 may be rounded
    itself, by 2^-12 at the most.  So weights are off by 2^-11 at the most, however large the scores are."""
    rng = np.random.default_rng(int(step * 4096))
    total = n + rows
    j = rng.integers(0, 30, total) + (np.arange(total) >= n // 2) * 30  # another maximum half way
    keys, q = np.zeros((total, dim)), np.zeros((rows, hq, dim))
    keys[:, 0], keys[:, 1] = 2.0 ** (power // 2), j
    q[:, :, 0], q[:, :, 1] = sign * 2.0 ** (power - power // 2), 2.0 ** (power - 22)
    values = rng.standard_normal((total, dim))
    r, _, out, lse = lane(dev, rng, n, rows, dim, keys, values, q, step * 2.0 ** (22 - power))
    slots = np.array([r.where(0, t) for t in range(total)])
    v = cache_ref.bf16_value(r.v[0, slots[:, 0], 0, slots[:, 1]]).astype(np.float64)
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    for i in range(rows):
        m = n + i + 1
        s = step * j[:m]
        w = np.exp(s - s.max())
        want, wabs = w @ v[:m] / w.sum(), w @ np.abs(v[:m]) / w.sum()
        tol = wabs * (2.0**-8 + 2.0**-11 + 2 * m * 2.0**-24) * 1.01 + np.abs(want) * 2.0**-8 * 1.01
        assert (np.abs(got[i] - want) <= tol).all(), (i, np.max(np.abs(got[i] - want) / tol))
        base = sign * step * 2.0**22
        assert np.abs(gl[i] - (base + s.max() + np.log(w.sum()))).max() <= 2.0**-21 * (abs(base) + 100)


@pytest.mark.parametrize("pattern", ["up", "down", "hump", "dip", "below", "one step"])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim", [(9000, 64), (9000, 128), (9000, 256), (700, 128)])
def test_scores_from_far_below_zero_to_far_above(dev, n, dim, rows, hq, pattern):
    """Scores of steps of 64 over some thousands to either side of zero plus halves up to 3.5, exact in 32 bits: the
    references of one pair's parts are large negative, ordinary and large positive ones.  Bounds as above: the weights
    that count lie within 30 of the largest, whose own size is at most 2^15."""
    rng = np.random.default_rng(7)
    total = n + rows
    x = np.linspace(-1.0, 1.0, total)
    level = {"up": x, "down": -x, "hump": 1 - 2 * abs(x), "dip": 2 * abs(x) - 1, "below": x / 2 - 0.75,
             "one step": np.where(x < 0.1, -0.9, 0.9)}[pattern]
    a, j = np.round(level * 190), rng.integers(0, 8, total)
    keys, q = np.zeros((total, dim)), np.zeros((rows, hq, dim))
    keys[:, 0], keys[:, 1] = a, j
    q[:, :, 0], q[:, :, 1] = 64.0, 0.5
    q[1::2, :, 0] *= -1.0
    values = rng.standard_normal((total, dim))
    r, _, out, lse = lane(dev, rng, n, rows, dim, keys, values, q, 1.0)
    slots = np.array([r.where(0, t) for t in range(total)])
    v = cache_ref.bf16_value(r.v[0, slots[:, 0], 0, slots[:, 1]]).astype(np.float64)
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    for i in range(rows):
        m = n + i + 1
        s = (64.0 if i % 2 == 0 else -64.0) * a[:m] + 0.5 * j[:m]
        w = np.exp(s - s.max())
        want, wabs = w @ v[:m] / w.sum(), w @ np.abs(v[:m]) / w.sum()
        tol = wabs * (2.0**-8 + 2.0**-11 + 2 * m * 2.0**-24) * 1.01 + np.abs(want) * 2.0**-8 * 1.01
        assert (np.abs(got[i] - want) <= tol).all(), (i, np.max(np.abs(got[i] - want) / tol))
        top = s.max() + np.log(w.sum())
        assert np.abs(gl[i] - top).max() <= 2.0**-21 * (abs(top) + 100)


@pytest.mark.parametrize("power", [3, 6, 10, 18, 40])
@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim", [(0, 128), (100, 64), (300, 256), (9000, 128)])
def test_a_row_does_not_depend_on_the_others(dev, n, dim, rows, hq, power):
    """Bit for bit, whatever the scores of the rows beside it: theirs times 2^power, and values that they alone see."""
    rng = np.random.default_rng(9)
    c, r = ch.make(dev, 9, [n], [rows], hkv=1, page=16, dim=dim)
    x = rng.standard_normal((rows, hq, dim))
    mask = [1 << i | 1 for i in range(rows)]
    kw = dict(row_start=ch.ints([0, rows], dev), mask=ch.words(mask, dev), max_nodes=rows, want_lse=True)
    out, lse = abi.attn_tree(c, 0, ch.dev_bf16(cache_ref.bf16_bits(x), dev), dim**-0.5, **kw)
    x[1::2] *= 2.0**power
    for i in range(1, rows, 2):
        p, o = r.where(0, n + i)
        r.v[0, p, 0, o] = cache_ref.bf16_bits(np.full(dim, 3e38))
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    out2, lse2 = abi.attn_tree(c2, 0, ch.dev_bf16(cache_ref.bf16_bits(x), dev), dim**-0.5, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out[::2], out2[::2]) and torch.equal(lse[::2], lse2[::2])
    assert torch.isfinite(out2).all() and torch.isfinite(lse2).all()


@pytest.mark.parametrize("rows,hq", BLOCKS)
@pytest.mark.parametrize("n,dim", [(0, 128), (300, 64), (300, 256), (9000, 128)])
def test_scores_at_the_end_of_the_range(dev, n, dim, rows, hq):
    """Scores of 1.34375 2^127 of either sign (3.3e38 in log2, next to the largest of 32 bits), all alike: the mean of the
    values a row sees.  Beside them rows of scores 0."""
    rng = np.random.default_rng(5)
    total = n + rows
    keys, q = np.zeros((total, dim)), np.zeros((rows, hq, dim))
    keys[:, 0] = 1.34375 * 2.0**63
    q[:, :, 0] = (2.0**64 * np.array([1.0, -1.0, 0.0]))[np.arange(rows) % 3][:, None]
    values = rng.standard_normal((total, dim))
    r, _, out, lse = lane(dev, rng, n, rows, dim, keys, values, q, 1.0)
    t = np.arange(total)
    v = cache_ref.bf16_value(r.v[0, r.table[0, t // r.page], 0, t % r.page]).astype(np.float64)
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    for i in range(rows):
        m = n + i + 1
        want, wabs = v[:m].mean(0), np.abs(v[:m]).mean(0)
        assert (np.abs(got[i] - want) <= wabs * (2.0**-8 + 2 * m * 2.0**-24) * 1.01 + np.abs(want) * 2.0**-8 * 1.01).all(), i
        top = q[i, 0, 0] * keys[0, 0] + np.log(m)
        assert np.abs(gl[i] - top).max() <= 2.0**-21 * (abs(top) + 1)
