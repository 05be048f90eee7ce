"""GPU parity of the cache attention with the 64-bit reference.

Tolerance, from the arithmetic: a 32-bit score is off by at most e (the
reference's bound on its products and sums), so a weight by a factor within
2e + 2^-21 (exponential); the weight is rounded to bf16 for the product with v
(half a step, 2^-8); the sums of n terms in 32 bits add n 2^-24 of the summed
magnitudes, to the numerator and to the normaliser; the result is rounded once
more (2^-8 of itself)."""
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


@pytest.fixture(autouse=True)
def status(dev):
    ch.clean_status()
    yield
    assert ch.clean_status() == 0


def tree(rng, counts):
    """Ancestor masks of a random tree per lane."""
    out = []
    for n in counts:
        m = []
        for i in range(n):
            m.append((m[rng.integers(0, i)] if i else 0) | 1 << i)
        out += m
    return out


def compare(c, r, q, scale, start, mask, out, lse, layer=0):
    qh = cache_ref.bf16_value(ch.host_bits(q)).astype(np.float64)
    rows = int(start[-1])
    want, wl, wabs, err, seen = cache_ref.attention(r, layer, qh, np.float32(scale).astype(np.float64), start, mask)
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    part = (2 * err[:rows, :, None] + 2.0**-21 + 2.0**-8 + 2 * seen[:rows, None, None] * 2.0**-24)
    with np.errstate(invalid="ignore"):
        tol = wabs[:rows] * part * 1.01 + np.abs(want[:rows]) * 2.0**-8 * 1.01 + 1e-38
        fine = (np.abs(got[:rows] - want[:rows]) <= tol) | (np.isnan(want[:rows]) & np.isnan(got[:rows])) | \
            (want[:rows] == got[:rows])
        assert fine.all(), f"out: worst error / bound {np.nanmax(np.abs(got[:rows] - want[:rows]) / tol)}"
        ltol = err[:rows] + 2.0**-21 * (1 + np.abs(wl[:rows])) + seen[:rows, None] * 2.0**-24
        fine = (np.abs(gl[:rows] - wl[:rows]) <= ltol) | (wl[:rows] == gl[:rows]) | \
            (np.isnan(wl[:rows]) & np.isnan(gl[:rows]))
        assert fine.all(), f"lse: worst {np.nanmax(np.abs(gl[:rows] - wl[:rows]) / ltol)}"
    return got, gl


def check(dev, seed, lens, counts, hq, hkv, dim, page, kind="tree", scale=None, spread=1.0, null_start=False,
          max_nodes=None):
    rng = np.random.default_rng(seed)
    c, r = ch.make(dev, seed, lens, counts, hkv=hkv, page=page, dim=dim)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(start[-1])
    q = ch.dev_bf16(cache_ref.bf16_bits(rng.standard_normal((rows, hq, dim)) * spread), dev)
    mask = None if kind == "chain" else tree(rng, counts)
    scale = dim**-0.5 if scale is None else scale
    before = (ch.host_bits(c.k), ch.host_bits(c.v))
    out, lse = abi.attn_tree(c, 0, q, scale, row_start=None if null_start else ch.ints(start, dev),
                             mask=None if mask is None else ch.words(mask, dev),
                             max_nodes=max(counts) if max_nodes is None else max_nodes, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, scale, start, mask, out, lse)
    assert np.array_equal(before[0], ch.host_bits(c.k)) and np.array_equal(before[1], ch.host_bits(c.v))
    return out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 500, 1031])
def test_decode_lengths(dev, n, page, dim):
    """One row; its context ends before, on and behind pages and tiles (n counts the row's own slot)."""
    check(dev, n, [n - 1], [1], 4, 2, dim, page, kind="chain", null_start=True)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (8, 1), (32, 1), (40, 8), (24, 4), (6, 2)])
def test_heads(dev, hq, hkv):
    check(dev, hq, [70, 300, 0], [1, 1, 1], hq, hkv, 128, 32, kind="chain", null_start=True)


@pytest.mark.parametrize("counts", [[1], [2, 0, 5], [8] * 8, [64], [17, 1, 46], [0, 0, 9]])
@pytest.mark.parametrize("hq,hkv,dim", [(5, 1, 128), (8, 2, 64), (6, 1, 256), (16, 2, 128)])
def test_trees(dev, counts, hq, hkv, dim):
    rng = np.random.default_rng(sum(counts))
    check(dev, 11, [int(x) for x in rng.integers(0, 400, len(counts))], counts, hq, hkv, dim, 16)


@pytest.mark.parametrize("counts", [[3, 1], [64], [8, 8, 8]])
def test_chain_is_the_default_mask(dev, counts):
    check(dev, 12, [130, 5, 61][:len(counts)], counts, 8, 2, 128, 64, kind="chain")


def test_tiling_hint_does_not_change_the_bounds(dev):
    for hint in (1, 3, 64, 1000):
        check(dev, 13, [200, 31], [40, 24], 4, 1, 128, 32, max_nodes=hint)


def test_many_lanes(dev):
    check(dev, 14, [int(x) for x in np.random.default_rng(0).integers(0, 700, 64)], [1] * 64, 4, 2, 64, 16)


def test_long_context(dev):
    check(dev, 15, [20011, 9000], [4, 1], 4, 1, 128, 64)


def test_sharp_and_flat_scores(dev):
    """Scores over thousands (one slot takes all, at the tail, the head or the middle) and all alike."""
    check(dev, 16, [900], [3], 4, 2, 128, 64, scale=8.0, spread=4.0)
    check(dev, 17, [900], [3], 4, 2, 128, 64, scale=0.0)
    check(dev, 18, [900], [3], 4, 2, 128, 64, scale=-0.3)


def rising(dev, dim, n):
    """Keys whose scores grow from slot to slot, so that every tile has a new maximum."""
    c, r = ch.make(dev, 19, [n], [1], hkv=1, page=16, dim=dim)
    for s in range(n + 1):
        p, o = r.where(0, s)
        r.k[0, p, 0, o] = cache_ref.bf16_bits(np.full(dim, s / 64.0))
    return ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref), r


@pytest.mark.parametrize("scale", [0.25, -0.25, 40.0])
def test_running_maximum(dev, scale):
    c, r = rising(dev, 64, 700)
    q = ch.dev_bf16(cache_ref.bf16_bits(np.ones((1, 2, 64))), dev)
    out, lse = abi.attn_tree(c, 0, q, scale, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, scale, [0, 1], None, out, lse)


def test_rows_that_see_nothing(dev):
    """No context and an empty mask; beside rows that see something; and a lane of length 0."""
    c, r = ch.make(dev, 20, [0, 40, 0], [3, 2, 2], hkv=2, dim=128)
    q = torch.randn((7, 8, 128), device=dev).to(torch.bfloat16)
    mask, start = [0, 0b010, 0b111, 0, 0b01, 0, 0], [0, 3, 5, 7]
    out, lse = abi.attn_tree(c, 0, q, 0.1, row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=3,
                             want_lse=True)
    torch.cuda.synchronize()
    got, gl = compare(c, r, q, 0.1, start, mask, out, lse)
    for row in (0, 5, 6):
        assert not got[row].any() and np.isneginf(gl[row]).all()


def test_mask_bits_past_the_lane_s_rows_mean_nothing(dev):
    c, r = ch.make(dev, 21, [40], [3], hkv=1, dim=64)
    q = torch.randn((3, 2, 64), device=dev).to(torch.bfloat16)
    kw = dict(row_start=ch.ints([0, 3], dev), max_nodes=3)
    a = abi.attn_tree(c, 0, q, 0.1, mask=ch.words([0b1, 0b11, 0b101], dev), **kw)
    b = abi.attn_tree(c, 0, q, 0.1, mask=ch.words([0b1001, 2**64 - 8 + 3, 0b101 | 1 << 63], dev), **kw)
    assert torch.equal(a, b)


SPECIAL = [np.nan, np.inf, -np.inf, 3.3e38]


@pytest.mark.parametrize("value", SPECIAL)
def test_unseen_slots_never_reach_a_row(dev, value):
    """NaN, infinities and the largest values in drafted slots outside a row's mask, behind the last slot of a page,
    in free pages and in other lanes' slots: rows that do not see them are as without them."""
    lens, counts = [37, 100], [8, 8]
    c, r = ch.make(dev, 22, lens, counts, hkv=2, page=16, dim=128)
    start = [0, 8, 16]
    mask = [0b1, 0b11, 0b101, 0b1001, 0b10001, 0b100001, 0b1000001, 0b10000001] * 2
    q = torch.randn((16, 4, 128), device=dev).to(torch.bfloat16)
    kw = dict(row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=8, want_lse=True)
    clean, clean_lse = abi.attn_tree(c, 0, q, 0.1, **kw)
    bad = cache_ref.bf16_bits(np.full(128, value))
    touched = set()
    for b in range(2):
        for j in (3, 6):  # seen by the rows j alone
            p, o = r.where(b, lens[b] + j)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
        last = lens[b] + counts[b]
        for s in range(last, -(-last // 16) * 16):
            p, o = r.where(b, s)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
        touched |= {b * 8 + 3, b * 8 + 6}
    free = r.ref == 0
    r.k[0, free], r.v[0, free] = bad, bad
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    out, lse = abi.attn_tree(c2, 0, q, 0.1, **kw)
    torch.cuda.synchronize()
    rest = [i for i in range(16) if i not in touched]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if not np.isfinite(value):
        assert not torch.isfinite(out[sorted(touched)].float()).all(-1).any(), "a row that sees it shows it"


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_value_that_is_seen_shows(dev, value):
    """A non-finite value (not key) in one drafted slot: rows that see it have it in that column, the others not."""
    c, r = ch.make(dev, 23, [20], [4], hkv=1, page=16, dim=64)
    p, o = r.where(0, 22)  # node 2
    r.v[0, p, 0, o, 5] = cache_ref.bf16_bits(np.array([value]))[0]
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    q = torch.randn((4, 2, 64), device=dev).to(torch.bfloat16)
    mask = [0b1, 0b11, 0b101, 0b1101]
    out, lse = abi.attn_tree(c2, 0, q, 0.1, row_start=ch.ints([0, 4], dev), mask=ch.words(mask, dev), max_nodes=4,
                             want_lse=True)
    torch.cuda.synchronize()
    compare(c2, r, q, 0.1, [0, 4], mask, out, lse)
    bad = ~torch.isfinite(out.float())
    assert bad[2:, :, 5].all() and int(bad.sum()) == 4


def test_bad_pages_are_not_seen(dev):
    """A page id outside the pool and an entry of -1 inside the context: their slots drop out, the status says so."""
    c, r = ch.make(dev, 24, [100, 60], [1, 1], hkv=1, page=16, dim=64)
    for b, col, e in ((0, 2, 1 << 24), (0, 4, -1), (1, 0, -7)):
        c.table[b, col] = e
        r.table[b, col] = e
    q = torch.randn((2, 2, 64), device=dev).to(torch.bfloat16)
    out, lse = abi.attn_tree(c, 0, q, 0.1, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, 0.1, [0, 1, 2], None, out, lse)
    assert ch.clean_status() == 128


def test_lengths_past_the_table_and_below_zero(dev):
    c, r = ch.make(dev, 25, [100, 60, 30], [1, 1, 1], hkv=1, page=16, dim=64)
    for b, n in ((0, 2**31 - 1), (1, -5)):
        c.len[b] = n
    r.len[0] = r.table.shape[1] * 16
    r.len[1] = 0
    q = torch.randn((3, 2, 64), device=dev).to(torch.bfloat16)
    out, lse = abi.attn_tree(c, 0, q, 0.1, want_lse=True)
    torch.cuda.synchronize()
    got, gl = compare(c, r, q, 0.1, [0, 1, 2, 3], [0, 1, 1], out, lse)
    assert ch.clean_status() == 128


def test_strided_rows_and_rows_behind_the_last_lane(dev):
    c, r = ch.make(dev, 26, [33, 18], [2, 1], hkv=2, page=16, dim=128, layers=3)
    buf = torch.randn((5, 4 * 128 + 40), device=dev).to(torch.bfloat16)
    ob = torch.full((5, 4 * 128 + 16), 55.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((5, 4), 55.0, device=dev)
    q = buf[:, 8:8 + 512].view(5, 512)
    abi.attn_tree(c, 2, q, 0.1, row_start=ch.ints([0, 2, 3], dev), max_nodes=2, out=ob[:, :512], lse=lse)
    torch.cuda.synchronize()
    compare(c, r, q[:3].reshape(3, 4, 128), 0.1, [0, 2, 3], None, ob[:3, :512].reshape(3, 4, 128), lse[:3], layer=2)
    assert (ob[3:] == 55.0).all() and (ob[:, 512:] == 55.0).all() and (lse[3:] == 55.0).all()


def test_same_from_call_to_call_and_in_graphs(dev):
    """Bit-identical results of repeated calls, of two graphs with a workspace each replayed on two streams, and of
    calls of other sizes in between on the same workspace."""
    c, r = ch.make(dev, 27, [3000, 500, 0, 90], [8, 8, 8, 8], hkv=2, page=32, dim=128)
    q = torch.randn((32, 10, 128), device=dev).to(torch.bfloat16)
    start = ch.ints([0, 8, 16, 24, 32], dev)
    kw = dict(row_start=start, max_nodes=8, want_lse=True)
    ws = abi.attn_tree_workspace(c, 32, 10)
    first, fl = abi.attn_tree(c, 0, q, 0.1, workspace=ws, **kw)
    abi.attn_tree(c, 0, q[:4, :2].contiguous(), 0.1, workspace=ws)
    again, al = abi.attn_tree(c, 0, q, 0.1, workspace=ws, **kw)
    assert torch.equal(first, again) and torch.equal(fl, al)
    graphs, outs, streams = [], [], [torch.cuda.Stream(dev) for _ in range(2)]
    for s in streams:
        w = abi.attn_tree_workspace(c, 32, 10)
        o = torch.zeros_like(first)
        s.wait_stream(torch.cuda.current_stream(dev))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            abi.attn_tree(c, 0, q, 0.1, row_start=start, max_nodes=8, out=o, workspace=w)
        graphs.append((g, w))
        outs.append(o)
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


def test_another_stream(dev):
    c, r = ch.make(dev, 28, [100], [1], hkv=2, page=32, dim=128)
    q = torch.randn((1, 4, 128), device=dev).to(torch.bfloat16)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    out, lse = abi.attn_tree(c, 0, q, 0.1, want_lse=True, stream=s)
    s.synchronize()
    compare(c, r, q, 0.1, [0, 1], None, out, lse)


def test_workspace_too_small_is_refused(dev):
    c, _ = ch.make(dev, 29, [10], [1])
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=dev)
    with pytest.raises(abi.Nvfp4Error) as e:
        abi.attn_tree(c, 0, q, 0.1, workspace=torch.zeros(0, dtype=torch.uint8, device=dev).new_zeros(8))
    assert e.value.status == abi.NVFP4_ERR_SCRATCH


def test_helper_refuses(dev):
    c, _ = ch.make(dev, 29, [10], [1])
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=dev)
    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q.cpu()), dict(row_start=ch.ints([0], dev)),
                dict(mask=ch.ints([1], dev)), dict(out=torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=dev))):
        kw = dict(q=q)
        kw.update(bad)
        x = kw.pop("q")
        with pytest.raises(ValueError):
            abi.attn_tree(c, 0, x, 0.1, **kw)


# ------------------- lanes of more than 128 query rows to a cached head (heads of 64 and 128)

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [0, 1, 64, 127, 128, 192, 1000])
def test_wide_trees_at_tile_borders(dev, n, dim):
    """The drafted slots begin before, on and behind a tile's border and reach into a second one."""
    check(dev, 40 + n, [n], [64], 8, 2, dim, 16)


@pytest.mark.parametrize("counts,hq,hkv", [([33], 4, 1), ([64], 5, 1), ([43], 3, 1), ([5, 59], 32, 1), ([64], 32, 1),
                                           ([1, 40, 0, 3, 20], 8, 2), ([2] * 6 + [50], 12, 2), ([9, 9], 15, 1)])
def test_wide_heads_and_lanes(dev, counts, hq, hkv):
    """A second half with a few rows, rows split between the halves, several blocks to a lane, narrow lanes between."""
    lens = [int(x) for x in np.random.default_rng(hq).integers(0, 900, len(counts))]
    check(dev, 41, lens, counts, hq, hkv, 128, 32)
    check(dev, 42, lens, counts, hq, hkv, 64, 16, kind="chain")


def test_wide_long_context(dev):
    """Pairs cut between CTAs and joined."""
    check(dev, 43, [9000, 20011], [40, 24], 8, 1, 128, 64)


@pytest.mark.parametrize("scale,spread", [(8.0, 4.0), (0.0, 1.0), (-0.3, 1.0)])
def test_wide_sharp_and_flat_scores(dev, scale, spread):
    check(dev, 44, [900], [40], 8, 2, 128, 64, scale=scale, spread=spread)


@pytest.mark.parametrize("power", [22, 26, 33, 60])
@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("n", [0, 300, 9000])
def test_scores_past_the_headroom_s_own_rounding(dev, n, rows, power):
    """Scores of some 2^power for every second row: their rounding alone may pass 2^32; between rows of ordinary ones."""
    rng = np.random.default_rng(51)
    c, r = ch.make(dev, 51, [n], [rows], hkv=2, page=64, dim=128)
    x = rng.standard_normal((rows, 8, 128))
    x[::2] *= 2.0**power
    q = ch.dev_bf16(cache_ref.bf16_bits(x), dev)
    out, lse = abi.attn_tree(c, 0, q, 0.1, row_start=ch.ints([0, rows], dev), max_nodes=rows, want_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    compare(c, r, q, 0.1, [0, rows], None, out, lse)


@pytest.mark.parametrize("scale", [0.25, -0.25, 40.0])
def test_wide_running_maximum(dev, scale):
    """Every tile has a new maximum, for every second row; the others' scores fall."""
    rows = 36
    c, r = ch.make(dev, 45, [700], [rows], hkv=1, page=16, dim=64)
    for s in range(700 + rows):
        p, o = r.where(0, s)
        r.k[0, p, 0, o] = cache_ref.bf16_bits(np.full(64, s / 64.0))
    c = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    x = np.ones((rows, 4, 64))
    x[1::2] = -1.0
    q = ch.dev_bf16(cache_ref.bf16_bits(x), dev)
    out, lse = abi.attn_tree(c, 0, q, scale, row_start=ch.ints([0, rows], dev), max_nodes=rows, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, scale, [0, rows], None, out, lse)


def test_wide_rows_that_see_nothing(dev):
    rows = 48
    c, r = ch.make(dev, 46, [0, 20], [40, 8], hkv=1, dim=128)
    q = torch.randn((rows, 8, 128), device=dev).to(torch.bfloat16)
    mask = [0 if i % 3 == 0 else 1 << i | 1 for i in range(40)] + [0] * 8
    start = [0, 40, 48]
    out, lse = abi.attn_tree(c, 0, q, 0.1, row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=40,
                             want_lse=True)
    torch.cuda.synchronize()
    got, gl = compare(c, r, q, 0.1, start, mask, out, lse)
    assert not got[0:40:3].any() and np.isneginf(gl[0:40:3]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("value", SPECIAL)
def test_wide_unseen_slots_never_reach_a_row(dev, value, dim):
    lens, counts = [100, 37], [40, 24]
    c, r = ch.make(dev, 47, lens, counts, hkv=2, page=16, dim=dim)
    start = [0, 40, 64]
    mask = [1 << i | 1 for i in range(40)] + [1 << i | 1 for i in range(24)]
    q = torch.randn((64, 16, dim), device=dev).to(torch.bfloat16)
    kw = dict(row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=40, want_lse=True)
    clean, clean_lse = abi.attn_tree(c, 0, q, 0.1, **kw)
    bad = cache_ref.bf16_bits(np.full(dim, value))
    touched = set()
    for b in range(2):
        for j in (3, 11, 20):  # seen by the rows j alone
            p, o = r.where(b, lens[b] + j)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
            touched.add(start[b] + j)
        last = lens[b] + counts[b]
        for s in range(last, -(-last // 16) * 16):
            p, o = r.where(b, s)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
    free = r.ref == 0
    r.k[0, free], r.v[0, free] = bad, bad
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    out, lse = abi.attn_tree(c2, 0, q, 0.1, **kw)
    torch.cuda.synchronize()
    rest = [i for i in range(64) if i not in touched]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if not np.isfinite(value):
        assert not torch.isfinite(out[sorted(touched)].float()).all(-1).any()


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_wide_value_that_is_seen_shows(dev, value):
    c, r = ch.make(dev, 48, [120], [40], hkv=1, page=16, dim=128)
    for node, d in ((2, 5), (30, 100)):
        p, o = r.where(0, 120 + node)
        r.v[0, p, 0, o, d] = cache_ref.bf16_bits(np.array([value]))[0]
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    q = torch.randn((40, 4, 128), device=dev).to(torch.bfloat16)
    mask = [1 << i | (1 << 2 if i in (7, 33) else 0) | (1 << 30 if i in (31, 33) else 0) for i in range(40)]
    out, lse = abi.attn_tree(c2, 0, q, 0.1, row_start=ch.ints([0, 40], dev), mask=ch.words(mask, dev), max_nodes=40,
                             want_lse=True)
    torch.cuda.synchronize()
    compare(c2, r, q, 0.1, [0, 40], mask, out, lse)
    bad = ~torch.isfinite(out.float())
    assert bad[[2, 7, 33], :, 5].all() and bad[[30, 31, 33], :, 100].all() and int(bad.sum()) == 24


def test_wide_bad_pages_are_not_seen(dev):
    c, r = ch.make(dev, 49, [300, 60], [40, 1], hkv=1, page=16, dim=128)
    for b, col, e in ((0, 2, 1 << 24), (0, 9, -1), (0, 20, 1 << 20), (1, 0, -7)):
        c.table[b, col] = e
        r.table[b, col] = e
    q = torch.randn((41, 4, 128), device=dev).to(torch.bfloat16)
    out, lse = abi.attn_tree(c, 0, q, 0.1, row_start=ch.ints([0, 40, 41], dev), max_nodes=40, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, 0.1, [0, 40, 41], None, out, lse)
    assert ch.clean_status() == 128


def test_wide_same_from_call_to_call_and_in_a_graph(dev):
    c, r = ch.make(dev, 50, [3000, 500], [40, 24], hkv=2, page=32, dim=128)
    q = torch.randn((64, 16, 128), device=dev).to(torch.bfloat16)
    ws = abi.attn_tree_workspace(c, 64, 16)
    kw = dict(row_start=ch.ints([0, 40, 64], dev), max_nodes=40, workspace=ws)
    first = abi.attn_tree(c, 0, q, 0.1, **kw)
    abi.attn_tree(c, 0, q[:2], 0.1, workspace=ws)
    out = torch.zeros_like(first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.attn_tree(c, 0, q, 0.1, out=out, **kw)
    for _ in range(10):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        out.zero_()
