"""The attention's remaining paths against the 64-bit reference (test_gpu_attn's
bounds): heads of 256 in both block sizes where references rise, slots are unseen or
hold anything and pairs are cut between CTAs; parts of several blocks to a lane joined;
blocks chosen narrower than the lanes are."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi
from test_gpu_attn import SPECIAL, check, compare

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


def cut(lens, counts, hq, hkv, dim, max_nodes, ctas=148):
    """(blocks to a lane, whether pairs are cut) by the schedule's rule."""
    g = hq // hkv
    r = min(max_nodes, sum(counts)) * g
    block = 16 if r <= 16 else 32 if r <= 32 else 64 if r <= 64 else 128 if r <= 128 or dim > 128 else 256
    width = -(-max(counts) // (block // g))
    tiles = [-(-(n + m) // 128) for n, m in zip(lens, counts) if m]
    pairs = len(tiles) * hkv
    whole = -(-pairs * width // ctas) * max(tiles) <= sum(tiles) * hkv * width // ctas + 8
    return width, not whole


CASES = [  # lens, counts, hq, hkv, dim, page, max_nodes, blocks to a lane
    ([9001], [40], 6, 1, 256, 16, 40, 2), ([9001, 4000], [40, 24], 12, 2, 256, 64, 40, 2),
    ([20011], [64], 8, 1, 256, 128, 64, 4), ([9001], [21], 6, 1, 256, 16, 21, 1), ([9001, 300], [2, 9], 6, 1, 256, 32, 9, 1),
    ([9000], [64], 8, 1, 128, 32, 1, 32), ([9000], [40], 3, 1, 128, 64, 1, 8), ([9000, 5000], [20, 20], 8, 2, 64, 16, 3, 5),
    ([9000], [64], 32, 1, 128, 64, 64, 8), ([20000], [64], 16, 1, 64, 64, 64, 4), ([12000], [33], 8, 2, 128, 16, 2, 9),
    ([9000], [64], 5, 1, 256, 256, 2, 22)]


@pytest.mark.parametrize("lens,counts,hq,hkv,dim,page,max_nodes,blocks", CASES)
def test_parts_of_several_blocks(dev, lens, counts, hq, hkv, dim, page, max_nodes, blocks):
    assert cut(lens, counts, hq, hkv, dim, max_nodes) == (blocks, True)
    check(dev, 60 + blocks, lens, counts, hq, hkv, dim, page, max_nodes=max_nodes)


@pytest.mark.parametrize("scale", [0.25, -0.25, 40.0])
@pytest.mark.parametrize("n", [700, 9000])
@pytest.mark.parametrize("dim,rows,hq", [(256, 1, 2), (256, 3, 6), (256, 40, 3), (128, 1, 2), (128, 30, 4), (128, 40, 4)])
def test_running_maximum(dev, dim, rows, hq, n, scale):
    """Every tile has a new maximum, for every second row; the others' scores fall."""
    c, r = ch.make(dev, 61, [n], [rows], hkv=1, page=16, dim=dim)
    t = np.arange(n + rows)
    r.k[0, r.table[0, t // 16], 0, t % 16] = cache_ref.bf16_bits(np.repeat(t[:, None] / 64.0, dim, 1))
    c = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    x = np.ones((rows, hq, dim))
    x[1::2] = -1.0
    q = ch.dev_bf16(cache_ref.bf16_bits(x), dev)
    out, lse = abi.attn_tree(c, 0, q, scale, row_start=ch.ints([0, rows], dev), max_nodes=rows, want_lse=True)
    torch.cuda.synchronize()
    compare(c, r, q, scale, [0, rows], None, out, lse)


@pytest.mark.parametrize("scale,spread", [(8.0, 4.0), (0.0, 1.0), (-0.3, 1.0)])
@pytest.mark.parametrize("rows,hq", [(3, 4), (40, 6)])
def test_sharp_and_flat_scores(dev, rows, hq, scale, spread):
    for n in (900, 9000):
        check(dev, 62, [n], [rows], hq, 1, 256, 64, scale=scale, spread=spread)


@pytest.mark.parametrize("value", SPECIAL)
@pytest.mark.parametrize("rows,hq,hkv", [(8, 4, 2), (40, 6, 2)])
@pytest.mark.parametrize("n", [100, 9000])
def test_unseen_slots_never_reach_a_row(dev, value, rows, hq, hkv, n):
    """Heads of 256: two ring entries to a tile of V, in blocks of 16 and of 128 rows."""
    c, r = ch.make(dev, 63, [n, 37], [rows, 8], hkv=hkv, page=16, dim=256)
    start = [0, rows, rows + 8]
    mask = [1 << i | 1 for i in range(rows)] + [1 << i | 1 for i in range(8)]
    q = torch.randn((rows + 8, hq, 256), device=dev).to(torch.bfloat16)
    kw = dict(row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=rows, want_lse=True)
    clean, clean_lse = abi.attn_tree(c, 0, q, 0.06, **kw)
    bad = cache_ref.bf16_bits(np.full(256, value))
    touched = set()
    for b, (length, m) in enumerate(((n, rows), (37, 8))):
        for j in (3, m - 2):  # seen by the rows j alone
            p, o = r.where(b, length + j)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
            touched.add(start[b] + j)
        for s in range(length + m, -(-(length + m) // 16) * 16):
            p, o = r.where(b, s)
            r.v[0, p, :, o], r.k[0, p, :, o] = bad, bad
    free = r.ref == 0
    r.k[0, free], r.v[0, free] = bad, bad
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    out, lse = abi.attn_tree(c2, 0, q, 0.06, **kw)
    torch.cuda.synchronize()
    rest = [i for i in range(rows + 8) if i not in touched]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    if not np.isfinite(value):
        assert not torch.isfinite(out[sorted(touched)].float()).all(-1).any(), "a row that sees it shows it"


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("rows,hq", [(8, 2), (40, 6)])
def test_a_value_that_is_seen_shows(dev, value, rows, hq):
    """In either half of a head of 256."""
    c, r = ch.make(dev, 64, [120], [rows], hkv=1, page=16, dim=256)
    for node, d in ((2, 5), (5, 200)):
        p, o = r.where(0, 120 + node)
        r.v[0, p, 0, o, d] = cache_ref.bf16_bits(np.array([value]))[0]
    c2 = ch.device_cache(dev, r.k, r.v, r.table, r.len, r.ref)
    q = torch.randn((rows, hq, 256), device=dev).to(torch.bfloat16)
    mask = [1 << i | (1 << 2 if i in (6, 7) else 0) | (1 << 5 if i == 7 else 0) for i in range(rows)]
    out, lse = abi.attn_tree(c2, 0, q, 0.06, row_start=ch.ints([0, rows], dev), mask=ch.words(mask, dev), max_nodes=rows,
                             want_lse=True)
    torch.cuda.synchronize()
    compare(c2, r, q, 0.06, [0, rows], mask, out, lse)
    bad = ~torch.isfinite(out.float())
    assert bad[[2, 6, 7], :, 5].all() and bad[[5, 7], :, 200].all() and int(bad.sum()) == 5 * hq


@pytest.mark.parametrize("rows,hq", [(8, 2), (40, 6)])
def test_rows_that_see_nothing_and_bad_pages(dev, rows, hq):
    c, r = ch.make(dev, 65, [0, 300], [rows, 8], hkv=1, page=16, dim=256)
    q = torch.randn((rows + 8, hq, 256), device=dev).to(torch.bfloat16)
    mask = [0 if i % 3 == 0 else 1 << i | 1 for i in range(rows)] + [1] * 8
    start = [0, rows, rows + 8]
    for b, col, e in ((1, 2, 1 << 24), (1, 9, -1)):
        c.table[b, col] = e
        r.table[b, col] = e
    out, lse = abi.attn_tree(c, 0, q, 0.06, row_start=ch.ints(start, dev), mask=ch.words(mask, dev), max_nodes=rows,
                             want_lse=True)
    torch.cuda.synchronize()
    got, gl = compare(c, r, q, 0.06, start, mask, out, lse)
    assert not got[0:rows:3].any() and np.isneginf(gl[0:rows:3]).all()
    assert ch.clean_status() == 128
