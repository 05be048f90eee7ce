"""GPU parity of the rotary append with the 64-bit reference.  A result is one
bf16 rounding (half a step, 2^-8 of the value) of a 32-bit rotation: two
products and a sum of values up to |x| + |y| with sine and cosine good to a few
steps of 2^-24 each, within 2^-20 (|x| + |y|) together."""
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


def check(dev, seed, lens, counts, hq, hkv, dim, rot, axes, style, page, layer=1, far=0, pad=0, use_axis=True,
          start_null=False, behind=0):
    rng = np.random.default_rng(seed)
    c, r = ch.make(dev, seed, lens, counts, layers=2, hkv=hkv, page=page, dim=dim)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(start[-1]) + behind
    wide = (hq + 2 * hkv) * dim
    ybuf = torch.from_numpy(rng.standard_normal((rows, wide + pad)).astype(np.float32) * 3).to(dev)
    y = ybuf[:, :wide]
    half = rot // 2
    pos = (rng.integers(0, 5000, (axes, rows)) + far).astype(np.int32)
    f = 10000.0 ** (-np.arange(half) / max(half, 1))
    axis = (np.arange(half) % axes).astype(np.uint8) if use_axis else np.zeros(half, np.uint8)
    qbuf = torch.full((rows, hq * dim + pad), 77.0, dtype=torch.bfloat16, device=dev)
    q = qbuf[:, :hq * dim]
    abi.rope_append(c, layer, y, hq, torch.from_numpy(f).to(dev) if half else None, ch.ints(pos, dev),
                    pair_axis=torch.from_numpy(axis).to(dev) if half and use_axis else None, style=style,
                    row_start=None if start_null else ch.ints(start, dev), q=q)
    torch.cuda.synchronize()
    yh = y.cpu().numpy()
    live = int(start[-1])
    want, mag = cache_ref.rope(yh[:live], hq + 2 * hkv, dim, pos[:, :live], axis, f, style)
    want[:, hq + hkv:] = yh[:live].reshape(live, -1, dim)[:, hq + hkv:]
    tol = np.abs(want) * 2.0**-8 + mag * 2.0**-20
    got = q.float().cpu().numpy().reshape(rows, hq, dim)
    assert (np.abs(got[:live] - want[:, :hq]) <= tol[:, :hq]).all()
    assert (qbuf[live:] == 77.0).all() and (qbuf[:, hq * dim:] == 77.0).all()
    # the cache: the rows' slots hold them, everything else its old bits
    k, v = ch.host_bits(c.k), ch.host_bits(c.v)
    for b in range(len(lens)):
        for i in range(counts[b]):
            p, o = r.where(b, lens[b] + i)
            row = start[b] + i
            gk, gv = cache_ref.bf16_value(k[layer, p, :, o]), cache_ref.bf16_value(v[layer, p, :, o])
            assert (np.abs(gk - want[row, hq:hq + hkv]) <= tol[row, hq:hq + hkv]).all()
            assert np.array_equal(v[layer, p, :, o], cache_ref.bf16_bits(want[row, hq + hkv:])), "values: one rounding"
            assert np.array_equal(gv.shape, gk.shape)
            k[layer, p, :, o], v[layer, p, :, o] = r.k[layer, p, :, o], r.v[layer, p, :, o]
    assert np.array_equal(k, r.k) and np.array_equal(v, r.v), "a slot that is no row's was written"
    assert np.array_equal(c.len.cpu().numpy(), r.len)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 0), (256, 64), (256, 256)])
def test_matches_reference(dev, dim, rot, style):
    check(dev, dim + rot, [0, 15, 16, 40], [3, 1, 0, 5], 6, 2, dim, rot, 3, style, 16)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (40, 40), (40, 8), (24, 4)])
def test_heads(dev, hq, hkv):
    check(dev, hq, [7, 0], [1, 1], hq, hkv, 128, 128, 1, 0, 64, start_null=True, use_axis=False)


def test_one_row(dev):
    check(dev, 1, [0], [1], 1, 1, 64, 64, 1, 1, 16, start_null=True)


def test_a_prompt_over_many_pages(dev):
    check(dev, 2, [5, 100], [700, 301], 4, 1, 128, 128, 2, 0, 32)


def test_far_positions_keep_their_phase(dev):
    check(dev, 3, [20, 3], [4, 2], 4, 2, 128, 128, 4, 0, 16, far=2_000_000_000)


def test_strided_rows_and_rows_behind_the_last_lane(dev):
    check(dev, 4, [20, 3], [4, 2], 4, 2, 128, 64, 2, 1, 16, pad=24, behind=3)


def test_axis_past_the_last_takes_the_last(dev):
    """pair_axis values of 255 over 2 axes rotate by the second axis."""
    c, _ = ch.make(dev, 5, [0], [1], layers=1, hkv=1, dim=64)
    y = torch.randn((1, 192), device=dev)
    f = torch.ones(32, dtype=torch.float64, device=dev)
    pos = ch.ints([[1], [2]], dev)
    a = abi.rope_append(c, 0, y, 1, f, pos, pair_axis=torch.full((32,), 255, dtype=torch.uint8, device=dev))
    b = abi.rope_append(c, 0, y, 1, f, pos, pair_axis=torch.ones(32, dtype=torch.uint8, device=dev))
    assert torch.equal(a, b)


def test_rows_without_a_page_of_their_own_are_not_appended(dev):
    """No page, a page id outside the pool, a shared page, a slot past the table: q is written, the pools are not."""
    c, r = ch.make(dev, 6, [4, 4, 4, 64], [1, 1, 1, 0], layers=1, hkv=1, width_extra=0)
    c.table[0, 0] = -1
    c.table[1, 0] = 1 << 20
    c.ref[int(r.table[2, 0])] = 2
    y = torch.randn((4, 5 * 64), device=dev)
    q = abi.rope_append(c, 0, y, 3, None, None)
    torch.cuda.synchronize()
    assert torch.equal(q.view(4, -1), y[:, :192].to(torch.bfloat16))
    assert np.array_equal(ch.host_bits(c.k), r.k) and np.array_equal(ch.host_bits(c.v), r.v)
    assert ch.clean_status() == 128


def test_helper_refuses(dev):
    c, _ = ch.make(dev, 5, [0], [1], hkv=1, dim=64)
    y = torch.randn((1, 192), device=dev)
    f = torch.ones(32, dtype=torch.float64, device=dev)
    pos = ch.ints([1], dev)
    for bad in (dict(y=y.half()), dict(y=y[:, :191]), dict(positions=pos.long()), dict(inv_freq=f.float()),
                dict(positions=ch.ints([1, 2], dev)), dict(row_start=ch.ints([0], dev)), dict(y=y.cpu())):
        kw = dict(y=y, inv_freq=f, positions=pos, row_start=None)
        kw.update(bad)
        with pytest.raises(ValueError):
            abi.rope_append(c, 0, kw["y"], 1, kw["inv_freq"], kw["positions"], row_start=kw["row_start"])
