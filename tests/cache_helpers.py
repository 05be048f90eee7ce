"""Random paged caches for the cache operators' GPU tests, on the device and as the 64-bit reference."""
import numpy as np
import torch

from cache_ref import RefCache, bf16_bits
from nvfp4_weight_streaming_decode_b200 import abi


def dev_bf16(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


def host_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def ints(values, dev):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device=dev)


def words(masks, dev):
    return torch.from_numpy(np.array([int(m) & (2**64 - 1) for m in masks], np.uint64).view(np.int64)).to(dev)


def make(dev, seed, lens, room, layers=1, hkv=2, page=16, dim=64, spare=4, width_extra=2):
    """A cache whose lane b holds lens[b] slots and pages for room[b] more, in scattered order; (cache, reference)."""
    rng = np.random.default_rng(seed)
    per = [-(-(n + m) // page) for n, m in zip(lens, room)]
    pages, width = max(sum(per) + spare, 1), max(per) + width_extra
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    ref = np.zeros(pages, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        ref[order[at:at + n]] = 1
        at += n
    shape = (layers, pages, hkv, page, dim)
    k, v = bf16_bits(rng.standard_normal(shape)), bf16_bits(rng.standard_normal(shape))
    length = np.array(lens, np.int32)
    return device_cache(dev, k, v, table, length, ref), RefCache(k, v, table, length, ref)


def device_cache(dev, k, v, table, length, ref):
    return abi.Cache(dev_bf16(k, dev), dev_bf16(v, dev), ints(table, dev), ints(length, dev), ints(ref, dev))


def assert_same(cache, ref, what=""):
    torch.cuda.synchronize()
    assert np.array_equal(cache.table.cpu().numpy(), ref.table), f"{what}: tables differ"
    assert np.array_equal(cache.len.cpu().numpy(), ref.len), f"{what}: lengths differ"
    assert np.array_equal(cache.ref.cpu().numpy(), ref.ref), f"{what}: reference counts differ"
    assert np.array_equal(host_bits(cache.k), ref.k), f"{what}: keys differ"
    assert np.array_equal(host_bits(cache.v), ref.v), f"{what}: values differ"
    assert not cache.scratch[4 * cache.lanes:].any(), f"{what}: the counter was left set"


def clean_status():
    return abi.nvfp4_device_status()
