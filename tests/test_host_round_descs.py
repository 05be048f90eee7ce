"""CPU tests of the descriptors of a round's rotary append and attention: what the
captured round would name must be the caller's and have the widest round's rows."""
import types

import pytest
import torch

from nvfp4_weight_streaming_decode_b200 import abi

BF16, HOST = torch.bfloat16, torch.device("cpu")


def cache():
    # of a cache, the records need no more than this; nothing is launched here
    return types.SimpleNamespace(device=HOST, head_dim=64, kv_heads=1, lanes=8, _at=1)


def attn(**kw):
    f = dict(q=torch.zeros((8, 2, 64), dtype=BF16), out=torch.zeros((8, 128), dtype=BF16),
             workspace=torch.zeros(64, dtype=torch.uint8), lse=None)
    f.update(kw)
    return abi.desc_attn(cache(), 0, f["q"], 0.1, f["out"], f["workspace"], f["lse"]), f


def rope(rotated=True, **kw):
    f = dict(y=torch.zeros((8, 4 * 64)), q=torch.zeros((8, 2, 64), dtype=BF16),
             inv_freq=torch.ones(32, dtype=torch.float64) if rotated else None,
             positions=torch.zeros(8, dtype=torch.int32) if rotated else None)
    f.update(kw)
    return abi.desc_rope(cache(), 0, f["y"], 2, f["inv_freq"], f["positions"], f["q"]), f


def test_what_a_descriptor_names_is_kept():
    for make in (attn, lambda: attn(lse=torch.zeros((8, 2))), rope, lambda: rope(rotated=False)):
        d, f = make()
        for t in f.values():
            assert t is None or any(k is t for k in d._keep)


@pytest.mark.parametrize("name", ["q", "out", "workspace"])
def test_attention_without_its_tensors_is_refused(name):
    with pytest.raises(ValueError, match=name):
        attn(**{name: None})


@pytest.mark.parametrize("name", ["y", "q"])
@pytest.mark.parametrize("rotated", [True, False])
def test_append_without_its_tensors_is_refused(name, rotated):
    with pytest.raises(ValueError, match=name):
        rope(rotated, **{name: None})


@pytest.mark.parametrize("rows", [1, 4, 7])
def test_fewer_rows_than_the_widest_round_are_refused(rows):
    q = torch.zeros((rows, 2, 64), dtype=BF16)
    for kw in (dict(q=q, out=q.clone()), dict(q=q), dict(out=q)):
        with pytest.raises(ValueError, match="8 rows"):
            attn(**kw)
    y, pos = torch.zeros((rows, 4 * 64)), torch.zeros(rows, dtype=torch.int32)
    for rotated, kw in ((True, dict(y=y, q=q, positions=pos)), (False, dict(y=y, q=q)), (False, dict(y=y)),
                        (True, dict(q=q))):
        with pytest.raises(ValueError, match="8 rows"):
            rope(rotated, **kw)
    with pytest.raises(ValueError, match="positions"):
        rope(positions=pos)


def test_more_rows_are_fine():
    attn(q=torch.zeros((9, 2, 64), dtype=BF16), out=torch.zeros((9, 2, 64), dtype=BF16))
    rope(False, y=torch.zeros((9, 256)), q=torch.zeros((9, 128), dtype=BF16))
