"""CPU tests of the cache operators' argument checks: each call returns its
status before the library touches CUDA.  And of the 64-bit references
themselves on hand-worked cases."""
import ctypes
import types

import numpy as np
import pytest

import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi

P = 1 << 20  # a fake, aligned "device" pointer: never dereferenced on these paths
ARG, M, SHAPE, ALIGN, SCRATCH = (abi.NVFP4_ERR_ARG, abi.NVFP4_ERR_M, abi.NVFP4_ERR_SHAPE, abi.NVFP4_ERR_ALIGN,
                                 abi.NVFP4_ERR_SCRATCH)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from nvfp4_weight_streaming_decode_b200 import build
    build.build()
    return abi.load()


def cache(**kw):
    f = dict(k=P, v=P, table=P, len=P, ref=P, scratch=P, layers=2, pages=64, kv_heads=2, page_size=16, head_dim=128,
             lanes=4, max_pages=16, reserved=0)
    f.update(kw)
    return abi.Nvfp4Cache(**f)


BAD_CACHES = [(dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(len=None), ARG),
              (dict(ref=None), ARG), (dict(scratch=None), ARG), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
              (dict(page_size=512), SHAPE), (dict(page_size=0), SHAPE), (dict(head_dim=96), SHAPE),
              (dict(head_dim=0), SHAPE), (dict(lanes=0), SHAPE), (dict(lanes=65), SHAPE), (dict(kv_heads=0), SHAPE),
              (dict(kv_heads=257), SHAPE), (dict(layers=0), SHAPE), (dict(pages=0), SHAPE),
              (dict(pages=(1 << 24) + 1), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 20) + 1), SHAPE),
              (dict(pages=1 << 24, page_size=256, kv_heads=1), SHAPE), (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN),
              (dict(table=P + 2), ALIGN), (dict(len=P + 1), ALIGN), (dict(ref=P + 2), ALIGN),
              (dict(scratch=P + 2), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_cache_is_refused_by_every_call(kw, status):
    c = ctypes.byref(cache(**kw))
    assert abi.nvfp4_cache_fork(c, P, None) == status
    assert abi.nvfp4_cache_reserve(c, P, None, None) == status
    assert abi.nvfp4_cache_compact(c, P, P, 8, None) == status
    assert abi.nvfp4_cache_trim(c, P, None) == status
    assert abi.nvfp4_rope_append(ctypes.byref(rope(cache(**kw))), None) == status
    assert abi.nvfp4_attn_tree(ctypes.byref(attn(cache(**kw))), None) == status


def test_page_operations_refuse():
    c = ctypes.byref(cache())
    assert abi.nvfp4_cache_fork(None, P, None) == ARG
    assert abi.nvfp4_cache_fork(c, None, None) == ARG
    assert abi.nvfp4_cache_fork(c, P + 2, None) == ALIGN
    assert abi.nvfp4_cache_reserve(c, None, None, None) == ARG
    assert abi.nvfp4_cache_reserve(c, P, P + 1, None) == ALIGN
    assert abi.nvfp4_cache_trim(c, None, None) == ARG
    assert abi.nvfp4_cache_trim(c, P + 2, None) == ALIGN
    assert abi.nvfp4_cache_compact(c, None, P, 4, None) == ARG
    assert abi.nvfp4_cache_compact(c, P, P, 0, None) == SHAPE
    assert abi.nvfp4_cache_compact(c, P, P, 65, None) == SHAPE
    assert abi.nvfp4_cache_compact(c, P, P + 2, 4, None) == ALIGN


def rope(c=None, **kw):
    c = cache() if c is None else c
    f = dict(cache=ctypes.pointer(c), layer=1, rows=4, q_heads=8, rot_dim=128, style=0, axes=1, y=P, ldy=12 * 128,
             row_start=None, positions=P, ldp=4, pair_axis=None, inv_freq=P, q=P, ldq=1024)
    f.update(kw)
    return abi.Nvfp4RopeArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), ARG), (dict(q=None), ARG), (dict(positions=None), ARG), (dict(inv_freq=None), ARG),
    (dict(style=2), ARG), (dict(rows=0), M), (dict(rows=5), M), (dict(rows=65536, row_start=P, ldp=65536), M),
    (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE), (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(rot_dim=136), SHAPE), (dict(rot_dim=144), SHAPE), (dict(rot_dim=-16), SHAPE), (dict(rot_dim=8), SHAPE),
    (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(ldp=3), SHAPE), (dict(ldy=12 * 128 - 4), SHAPE),
    (dict(ldq=1016), SHAPE), (dict(y=P + 8), ALIGN), (dict(q=P + 8), ALIGN), (dict(ldy=12 * 128 + 2), ALIGN),
    (dict(ldq=1028), ALIGN), (dict(row_start=P + 2), ALIGN), (dict(positions=P + 1), ALIGN),
    (dict(inv_freq=P + 4), ALIGN)])
def test_rope_refuses(kw, status):
    assert abi.nvfp4_rope_append(ctypes.byref(rope(**kw)), None) == status


def attn(c=None, **kw):
    c = cache() if c is None else c
    f = dict(cache=ctypes.pointer(c), layer=0, rows=4, q_heads=8, max_nodes=1, scale=0.1, reserved=0, q=P, ldq=1024,
             row_start=None, mask=None, out=P, ldo=1024, lse=None, workspace=P, workspace_bytes=1 << 30)
    f.update(kw)
    return abi.Nvfp4AttnArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(workspace=None), ARG), (dict(rows=0), M), (dict(rows=5), M),
    (dict(rows=65, row_start=P), M), (dict(layer=2), SHAPE), (dict(q_heads=9), SHAPE), (dict(q_heads=66), SHAPE),
    (dict(max_nodes=0), SHAPE), (dict(ldq=1016), SHAPE), (dict(ldo=1016), SHAPE), (dict(q=P + 8), ALIGN),
    (dict(out=P + 2), ALIGN), (dict(workspace=P + 8), ALIGN), (dict(ldq=1028), ALIGN), (dict(ldo=1028), ALIGN),
    (dict(row_start=P + 2), ALIGN), (dict(mask=P + 4), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_attention_refuses(kw, status):
    assert abi.nvfp4_attn_tree(ctypes.byref(attn(**kw)), None) == status


def test_attention_refuses_tables_past_its_schedule():
    c = cache(lanes=64, kv_heads=256, pages=1024, page_size=256, max_pages=1 << 17)
    a = attn(c, q_heads=256, ldq=256 * 128, ldo=256 * 128)
    assert abi.nvfp4_attn_tree(ctypes.byref(a), None) == SHAPE


def test_attention_workspace_sizes():
    assert abi.nvfp4_attn_tree_workspace(8, 40, 8, 128, 0)[0] == ARG
    assert abi.nvfp4_attn_tree_workspace(0, 40, 8, 128, 148)[0] == M
    assert abi.nvfp4_attn_tree_workspace(65, 40, 8, 128, 148)[0] == M
    for bad in ((8, 41, 8, 128), (8, 0, 8, 128), (8, 40, 0, 128), (8, 40, 8, 80), (8, 33, 1, 128)):
        assert abi.nvfp4_attn_tree_workspace(*bad, 148)[0] == SHAPE
    for dim in (64, 128, 256):
        st, n = abi.nvfp4_attn_tree_workspace(64, 64, 8, dim, 148)
        assert st == abi.NVFP4_OK and 0 < n < 1 << 30


def between(kind, args):
    return abi.Nvfp4GemmDesc(kind, ctypes.cast(ctypes.pointer(args), ctypes.c_void_p))


def test_round_refuses_nodes_it_cannot_run():
    """One row per lane and 8 lanes, in a chained round; each node's own checks at 8 rows."""
    ok8 = cache(lanes=8)
    cases = [(between(2, rope(ok8, row_start=P, ldp=8)), 1, ARG), (between(3, attn(ok8, row_start=P)), 1, ARG),
             (between(2, rope(cache(lanes=7), ldp=8)), 1, M), (between(3, attn(cache(lanes=4))), 1, M),
             (between(2, rope(ok8, ldp=7)), 1, SHAPE), (between(3, attn(ok8, ldo=8)), 1, SHAPE),
             (between(2, rope(cache(lanes=8, k=None), ldp=8)), 1, ARG), (between(2, rope(ok8, ldp=8)), 0, ARG),
             (between(3, attn(ok8)), 0, ARG), (abi.Nvfp4GemmDesc(2, None), 1, ARG), (abi.Nvfp4GemmDesc(3, None), 1, ARG)]
    for d, mode, status in cases:
        st, h = abi.nvfp4_round_create_ex([d], mode)
        assert (st, h) == (status, None)


def beam(**kw):
    f = dict(logits=P, groups=2, beams=4, V=1000, ldv=1000, scores=P, finished=None, eos=2, scores_out=P, parent=P,
             token=P, finished_out=None, workspace=P, workspace_bytes=1 << 30, stream=None)
    f.update(kw)
    return abi.nvfp4_beam_select(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), ARG), (dict(scores=None), ARG), (dict(scores_out=None), ARG), (dict(parent=None), ARG),
    (dict(token=None), ARG), (dict(workspace=None), ARG), (dict(groups=0), M), (dict(beams=0), M),
    (dict(groups=17), M), (dict(groups=1 << 30, beams=1 << 30), M), (dict(V=0), SHAPE),
    (dict(V=(1 << 20) + 4, ldv=(1 << 20) + 4), SHAPE), (dict(ldv=996), SHAPE), (dict(finished=P, eos=1000), SHAPE),
    (dict(finished=P, eos=-1), SHAPE), (dict(logits=P + 4), ALIGN), (dict(ldv=1002), ALIGN), (dict(scores=P + 2), ALIGN),
    (dict(workspace=P + 8), ALIGN), (dict(parent=P + 1), ALIGN)])
def test_beam_select_refuses(kw, status):
    assert beam(**kw) == status


def test_beam_workspace_sizes():
    assert abi.nvfp4_beam_select_workspace(1, 65, 100, 148)[0] == M
    assert abi.nvfp4_beam_select_workspace(1, 4, 0, 148)[0] == SHAPE
    assert abi.nvfp4_beam_select_workspace(1, 4, 10, 0)[0] == ARG
    for g, w, v in ((1, 1, 1), (1, 64, 1 << 20), (8, 8, 151936), (64, 1, 5)):
        st, n = abi.nvfp4_beam_select_workspace(g, w, v, 148)
        assert st == abi.NVFP4_OK and 256 <= n < 1 << 27


def test_struct_layouts_match_the_header(tmp_path):
    """sizeof and the last field's offset of the argument structs, as a C compiler lays them out."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "sizes.c"
    src.write_text("#include <stdio.h>\n#include \"nvfp4decode.h\"\nint main(void) { printf(\"%zu %zu %zu %zu %zu %zu\\n\","
                   "sizeof(nvfp4_cache), offsetof(nvfp4_cache, reserved), sizeof(nvfp4_rope_args),"
                   "offsetof(nvfp4_rope_args, ldq), sizeof(nvfp4_attn_args), offsetof(nvfp4_attn_args, workspace_bytes));"
                   "return 0; }\n")
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(abi.Nvfp4Cache), abi.Nvfp4Cache.reserved.offset, ctypes.sizeof(abi.Nvfp4RopeArgs),
                   abi.Nvfp4RopeArgs.ldq.offset, ctypes.sizeof(abi.Nvfp4AttnArgs),
                   abi.Nvfp4AttnArgs.workspace_bytes.offset]


def test_packed_records_have_the_structs_layout():
    """The bytes the helpers pass are the ctypes structures field by field."""
    r = abi.Nvfp4RopeArgs.from_buffer_copy(abi._ROPE_ARGS.pack(*range(1, 17)))
    assert ctypes.sizeof(r) == abi._ROPE_ARGS.size and ctypes.addressof(r.cache.contents) == 1
    names = [n for n, _ in r._fields_][1:]
    assert [getattr(r, n) for n in names] == list(range(2, 17))
    a = abi.Nvfp4AttnArgs.from_buffer_copy(abi._ATTN_ARGS.pack(*range(1, 17)))
    assert ctypes.sizeof(a) == abi._ATTN_ARGS.size and ctypes.addressof(a.cache.contents) == 1
    assert [getattr(a, n) for n in [n for n, _ in a._fields_][1:]] == list(range(2, 17))


def test_helpers_refuse_host_tensors():
    import torch
    k = torch.zeros((1, 2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        abi.Cache(k, k, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                  torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device memory"):
        abi.beam_select(torch.zeros((4, 8)), torch.zeros((1, 4)))


# ------------------------------------------- the references, by hand

def tiny():
    k = np.arange(1 * 4 * 1 * 16 * 2, dtype=np.uint16).reshape(1, 4, 1, 16, 2)
    table = np.array([[2, -1], [0, -1]], np.int32)
    return cache_ref.RefCache(k, k + 1000, table, np.array([3, 2], np.int32), np.array([1, 0, 1, 0], np.int32))


def test_helpers_refuse_a_stream_of_another_device():
    torch = pytest.importorskip("torch")
    here, there = torch.device("cuda", 0), types.SimpleNamespace(device=torch.device("cuda", 1))
    on = types.SimpleNamespace(device=here)  # of the tensors, no more than their device is looked at
    for call in (lambda: abi.rope_append(on, 0, None, 8, None, None, stream=there),
                 lambda: abi.attn_tree(on, 0, None, 1.0, stream=there),
                 lambda: abi.beam_select(on, None, stream=there)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_reference_fork_reserve_compact_trim():
    c = tiny()
    c.fork([0, 0])
    assert c.table.tolist() == [[2, -1], [2, -1]] and c.ref.tolist() == [0, 0, 2, 0] and c.len.tolist() == [3, 3]
    assert c.reserve([1, 14])  # lane 0 copies page 2 to page 0; lane 1 keeps it and takes page 1
    assert c.table.tolist() == [[0, -1], [2, 1]] and c.ref.tolist() == [1, 1, 1, 0]
    assert np.array_equal(c.k[0, 0, 0, :3], c.k[0, 2, 0, :3]) and not np.array_equal(c.k[0, 0, 0, 3], c.k[0, 2, 0, 3])
    want = c.k[0, 2, 0, [4, 7]].copy()
    c.compact([0, 2], [[0, 0], [1, 4]])
    assert c.len.tolist() == [3, 5] and np.array_equal(c.k[0, 2, 0, 3:5], want)
    assert c.table.tolist() == [[0, -1], [2, -1]] and c.ref.tolist() == [1, 0, 1, 0]
    assert not c.reserve([40, 0]) and c.table.tolist() == [[0, -1], [2, -1]]
    c.trim([0, 5])
    assert c.table.tolist() == [[-1, -1], [2, -1]] and c.ref.tolist() == [0, 0, 1, 0] and c.len.tolist() == [0, 5]


def test_reference_rope_and_attention_and_beam():
    out, _ = cache_ref.rope(np.array([[1.0, 0.0, 2.0, 0.0]]), 1, 4, np.array([[1]]), [0, 0], [np.pi / 2, 0.0], 0)
    assert np.allclose(out[0, 0], [-2.0, 0.0, 1.0, 0.0])  # pair (0, 2) by a quarter turn
    c = tiny()
    one = cache_ref.bf16_bits(np.ones(2))
    c.k[:], c.v[:] = 0, one
    c.v[0, 2, 0, 3] = cache_ref.bf16_bits(np.array([5.0, -3.0]))
    out, lse, _, _, seen = cache_ref.attention(c, 0, np.ones((1, 1, 2)), 1.0, [0, 1, 1], [1])
    assert seen[0] == 4 and np.isclose(lse[0, 0], np.log(4.0)) and np.allclose(out[0, 0], [2.0, 0.0])
    s, p, t, f = cache_ref.beam(np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]])), np.array([[0.0, -0.1]]), None, 0)
    assert p.tolist() == [[1, 0]] and t.tolist() == [[2, 0]] and f.tolist() == [[0, 1]]
    assert np.allclose(s, [[np.log(0.7) - 0.1, np.log(0.5)]])
