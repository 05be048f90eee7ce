"""The cache's operators together, as decoding uses them: a decode round with
attention between its GEMMs, a beam search, and drafting with verification."""
import numpy as np
import pytest
import torch

import cache_helpers as ch
import cache_ref
from nvfp4_weight_streaming_decode_b200 import abi
from nvfp4_weight_streaming_decode_b200.workloads import SyntheticRound

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


@pytest.mark.parametrize("kv_heads,context", [(2, 300), (4, 0)])
def test_round_with_attention(dev, kv_heads, context):
    """Replay equals the direct calls bit for bit; the attention of each layer is the reference's on the round's own
    q/k/v outputs; o reads it."""
    r = SyntheticRound.build(dev, layers=2, hidden=512, ffn=1024, vocab=2048, workload_id=11, kv_heads=kv_heads,
                             context=context)
    rnd = abi.Round(r.descs)
    assert rnd.nodes >= len(r.descs)
    heads, D = 4, 128
    for M in (1, 3, 8):
        for b in ("a0", "a1", "yo0", "yo1", "logits"):
            r.bufs[b].zero_()
        k0, v0 = r.cache.k.clone(), r.cache.v.clone()
        r.run_direct(M)
        torch.cuda.synchronize()
        direct = {b: r.bufs[b].clone() for b in ("a0", "a1", "yo0", "yo1", "logits")}
        kd, vd = r.cache.k.clone(), r.cache.v.clone()
        for b in direct:
            r.bufs[b].zero_()
        r.cache.k.copy_(k0)
        r.cache.v.copy_(v0)
        rnd.replay(M, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for b, t in direct.items():
            assert torch.equal(r.bufs[b], t), (M, b)
        assert torch.equal(r.cache.k, kd) and torch.equal(r.cache.v, vd)
        # layer 1 against the reference: its q/k/v output rotated, appended and attended to
        y = r.bufs["yqkv1"][:M].cpu().numpy()
        f = r.bufs["inv_freq"].cpu().numpy()
        x, _ = cache_ref.rope(y, heads + 2 * kv_heads, D, np.full((1, M), context), np.zeros(64, int), f, 0)
        ref = cache_ref.RefCache(ch.host_bits(kd), ch.host_bits(vd), r.cache.table.cpu().numpy(),
                                 r.cache.len.cpu().numpy(), r.cache.ref.cpu().numpy())
        for b in range(M):
            p, o = ref.where(b, context)
            got = cache_ref.bf16_value(ref.k[1, p, :, o])
            assert np.allclose(got, x[b, heads:heads + kv_heads], rtol=2.0**-7, atol=1e-4)
        q = cache_ref.bf16_value(cache_ref.bf16_bits(x[:, :heads])).astype(np.float64)
        # a rotated value may fall to the other side of a bf16 border than in 64 bits: one step of q, which moves a
        # score by at most 2^-7 of the summed magnitudes
        want, _, wabs, err, _ = cache_ref.attention(ref, 1, q, float(np.float32(D**-0.5)), list(range(M + 1)) + [M] * (8 - M), None)
        got = r.bufs["a1"][:M].float().cpu().numpy().reshape(M, heads, D)
        slack = 2 * err[:, :, None] * 2.0**17 / (D + 4) + 2.0**-6
        assert (np.abs(got - want) <= wabs * slack + np.abs(want) * 2.0**-8 + 1e-6).all()
    rnd.close()


def step(c, layer_in, q_heads, f, pos, scale, start=None, mask=None, nodes=1):
    """One layer's rotary append and attention of rows layer_in."""
    q = abi.rope_append(c, 0, layer_in, q_heads, f, pos, row_start=start)
    return abi.attn_tree(c, 0, q, scale, row_start=start, mask=mask, max_nodes=nodes)


class Tiny:
    """One attention layer over drawn embeddings and a drawn output matrix; logits of a token history in 64 bits too."""

    def __init__(self, dev, seed, vocab=64, hq=4, hkv=2, dim=64):
        rng = np.random.default_rng(seed)
        self.dev, self.hq, self.hkv, self.dim, self.vocab = dev, hq, hkv, dim, vocab
        self.embed = (rng.standard_normal((vocab, (hq + 2 * hkv) * dim)) * 0.8).astype(np.float32)
        self.out = rng.standard_normal((hq * dim, vocab)) * 0.25
        self.f = 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
        self.e_dev, self.o_dev = torch.from_numpy(self.embed).to(dev), torch.from_numpy(self.out.astype(np.float32)).to(dev)
        self.f_dev, self.scale = torch.from_numpy(self.f).to(dev), dim**-0.5

    def logits(self, attn):
        return attn.float().reshape(attn.shape[0], -1) @ self.o_dev

    def exact(self, tokens):
        """Logits behind a token history, every key and value anew (rounded to bf16 where the cache is)."""
        n = len(tokens)
        x, _ = cache_ref.rope(self.embed[tokens], self.hq + 2 * self.hkv, self.dim, np.arange(n)[None], np.zeros(self.dim // 2, int),
                              self.f, 0)
        x[:, self.hq + self.hkv:] = self.embed[tokens].reshape(n, -1, self.dim)[:, self.hq + self.hkv:]  # values keep theirs
        b = cache_ref.bf16_value(cache_ref.bf16_bits(x)).astype(np.float64)
        q, k, v = b[-1, :self.hq], b[:, self.hq:self.hq + self.hkv], b[:, self.hq + self.hkv:]
        o = np.zeros((self.hq, self.dim))
        for h in range(self.hq):
            s = self.scale * k[:, h // 2] @ q[h]
            p = np.exp(s - s.max())
            o[h] = p @ v[:, h // 2] / p.sum()
        return o.reshape(-1) @ self.out


def test_beam_search(dev):
    """Sixteen steps of two groups of four beams: select, fork, reserve, append, attend, commit.  Every step's logits
    are those of the beams' token histories, computed anew; at the end all pages can be freed."""
    m, groups, beams, lanes = Tiny(dev, 3), 2, 4, 8
    c = abi.Cache.empty(1, 60, m.hkv, 16, m.dim, lanes, 8, dev)
    ones = ch.ints([1] * lanes, dev)
    hist = [[7 + i // beams] for i in range(lanes)]
    scores = torch.full((groups, beams), -np.inf, device=dev)
    scores[:, 0] = 0.0
    ws = abi.beam_select_workspace(groups, beams, m.vocab, dev)
    work = abi.attn_tree_workspace(c, lanes, m.hq)
    for t in range(16):
        c.reserve(ones)
        tok = torch.tensor([h[-1] for h in hist], device=dev)
        q = abi.rope_append(c, 0, m.e_dev[tok].contiguous(), m.hq, m.f_dev, ch.ints([t] * lanes, dev))
        x = m.logits(abi.attn_tree(c, 0, q, m.scale, workspace=work))
        c.compact(ones)
        got = x.cpu().numpy()
        for i in range(lanes):
            want = m.exact(hist[i])
            assert np.abs(got[i] - want).max() <= 0.02 * np.abs(want).max(), (t, i)
        s0 = scores.cpu().numpy()
        scores, parent, token, _ = abi.beam_select(x, scores, workspace=ws)
        s, p, tk = scores.cpu().numpy(), parent.cpu().numpy().reshape(-1), token.cpu().numpy().reshape(-1)
        rs, rp, rt, _ = cache_ref.beam(got, s0.astype(np.float64), None, -1)
        assert np.array_equal(p, rp.reshape(-1)) and np.array_equal(tk, rt.reshape(-1))
        assert np.allclose(s, rs, rtol=1e-6, atol=1e-6)
        c.fork(parent.view(-1))
        hist = [hist[a] + [int(b)] for a, b in zip(p, tk)]
    c.fork(ch.ints([-1] * lanes, dev))
    assert not c.ref.any() and (c.table == -1).all()


def test_draft_and_verify(dev):
    """A tree of drafts per lane is appended and attended in one call; each node's logits are those of its path's
    history; the accepted path is compacted and decoding goes on from it."""
    m, lanes = Tiny(dev, 4), 3
    rng = np.random.default_rng(5)
    c = abi.Cache.empty(1, 40, m.hkv, 16, m.dim, lanes, 12, dev)
    hist = [[1], [2, 9, 4], []]
    pos = lambda h: list(range(len(h)))  # noqa: E731
    # prompts: chains of different lengths, one lane empty
    start = np.concatenate([[0], np.cumsum([len(h) for h in hist])])
    toks = [t for h in hist for t in h]
    c.reserve(ch.ints([len(h) for h in hist], dev))
    step(c, m.e_dev[torch.tensor(toks, device=dev)].contiguous(), m.hq, m.f_dev, ch.ints([p for h in hist for p in pos(h)], dev),
         m.scale, ch.ints(start, dev), None, 3)
    c.compact(ch.ints([len(h) for h in hist], dev))
    for rnd in range(6):
        counts = [int(rng.integers(1, 9)) for _ in range(lanes)]
        start = np.concatenate([[0], np.cumsum(counts)])
        parents, tokens, masks, posn, paths = [], [], [], [], []
        for b, n in enumerate(counts):
            anc = []
            for i in range(n):
                par = int(rng.integers(-1, i)) if i else -1
                anc.append((anc[par] if par >= 0 else []) + [i])
                tokens.append(int(rng.integers(0, m.vocab)))
                masks.append(sum(1 << j for j in anc[-1]))
                posn.append(len(hist[b]) + len(anc[-1]) - 1)
            paths.append(anc)
        c.reserve(ch.ints(counts, dev))
        a = step(c, m.e_dev[torch.tensor(tokens, device=dev)].contiguous(), m.hq, m.f_dev, ch.ints(posn, dev), m.scale,
                 ch.ints(start, dev), ch.words(masks, dev), 8)
        got = m.logits(a).cpu().numpy()
        take, count = np.zeros((lanes, 8), np.int32), []
        for b in range(lanes):
            for i in range(counts[b]):
                want = m.exact(hist[b] + [tokens[start[b] + j] for j in paths[b][i]])
                assert np.abs(got[start[b] + i] - want).max() <= 0.02 * np.abs(want).max(), (rnd, b, i)
            path = paths[b][int(rng.integers(0, counts[b]))] if rng.random() < 0.8 else []
            take[b, :len(path)] = path
            count.append(len(path))
            hist[b] = hist[b] + [tokens[start[b] + j] for j in path]
        c.compact(ch.ints(count, dev), ch.ints(take, dev))
        assert c.len.cpu().tolist() == [len(h) for h in hist]
    c.trim(ch.ints([0] * lanes, dev))
    assert not c.ref.any()


def test_pools_past_32_bits(dev):
    """Pools of 4.3 G values: append, attention, fork with copy, compact in pages whose offsets need 64 bits."""
    pages, hkv, page, D = (1 << 20) + 16, 2, 16, 128
    k = torch.zeros((1, pages, hkv, page, D), dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    table = np.full((2, 6), -1, np.int32)
    table[0, :3] = [pages - 1, pages - 3, pages - 5]
    table[1, :3] = [pages - 11, pages - 2, pages - 8]
    ref = torch.ones(pages, dtype=torch.int32, device=dev)  # all taken but two at the far end
    ref[[pages - 7, pages - 9]] = 0
    c = abi.Cache(k, v, ch.ints(table, dev), ch.ints([0, 0], dev), ref)
    counts, f = [40, 37], torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).to(dev)
    rows = sum(counts)
    y = torch.randn((rows, (4 + 2 * hkv) * D), generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    start = ch.ints([0, 40, 77], dev)
    pos = ch.ints(list(range(40)) + list(range(37)), dev)
    q = abi.rope_append(c, 0, y, 4, f, pos, row_start=start)

    def small():
        """The pages in use, renumbered, as the reference."""
        used = sorted({int(p) for p in c.table.cpu().numpy().ravel() if p >= 0})
        at = {p: i for i, p in enumerate(used)}
        idx = torch.tensor(used, device=dev)
        tab = np.vectorize(lambda p: at.get(int(p), -1))(c.table.cpu().numpy()).astype(np.int32)
        return cache_ref.RefCache(ch.host_bits(k[:, idx]), ch.host_bits(v[:, idx]), tab, c.len.cpu().numpy(),
                                  np.ones(len(used), np.int32))
    r = small()
    x, _ = cache_ref.rope(y.cpu().numpy(), 4 + 2 * hkv, D, pos.cpu().numpy()[None], np.zeros(64, int), f.cpu().numpy(), 0)
    for lane, n in enumerate(counts):
        for i in range(n):
            p, o = r.where(lane, i)
            assert np.allclose(cache_ref.bf16_value(r.k[0, p, :, o]), x[40 * lane + i, 4:6], rtol=2.0**-7, atol=1e-4)
    c.compact(ch.ints(counts, dev))
    # lane 1 becomes lane 0's twin: its next slot takes a copy of the far last page
    c.fork(ch.ints([0, 0], dev))
    c.reserve(ch.ints([4, 4], dev))
    assert sorted(c.table[:, 2].tolist()) == [pages - 11, pages - 5]  # the lowest page that the fork freed
    more = torch.randn((8, (4 + 2 * hkv) * D), device=dev)
    q = abi.rope_append(c, 0, more, 4, f, ch.ints([40, 41, 42, 43] * 2, dev), row_start=ch.ints([0, 4, 8], dev))
    out, lse = abi.attn_tree(c, 0, q, 0.1, row_start=ch.ints([0, 4, 8], dev), max_nodes=4, want_lse=True)
    r = small()
    qh = cache_ref.bf16_value(ch.host_bits(q)).astype(np.float64)
    want, wl, wabs, err, seen = cache_ref.attention(r, 0, qh, float(np.float32(0.1)), [0, 4, 8], None)
    tol = wabs * (2 * err[:, :, None] + 2.0**-8 + 2.0**-20) * 1.01 + np.abs(want) * 2.0**-8 * 1.01
    assert (np.abs(out.float().cpu().numpy() - want) <= tol).all() and (seen == [41, 42, 43, 44] * 2).all()
    c.compact(ch.ints([2, 1], dev), ch.ints([[1, 3, 0, 0], [2, 0, 0, 0]], dev))
    r.compact([2, 1], [[1, 3, 0, 0], [2, 0, 0, 0]])
    s = small()
    for lane, n in ((0, 42), (1, 41)):
        for i in range(n):
            (p, o), (p2, o2) = r.where(lane, i), s.where(lane, i)
            assert np.array_equal(r.k[0, p, :, o], s.k[0, p2, :, o2]) and np.array_equal(r.v[0, p, :, o], s.v[0, p2, :, o2])


FIRST = """
import sys; sys.path[:0] = ['tests', '.']
import torch, cache_helpers as ch
from nvfp4_weight_streaming_decode_b200 import abi
dev = torch.device('cuda', 0)
c, r = ch.make(dev, 1, [200, 30], [4, 4], hkv=2, page=16, dim=128)
y, x, s = torch.randn((2, 8 * 128), device=dev), torch.randn((4, 3000), device=dev), torch.zeros((1, 4), device=dev)
one, keep = ch.ints([1, 1], dev), ch.ints([0, 1], dev)
q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device=dev)
work, ws = abi.attn_tree_workspace(c, 2, 4), abi.beam_select_workspace(1, 4, 3000, dev)
out = torch.zeros_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.fork(keep); c.reserve(one); abi.rope_append(c, 0, y, 4, None, None, q=q)
    abi.attn_tree(c, 0, q, 0.1, out=out, workspace=work); c.compact(one); c.trim(ch_len)
    b = abi.beam_select(x, s, workspace=ws)
g.replay(); torch.cuda.synchronize()
assert out.abs().sum() > 0 and c.len.tolist() == [200, 30] and (b[1] >= 0).all() and abi.nvfp4_device_status() == 0
print('captured first')
"""


def test_first_calls_may_be_captured(dev):
    """In a new process, every operator's first call inside a stream capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = FIRST.replace("ch_len", "keep_len").replace("one, keep =", "keep_len = ch.ints([200, 30], dev)\none, keep =")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured first", r.stderr[-2000:]
