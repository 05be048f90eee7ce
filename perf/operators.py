"""Measured cases of the operators around the decode GEMMs: attention over the
paged cache, rotary positions with the append to it, the cache's page
operations, and beam selection over the head's logits.

``own`` False computes each operator in its plain form (elementary torch
operations); True makes the calls a user makes of the framework.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a lane's first token: nothing cached but itself; pure latency
        dict(name="attn_first_token", op="attn", lanes=1, nodes=1, ragged=False, hq=40, hkv=8, d=128, page=16, ctx=0,
             tree="chain"),
        # the round's decode step: 8 lanes, 40 heads of 128 each with its own keys, ragged contexts
        dict(name="attn_round", op="attn", lanes=8, nodes=1, ragged=False, hq=40, hkv=40, d=128, page=64, ctx=4000,
             tree="chain"),
        # verify: 8 lanes x (1 + 7 drafts) over long ragged contexts, grouped heads
        dict(name="attn_verify", op="attn", lanes=8, nodes=8, ragged=False, hq=40, hkv=8, d=128, page=64, ctx=32768,
             tree="tree"),
        # one lane's wide tree of 64 nodes over a long context (the largest: 512 query rows per cached head)
        dict(name="attn_wide_tree", op="attn", lanes=1, nodes=64, ragged=False, hq=64, hkv=8, d=128, page=128,
             ctx=65537, tree="tree"),
        # long heads, short pages, lanes with different numbers of drafts
        dict(name="attn_d256_ragged", op="attn", lanes=5, nodes=8, ragged=True, hq=24, hkv=4, d=256, page=16,
             ctx=20011, tree="tree"),
        # the round's q/k/v output (8 rows of 15,360) rotated and appended
        dict(name="rope_round", op="rope", lanes=8, nodes=1, hq=40, hkv=40, d=128, rot=128, axes=1, style=0, page=64,
             ctx=2000),
        # verify rows with image positions on three axes, part of each head rotated, adjacent pairs
        dict(name="rope_verify_axes", op="rope", lanes=8, nodes=8, hq=24, hkv=4, d=256, rot=64, axes=3, style=1,
             page=16, ctx=100003),
        # a prompt's rows into the cache
        dict(name="rope_prompt", op="rope", lanes=3, nodes=2731, hq=40, hkv=8, d=128, rot=128, axes=1, style=0,
             page=64, ctx=100),
        # one beam step's reordering: fork by parent, then room for the next token (copies of shared last pages)
        dict(name="cache_beam_step", op="fork", lanes=8, layers=64, hkv=8, d=128, page=64, ctx=2031),
        # after verify: back to the committed length, room for 8 drafts, keep each lane's accepted path
        dict(name="cache_verify_accept", op="compact", lanes=8, nodes=8, layers=64, hkv=8, d=128, page=64, ctx=500),
        # a small vocabulary, one group of 4 beams
        dict(name="beam_small", op="beam", groups=1, beams=4, vocab=1000, done=False),
        # 8 groups of 8 beams over the head's 151,936 logits, some beams finished
        dict(name="beam_head", op="beam", groups=8, beams=8, vocab=151936, done=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "fork", "compact", "beam"])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    if op == "attn":
        g = rng.choice([1, 3, 4, 5, 6, 8])
        lanes = rng.randint(1, 8)
        nodes = min(_log(rng, 1, 64), 64 // lanes)
        ctx = _log(rng, 1, 32768 * 8 // max(lanes, 8))
        # no more multiplications than the largest listed case
        while lanes * nodes * g * hkv * d * ctx > 64 * 64 * 128 * 65537:
            ctx //= 2
        return dict(op="attn", lanes=lanes, nodes=nodes, ragged=rng.random() < 0.5, hq=g * hkv, hkv=hkv, d=d,
                    page=page, ctx=ctx, tree=rng.choice(["chain", "tree"]))
    if op == "rope":
        g = rng.choice([1, 3, 5, 8])
        lanes = rng.randint(1, 8)
        return dict(op="rope", lanes=lanes, nodes=_log(rng, 1, 1024), hq=g * hkv, hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), axes=rng.randint(1, 4), style=rng.randint(0, 1), page=page,
                    ctx=_log(rng, 1, 200000 // lanes))
    if op in ("fork", "compact"):
        case = dict(op=op, lanes=rng.randint(2, 8), layers=_log(rng, 1, 48), hkv=hkv, d=d, page=page,
                    ctx=_log(rng, 1, 900))
        if op == "compact":
            case["nodes"] = rng.randint(2, 8)
        return case
    return dict(op="beam", groups=rng.randint(1, 8), beams=rng.randint(1, 8), vocab=_log(rng, 50, 151936),
                done=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _spread(i):
    """Numbers of (0, 1] without an order to them, the first one 1."""
    return 1.0 - i * 0.6180339887 % 1.0


def _lens(case):
    """Ragged context lengths, the first lane at the case's own."""
    return [round((0.25 + 0.75 * _spread(i)) * case["ctx"]) for i in range(case["lanes"])]


def _counts(case):
    """Rows of each lane: all of them, or any number from one."""
    t = case["nodes"]
    return [max(1, round(t * _spread(i))) if case.get("ragged") else t for i in range(case["lanes"])]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pools(case, layers, pages, gen):
    shape = (layers, pages, case["hkv"], case["page"], case["d"])
    k = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    return k, v


def _paged(case, need, layers, gen, spare=3):
    """Page tables that hold `need` slots per lane, pages in scattered order."""
    page = case["page"]
    per = (need.long() + page - 1) // page
    most = int(per.max())
    total = int(per.sum())
    pages = total + spare
    order = torch.randperm(pages, generator=gen, device=DEV)[:total].to(torch.int32)
    width = most + 2
    col = torch.arange(width, device=DEV)
    used = col[None, :] < per[:, None]
    table = torch.full((case["lanes"], width), -1, dtype=torch.int32, device=DEV)
    table[used] = order
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[order.long()] = 1
    k, v = _pools(case, layers, pages, gen)
    return k, v, table, ref


def _row_layout(counts):
    start = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=DEV)
    start[1:] = counts.cumsum(0)
    lane = torch.repeat_interleave(torch.arange(counts.numel(), device=DEV), counts.long())
    node = torch.arange(lane.numel(), device=DEV) - start.long()[lane]
    return start, lane, node


def _tree_mask(node, gen):
    """Each node sees itself and its ancestors; a node's parent comes before it."""
    rows = node.numel()
    parent = (torch.rand(rows, generator=gen, device=DEV) * node).long().cpu().tolist()
    first = (torch.arange(rows, device=DEV) - node).cpu().tolist()
    nd = node.cpu().tolist()
    bits = []
    for r in range(rows):
        up = bits[first[r] + parent[r]] if nd[r] else 0
        bits.append(up | (1 << nd[r]))
    return bits


def _prepare_attn(case, seed):
    gen = _gen(seed)
    lens, counts = _ints(_lens(case)), _ints(_counts(case))
    start, lane, node = _row_layout(counts)
    k, v, table, ref = _paged(case, lens + counts, 1, gen)
    rows = int(start[-1])
    q = torch.randn((rows, case["hq"], case["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
    if case["tree"] == "chain":
        mask = None
    else:
        bits = _tree_mask(node, gen)
        mask = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=DEV)
    s = dict(op="attn", q=q, mask=mask, start=start if case["nodes"] > 1 else None, lane=lane, node=node,
             nodes=case["nodes"], most=int((lens + counts).max()), scale=case["d"] ** -0.5)
    return _with_cache(s, case, k, v, table, lens, ref)


def _prepare_rope(case, seed):
    gen = _gen(seed)
    lens, counts = _ints(_lens(case)), _ints(_counts(case))
    start, lane, node = _row_layout(counts)
    rows, d = int(start[-1]), case["d"]
    # far contexts need their table, not a page of memory per slot: lanes share the pool's pages below their length
    page = case["page"]
    first = lens.long() // page
    per = (lens.long() + counts + page - 1) // page - first
    total = int(per.sum())
    width = int((first + per).max()) + 1
    table = torch.zeros((case["lanes"], width), dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= first[:, None]) & (col < (first + per)[:, None])
    table[fresh] = 1 + torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table[col.expand_as(table) >= (first + per)[:, None]] = -1
    ref = torch.ones(total + 1, dtype=torch.int32, device=DEV)
    ref[0] = max(2, int(first.sum()))
    k, v = _pools(case, 2, total + 1, gen)
    width_y = (case["hq"] + 2 * case["hkv"]) * d
    y = torch.randn((rows, width_y), generator=gen, device=DEV)
    half = case["rot"] // 2
    inv_freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    base = lens.long()[lane] + node
    pos = torch.stack([base + 17 * a * (node % 13) for a in range(case["axes"])]).to(torch.int32).contiguous()
    axis = (torch.arange(half, device=DEV) * case["axes"] // half).to(torch.uint8)
    q = torch.zeros((rows, case["hq"], d), dtype=torch.bfloat16, device=DEV)
    s = dict(op="rope", y=y, pos=pos, inv_freq=inv_freq, axis=axis, q=q, style=case["style"], lane=lane, node=node,
             start=start if case["nodes"] > 1 else None, rot=case["rot"])
    return _with_cache(s, case, k, v, table, lens, ref)


def _prepare_pages(case, seed):
    gen = _gen(seed)
    lens = _ints(_lens(case)).clamp(min=1)
    lanes, page = case["lanes"], case["page"]
    if case["op"] == "fork":
        lens = lens + (lens % page == 0).int()  # a last page that is partly filled
        # beams of one sequence: as long as each other
        lens[:] = lens[0]
        spare = lanes + 2
        parent = torch.randint(0, lanes, (lanes,), generator=gen, device=DEV).sort().values.to(torch.int32)
        s = dict(op="fork", parent=parent, want=torch.ones(lanes, dtype=torch.int32, device=DEV))
        # as after earlier steps: the later beams hold the first one's full pages
        k, v, table, ref = _paged(case, lens, case["layers"], gen, spare=spare)
        full = int(lens[0]) // page
        shared = table[0, :full].long()
        old = table[1:, :full].reshape(-1).long()
        ref[old] = 0
        table[1:, :full] = table[0, :full]
        ref[shared] = lanes
    else:
        nodes = case["nodes"]
        spare = lanes * (nodes // page + 2)
        k, v, table, ref = _paged(case, lens, case["layers"], gen, spare=spare)
        pick = torch.rand((lanes, nodes), generator=gen, device=DEV) < 0.5
        pick[0] = torch.arange(nodes, device=DEV) % 2 == 1
        count = pick.sum(1).to(torch.int32)
        order = torch.where(pick, torch.arange(nodes, device=DEV), nodes).sort(1).values
        path = torch.where(order < nodes, order, 0).to(torch.int32).contiguous()
        s = dict(op="compact", back=lens.clone(), want=torch.full((lanes,), nodes, dtype=torch.int32, device=DEV),
                 path=path, count=count)
    width = table.shape[1] + 1
    table = torch.cat([table, torch.full((lanes, width - table.shape[1]), -1, dtype=torch.int32, device=DEV)], 1)
    return _with_cache(s, case, k, v, table.contiguous(), lens, ref)


def _with_cache(s, case, k, v, table, lens, ref):
    s.update(k=k, v=v, table=table, len=lens, ref=ref, page=case["page"])
    if own:
        from nvfp4_weight_streaming_decode_b200 import abi
        s["cache"] = abi.Cache(k=k, v=v, table=table, len=lens, ref=ref)
        if s["op"] == "attn":
            s["work"] = abi.attn_tree_workspace(s["cache"], s["q"].shape[0], s["q"].shape[1])
    return s


def _prepare_beam(case, seed):
    gen = _gen(seed)
    g, w, v = case["groups"], case["beams"], case["vocab"]
    ld = (v + 3) // 4 * 4
    logits = torch.randn((g * w, ld), generator=gen, device=DEV) * 2.5
    scores = -8.0 * torch.rand((g, w), generator=gen, device=DEV)
    done = (torch.rand((g, w), generator=gen, device=DEV) < 0.2).to(torch.uint8) if case["done"] else None
    s = dict(op="beam", logits=logits, scores=scores, done=done, vocab=v, eos=2)
    if own:
        from nvfp4_weight_streaming_decode_b200 import abi
        s["work"] = abi.beam_select_workspace(g, w, v, logits.device)
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "attn":
        return _prepare_attn(case, seed)
    if op == "rope":
        return _prepare_rope(case, seed)
    if op in ("fork", "compact"):
        return _prepare_pages(case, seed)
    return _prepare_beam(case, seed)


# ------------------------------------------------------------ plain forms

def _plain_attn(s):
    q, table, lens, page = s["q"], s["table"], s["len"], s["page"]
    rows, hq, d = q.shape
    hkv = s["k"].shape[2]
    g, n, t = hq // hkv, table.shape[0], s["nodes"]
    width = (s["most"] + page - 1) // page
    at = table[:, :width].clamp(min=0).long()
    # [lanes][kv heads][slots][d], in 32 bits
    k = s["k"][0][at].transpose(1, 2).reshape(n, hkv, width * page, d).float()
    v = s["v"][0][at].transpose(1, 2).reshape(n, hkv, width * page, d).float()
    slot = torch.arange(width * page, device=q.device)
    j = slot[None, :] - lens[:, None]
    jr = j[s["lane"]]
    if s["mask"] is None:
        drafted = jr <= s["node"][:, None]
    else:
        drafted = (s["mask"][:, None] >> jr.clamp(0, 63)) & 1 == 1
        drafted &= jr < 64
    seen_row = (jr < 0) | ((jr >= 0) & drafted)
    count = torch.zeros(n, dtype=torch.long, device=q.device).index_add_(0, s["lane"], torch.ones_like(s["lane"]))
    seen_row &= jr < count[s["lane"]][:, None]
    qp = torch.zeros((n, t, hq, d), device=q.device)
    qp[s["lane"], s["node"]] = q.float()
    seen = torch.zeros((n, t, width * page), dtype=torch.bool, device=q.device)
    seen[s["lane"], s["node"]] = seen_row
    qp = qp.reshape(n, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, t * g, d)
    x = torch.matmul(qp, k.transpose(2, 3)) * s["scale"]
    hide = ~seen[:, None, :, None, :]
    x = x.reshape(n, hkv, t, g, -1).masked_fill_(hide, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    o = torch.matmul(p.reshape(n, hkv, t * g, -1), v).reshape(n, hkv, t, g, d)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, t, hq, d)[s["lane"], s["node"]]
    lse = lse.permute(0, 2, 1, 3, 4).reshape(n, t, hq)[s["lane"], s["node"]]
    return o.to(torch.bfloat16), lse


def _turn(x, c, sn, rot, style):
    """Rotate the first `rot` values of each head of x [rows][heads][d]."""
    r = x[..., :rot]
    if style == 0:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rope(s):
    rows, hq, d = s["q"].shape
    hkv, page = s["k"].shape[2], s["page"]
    angle = s["pos"].double()[s["axis"].long()].T * s["inv_freq"]
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = s["y"].reshape(rows, hq + 2 * hkv, d)
    s["q"].copy_(_turn(y[:, :hq], c, sn, s["rot"], s["style"]))
    slot = s["len"].long()[s["lane"]] + s["node"]
    at, off = s["table"][s["lane"], slot // page].long(), slot % page
    s["k"][1][at, :, off] = _turn(y[:, hq:hq + hkv], c, sn, s["rot"], s["style"]).to(torch.bfloat16)
    s["v"][1][at, :, off] = y[:, hq + hkv:].to(torch.bfloat16)
    return s["q"], s["k"], s["v"]


def _plain_release(s, keep):
    """Lanes keep their first `keep` pages; the others lose a reference."""
    col = torch.arange(s["table"].shape[1], device=keep.device)
    drop = (col[None, :] >= keep[:, None]) & (s["table"] >= 0)
    s["ref"].index_add_(0, s["table"].clamp(min=0).reshape(-1).long(), -drop.reshape(-1).int())
    s["table"].masked_fill_(drop, -1)


def _plain_fork(s):
    old = s["table"]
    new = old[s["parent"].long()]
    s["ref"].index_add_(0, new.clamp(min=0).reshape(-1).long(), (new >= 0).reshape(-1).int())
    s["ref"].index_add_(0, old.clamp(min=0).reshape(-1).long(), -(old >= 0).reshape(-1).int())
    old.copy_(new)
    s["len"].copy_(s["len"][s["parent"].long()])


def _plain_reserve(s):
    """Room for `want` more slots: copies of shared last pages, then new pages,
    the lowest free ones in lane order."""
    table, lens, ref, page = s["table"], s["len"].long(), s["ref"], s["page"]
    n, width = table.shape
    lane = torch.arange(n, device=table.device)
    fill = lens % page
    lastc = (lens // page).clamp(max=width - 1)
    last = table[lane, lastc].long()
    write = (fill > 0) & (s["want"] > 0)
    before = ((last[None, :] == last[:, None]) & write[None, :] & (lane[None, :] < lane[:, None])).sum(1)
    copy = write & (ref[last.clamp(min=0)] - before > 1)
    col = torch.arange(width, device=table.device)
    held = (table >= 0).sum(1)
    upto = (lens + s["want"] + page - 1) // page
    fresh = (col[None, :] >= held[:, None]) & (col[None, :] < upto[:, None])
    take = fresh | ((col[None, :] == lastc[:, None]) & copy[:, None])
    # the n-th page taken (lane by lane, column by column) is the n-th free page
    nth = take.reshape(-1).cumsum(0).reshape(n, width) - 1
    free = (ref != 0).to(torch.int8).sort(stable=True).indices
    page_of = free[nth.clamp(0, free.numel() - 1)]
    dst = torch.where(copy, page_of[lane, lastc], last.clamp(min=0))
    ref.index_add_(0, last.clamp(min=0), -copy.int())
    ref.index_add_(0, page_of.reshape(-1), take.reshape(-1).int())
    table.copy_(torch.where(take, page_of.int(), table))
    part = (torch.arange(page, device=table.device)[None, :] < fill[:, None])[None, :, None, :, None]
    src = last.clamp(min=0)
    for pool in (s["k"], s["v"]):
        pool[:, dst] = torch.where(part, pool[:, src], pool[:, dst])


def _plain_compact(s):
    table, page, path, count = s["table"], s["page"], s["path"], s["count"]
    n, most = path.shape
    lane = torch.arange(n, device=table.device)[:, None].expand(n, most)
    j = torch.arange(most, device=table.device)[None, :].expand(n, most)
    lens = s["len"].long()[:, None]
    frm = torch.where(j < count[:, None], lens + path, lens + j)
    to = lens + j
    for pool in (s["k"], s["v"]):
        pool[:, table[lane, to // page].long(), :, to % page] = pool[:, table[lane, frm // page].long(), :, frm % page]
    s["len"] += count
    _plain_release(s, (s["len"] + page - 1) // page)


def _plain_pages(s):
    if s["op"] == "fork":
        _plain_fork(s)
        _plain_reserve(s)
    else:
        s["len"].copy_(torch.minimum(s["back"], s["len"]))
        _plain_release(s, (s["len"] + s["page"] - 1) // s["page"])
        _plain_reserve(s)
        _plain_compact(s)
    return s["k"], s["v"], s["table"], s["len"], s["ref"]


def _plain_beam(s):
    g, w = s["scores"].shape
    v = s["vocab"]
    # in 64 bits: candidates of different beams that nearly tie
    x = s["logits"][:, :v].reshape(g, w, v).double()
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    x = s["scores"].double()[..., None] + (x - lse)
    if s["done"] is not None:
        over = s["done"].bool()[..., None]
        eos = torch.arange(v, device=x.device) == s["eos"]
        x = torch.where(over, torch.where(eos, s["scores"].double()[..., None], -math.inf), x)
    best, at = x.reshape(g, w * v).sort(dim=1, descending=True, stable=True)
    best, at = best[:, :w], at[:, :w]
    none = best == -math.inf
    lane = torch.arange(g, device=x.device)[:, None] * w + at // v
    parent = torch.where(none, -1, lane).int()
    token = torch.where(none, -1, at % v).int()
    over = token == s["eos"]
    if s["done"] is not None:
        over |= s["done"].reshape(-1)[lane].bool() & ~none
    return best.float(), parent, token, over.to(torch.uint8)


# -------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if not own:
        if op == "attn":
            return _plain_attn(s)
        if op == "rope":
            return _plain_rope(s)
        if op in ("fork", "compact"):
            return _plain_pages(s)
        return _plain_beam(s)
    from nvfp4_weight_streaming_decode_b200 import abi
    if op == "attn":
        return abi.attn_tree(s["cache"], 0, s["q"], s["scale"], row_start=s["start"], mask=s["mask"],
                             max_nodes=s["nodes"], want_lse=True, workspace=s["work"])
    if op == "rope":
        abi.rope_append(s["cache"], 1, s["y"], s["q"].shape[1], s["inv_freq"], s["pos"], pair_axis=s["axis"],
                        style=s["style"], row_start=s["start"], q=s["q"])
        return s["q"], s["k"], s["v"]
    if op == "fork":
        s["cache"].fork(s["parent"])
        s["cache"].reserve(s["want"])
        return s["k"], s["v"], s["table"], s["len"], s["ref"]
    if op == "compact":
        s["cache"].trim(s["back"])
        s["cache"].reserve(s["want"])
        s["cache"].compact(s["count"], s["path"])
        return s["k"], s["v"], s["table"], s["len"], s["ref"]
    return abi.beam_select(s["logits"], s["scores"], vocab=s["vocab"], finished=s["done"], eos=s["eos"],
                           workspace=s["work"])


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "attn":
        lens, counts = _lens(case), _counts(case)
        slots, rows = sum(lens) + sum(counts), sum(counts)
        seen = sum(n * (m + n) for m, n in zip(lens, counts))
        return {"bytes": slots * case["hkv"] * case["d"] * 4 + rows * case["hq"] * (case["d"] * 4 + 4),
                "flops": 4 * seen * case["hq"] * case["d"]}
    if op == "rope":
        rows = case["lanes"] * case["nodes"]
        return {"bytes": rows * (case["hq"] + 2 * case["hkv"]) * case["d"] * 6, "flops": 0}
    if op == "fork":
        n = case["lanes"]
        copies = n * (1 - 1 / n) ** n  # beams that share their parent with an earlier one, on average
        slots = copies * ((case["ctx"] % case["page"]) or 1)
        return {"bytes": 2 * slots * case["layers"] * 2 * case["hkv"] * case["d"] * 2, "flops": 0}
    if op == "compact":
        slots = case["lanes"] * case["nodes"] / 2
        return {"bytes": 2 * slots * case["layers"] * 2 * case["hkv"] * case["d"] * 2, "flops": 0}
    rows = case["groups"] * case["beams"]
    return {"bytes": rows * case["vocab"] * 4, "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits; pages, tables and
    indices are copies or whole numbers and have none, but for what rope writes."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        lens, table, page = s["len"].tolist(), s["table"], s["page"]
        hkv = s["k"].shape[2]
        g = case["hq"] // hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        for b in range(case["lanes"]):
            rows = torch.nonzero(s["lane"] == b).reshape(-1)
            n = rows.numel()
            slots = torch.arange(lens[b] + n, device=DEV)
            pg, off = table[b][slots // page].long(), slots % page
            vis = torch.ones((n, lens[b] + n), dtype=torch.bool, device=DEV)
            for i in range(n):
                word = (1 << (i + 1)) - 1 if s["mask"] is None else int(s["mask"][rows[i]]) % (1 << 64)
                vis[i, lens[b]:] = torch.tensor([(word >> j) & 1 == 1 for j in range(n)], device=DEV)
            for h in range(hkv):
                kk = s["k"][0, pg, h, off].double()
                vv = s["v"][0, pg, h, off].double()
                for c in range(g):
                    sc = s["q"][rows, h * g + c].double() @ kk.T * s["scale"]
                    sc[~vis] = -math.inf
                    z = torch.logsumexp(sc, 1)
                    lse[rows, h * g + c] = z
                    out[rows, h * g + c] = torch.exp(sc - z[:, None]) @ vv
        return out, lse
    if op == "rope":
        rows, hq, d = s["q"].shape
        hkv, rot, page = s["k"].shape[2], s["rot"], s["page"]
        k, v = s["k"].double(), s["v"].double()
        y = s["y"].double().reshape(rows, hq + 2 * hkv, d)
        z = y.clone()
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if s["style"] == 0 else (2 * i, 2 * i + 1)
            th = (s["pos"][int(s["axis"][i])].double() * s["inv_freq"][i])[:, None]
            u, w = y[:, :hq + hkv, a], y[:, :hq + hkv, b]
            z[:, :hq + hkv, a] = u * torch.cos(th) - w * torch.sin(th)
            z[:, :hq + hkv, b] = w * torch.cos(th) + u * torch.sin(th)
        slot = s["len"].long()[s["lane"]] + s["node"]
        pg, off = s["table"][s["lane"], slot // page].long(), slot % page
        k[1, pg, :, off] = z[:, hq:hq + hkv]
        v[1, pg, :, off] = z[:, hq + hkv:]
        return z[:, :hq], k, v
    if op in ("fork", "compact"):
        return None
    g, w = s["scores"].shape
    x = s["logits"][:, :s["vocab"]].double()
    cand = s["scores"].double().reshape(-1, 1) + torch.log_softmax(x, 1)
    if s["done"] is not None:
        rows = torch.nonzero(s["done"].reshape(-1)).reshape(-1)
        cand[rows] = -math.inf
        cand[rows, s["eos"]] = s["scores"].double().reshape(-1)[rows]
    return cand.reshape(g, -1).topk(w, dim=1).values, None, None, None
