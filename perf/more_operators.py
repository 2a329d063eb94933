"""More of the serving operators, as cases that can be timed and compared: new tokens appended to a paged cache with
the position rotation on the way, attention over a paged cache held in 4 bits, and sparse attention over the blocks
that each token's scores selected, read in place from a paged cache.

``run`` computes the plain form (elementary torch operations in 32 bits, 64 for angles), or with ``own`` set the
library's calls, on what ``prepare`` made from the case and the seed.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 4               # cells of a selected block
GROUP = 16              # values that share a scale in a 4-bit cache
E4M3_MAX, E2M1_MAX = 448.0, 6.0
EXP_BIAS = 127          # stored exponent byte = e + 127
EXP_MIN, EXP_MAX = -100, 100
BASE = 10000.0          # of the rotation's frequencies


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token for each of 64 running sequences: queries and keys rotated, the cache written
        dict(name="append tokens bf16", op="append", seqs=64, longest=8192, new=1, q_heads=32, heads=4, dim=128, rot=128, page=64, cache="bf16", src="bf16"),
        # the keys and values of a batch of prompts, into an 8-bit cache
        dict(name="append prompts e4m3", op="append", seqs=6, longest=8192, new=0, q_heads=32, heads=4, dim=128, rot=128, page=64, cache="e4m3", src="bf16"),
        # the same into a 4-bit cache, and read back as the values that it holds (a swap to another cache)
        dict(name="append prompts e2m1", op="append", seqs=6, longest=8192, new=0, q_heads=32, heads=4, dim=128, rot=128, page=64, cache="e2m1", src="bf16"),
        # one sequence's token, a short context of the small shape: the latency of one call
        dict(name="attn4 1x1 @2050", op="attn", seqs=1, longest=2050, new=1, q_heads=8, heads=2, dim=128, page=64, cache="e2m1"),
        # one long sequence, one token: the split over the context
        dict(name="attn4 1x1 @255181", op="attn", seqs=1, longest=255181, new=1, q_heads=32, heads=4, dim=128, page=64, cache="e2m1"),
        # a running batch of ragged lengths, a token each
        dict(name="attn4 64x1 @16384", op="attn", seqs=64, longest=16384, new=1, q_heads=32, heads=4, dim=128, page=64, cache="e2m1"),
        # the same with three drafts beside each token
        dict(name="attn4 48x4 @16384", op="attn", seqs=48, longest=16384, new=4, q_heads=32, heads=4, dim=128, page=64, cache="e2m1"),
        # a prefill chunk at depth
        dict(name="attn4 1x1024 @61789", op="attn", seqs=1, longest=61789, new=1024, q_heads=32, heads=4, dim=128, page=64, cache="e2m1"),
        # one sequence's token over its 512 selected blocks and the open one
        dict(name="sparse 1x1 bf16", op="sparse", seqs=1, longest=61789, new=1, blocks=512, q_heads=32, heads=4, dim=128, page=64, cache="bf16"),
        # a token for each of 64 long sequences on the 4-bit cache
        dict(name="sparse 64x1 e2m1", op="sparse", seqs=64, longest=61789, new=1, blocks=512, q_heads=32, heads=4, dim=128, page=64, cache="e2m1"),
        # a token and three drafts, each with its own selection, on the 8-bit cache
        dict(name="sparse 32x4 e4m3", op="sparse", seqs=32, longest=30000, new=4, blocks=512, q_heads=32, heads=4, dim=128, page=64, cache="e4m3"),
        # a prefill chunk at depth, a selection for every query
        dict(name="sparse 1x1024 bf16", op="sparse", seqs=1, longest=61789, new=1024, blocks=512, q_heads=32, heads=4, dim=128, page=64, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sparse", "sparse"])
    heads, page = rng.choice([1, 2, 4]), rng.choice([16, 32, 64, 128])
    if op == "append":
        seqs, dim = _log(rng, 1, 64), rng.choice([64, 128])
        new = rng.choice([0, 1, rng.randint(2, 9)])
        return dict(op=op, seqs=seqs, longest=_log(rng, 16, 40000 // seqs + 16), new=new, q_heads=heads * rng.choice([1, 4, 8]), heads=heads, dim=dim, rot=dim // rng.choice([1, 1, 2]), page=page,
                    cache=rng.choice(["bf16", "e4m3", "e2m1"]), src=rng.choice(["bf16", "f32"]))
    group = rng.choice([4, 8])
    if op == "attn":
        kind = rng.choice(["token", "drafts", "chunk"])
        if kind == "chunk":
            return dict(op=op, seqs=_log(rng, 1, 4), longest=_log(rng, 1000, 16000), new=_log(rng, 17, 700), q_heads=group * heads, heads=heads, dim=128, page=page, cache="e2m1")
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, longest=_log(rng, 64, 400000 // seqs), new=1 if kind == "token" else rng.randint(2, 4), q_heads=group * heads, heads=heads, dim=128, page=page, cache="e2m1")
    seqs = _log(rng, 1, 64)
    new = rng.choice([1, 1, rng.randint(2, 4), _log(rng, 5, 800 // seqs + 5)])
    return dict(op=op, seqs=seqs, longest=_log(rng, 64, 400000 // seqs), new=new, blocks=_log(rng, 16, 512), q_heads=group * heads, heads=heads, dim=128, page=page,
                cache=rng.choice(["bf16", "e4m3", "e2m1"]))


def _lengths(case):
    """Context lengths of the case's sequences: the longest, then lengths spread evenly below it."""
    n, top = case["seqs"], case["longest"]
    least = min(top, max(1, case["new"]))
    return [top] + [least + int((top - least) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _news(case):
    """New tokens of each sequence: the same number for all (the whole of a shorter one), or whole sequences where it is 0."""
    return [min(case["new"] or n, n) for n in _lengths(case)]


# ------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _pages(case, g):
    """The page table of the sequences, in an order that allocation and release have mixed, and the pool's pages."""
    counts = [-(-n // case["page"]) for n in _lengths(case)]
    total = sum(counts) + 3
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    return table, total


def _two_to(e):
    """2^e in 32 bits, |e| <= 126, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _tops(x, most, bits):
    """The rows' largest finite magnitudes, and for each the least e with that <= most * 2^e (most = m * 2^bits, m in [0.5, 1))."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(m > most / 2.0 ** bits, e - bits + 1, e - bits).clamp(EXP_MIN, EXP_MAX)
    return torch.where(top == 0, EXP_MIN, e)


def _encode8(x):
    """e4m3 codes of the rows' values, and one exponent for each: the least e with max|x| <= 448 * 2^e."""
    x = x.float()
    e = _tops(x, E4M3_MAX, 9)
    y = (x * _two_to(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return torch.where(torch.isfinite(x), y, math.nan).to(torch.float8_e4m3fn), (e + EXP_BIAS).to(torch.uint8)


def _encode4(x):
    """e2m1 codes (two a byte, the even one below), an e4m3 scale for each 16 values, and one exponent for each row: the
    least e with max|x| <= 6 * 448 * 2^e; a scale is the e4m3 value nearest to a sixth of its values' largest over 2^e."""
    x = x.float()
    e = _tops(x, E4M3_MAX * E2M1_MAX, 12)
    y = (x * _two_to(-e)[..., None]).unflatten(-1, (-1, GROUP))
    s = (y.abs().amax(-1) / E2M1_MAX).clamp(max=E4M3_MAX)
    s = torch.where(torch.isfinite(y).all(-1), s, math.nan).to(torch.float8_e4m3fn)
    r = torch.where(s.float()[..., None] > 0, y.abs() / s.float()[..., None], 0.0)
    code = ((r > 0.25).byte() + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0)).byte()
    code = (code | (torch.signbit(y).byte() << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s, (e + EXP_BIAS).to(torch.uint8)


def _decode4(codes, scales, exps):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    m, x = c & 1, (c >> 1) & 3
    v = torch.where(x > 0, (1.0 + 0.5 * m) * torch.exp2(x.float() - 1.0), 0.5 * m) * (1 - 2 * (c >> 3))
    v = v.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]
    return v.flatten(-2) * _two_to(exps.int() - EXP_BIAS)[..., None]


def _scale_places(s, rows):
    """Places of the rows' scales, which lie page by page, head by head: [rows, heads] into [pages * heads * page]."""
    page, h = s["case"]["page"], s["case"]["heads"]
    return ((rows // page)[..., None] * h + torch.arange(h, device=DEV)) * page + (rows % page)[..., None]


def _pool(case, g, pages):
    """A pool of pages with keys and values of normalised layers: unit rows with a few large channels."""
    page, h, d = case["page"], case["heads"], case["dim"]
    rows = pages * page
    wide = 1.0 + 3.0 * (torch.rand(h, d, device=DEV, generator=g) < 0.03)
    k = _normal(g, rows, h, d) * wide.bfloat16()
    v = _normal(g, rows, h, d)
    p = dict(K=k, V=v, K_exp=None, V_exp=None, K_scale=None, V_scale=None)
    for x, y in (("K", k), ("V", v)):
        if case["cache"] == "e4m3":
            p[x], p[x + "_exp"] = _encode8(y)
        elif case["cache"] == "e2m1":
            p[x], scale, p[x + "_exp"] = _encode4(y)
            p[x + "_scale"] = scale.view(pages, page, h, d // GROUP).transpose(1, 2).contiguous()
    return p


def _selection(case, g, seq, pos):
    """Each token's best blocks of those complete at its position, ascending: scores that the tokens of a sequence share in part."""
    k = case["blocks"]
    full = (pos + 1) // BLOCK
    width = max(k, (case["longest"] + BLOCK) // BLOCK)
    common = torch.randn(case["seqs"], width, device=DEV, generator=g)
    score = torch.randn(len(pos), width, device=DEV, generator=g) + 1.5 * common[seq]
    at = torch.arange(width, device=DEV)[None]
    score.masked_fill_(at >= full[:, None], -math.inf)
    best = score.topk(k, -1).indices
    best = torch.where(best < full[:, None], best, 1 << 30).sort(-1).values
    return torch.where(best < 1 << 30, best, -1).int(), full.clamp(max=k).int()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    lens, news = _lengths(case), _news(case)
    s = {"case": case, "kv_len": _i32(lens), "cu": _i32(_starts(news)), "longest": max(lens), "max_q": max(news)}
    s["table"], pages = _pages(case, g)
    s |= _pool(case, g, pages)
    n, h, d = sum(news), case["heads"], case["dim"]
    seq, place = _owners(s["cu"], n)
    s["pos"] = s["kv_len"][seq] - _i32(news)[seq] + place.int()
    if case["op"] == "append":
        t = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        wide = 1.0 + 3.0 * (torch.rand(h, d, device=DEV, generator=g) < 0.03)
        s["k"] = (_normal(g, n, h, d, dtype=torch.float32) * wide).to(t)
        s["v"], s["q"] = _normal(g, n, h, d, dtype=t), _normal(g, n, case["q_heads"], d, dtype=t)
        s["q_out"] = torch.zeros_like(s["q"])
        if case["cache"] == "e2m1":  # the new cells of each sequence, read back
            most = max(news)
            cell = _i32(lens)[:, None] - _i32(news)[:, None] + torch.arange(most, device=DEV, dtype=torch.int32)[None]
            s["cells"], s["n_cells"] = cell.contiguous(), _i32(news)
            s["K_out"], s["V_out"] = (torch.zeros(len(lens), most, h, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    else:
        s["q"] = _normal(g, n, case["q_heads"], d)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(n, case["q_heads"], device=DEV)
        if case["op"] == "sparse":
            s["blocks"], s["counts"] = _selection(case, g, seq, s["pos"].long())
    if own:  # the handle and the workspaces that a user's program keeps
        import gather_qsa_pool_gb300 as qsa

        s["qsa"] = qsa
        s["cache"] = qsa.PagedCache(s["K"], s["V"], case["page"], K_exp=s["K_exp"], V_exp=s["V_exp"], K_scale=s["K_scale"], V_scale=s["V_scale"])
        if case["op"] == "attn":
            size = qsa.paged_attn_workspace_size(n, case["seqs"], s["max_q"], case["q_heads"], h, d)
            s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ passes

def run(s):
    return _OWN[s["case"]["op"]](s) if own else _PLAIN[s["case"]["op"]](s)


def _appended(s):
    if s["case"]["cache"] == "e2m1":
        return [s["q_out"], s["K_out"], s["V_out"]]
    return [s["q_out"]] + [s[x] for x in ("K", "V", "K_exp", "V_exp") if s[x] is not None]


def _own_append(s):
    qsa, c = s["qsa"], s["case"]
    qsa.paged_append(s["cache"], s["table"], s["cu"], s["kv_len"], s["k"], s["v"], BASE, c["rot"], q=s["q"], q_out=s["q_out"])
    if c["cache"] == "e2m1":
        qsa.paged_read(s["cache"], s["table"], s["kv_len"], s["n_cells"], s["max_q"], s["K_out"], s["V_out"], pos=s["cells"])
    return _appended(s)


def _own_attn(s):
    s["qsa"].paged_attn(s["cache"], s["table"], s["cu"], s["kv_len"], s["q"], s["out"], s["case"]["dim"] ** -0.5, s["max_q"], lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _own_sparse(s):
    s["qsa"].paged_sparse_attn(s["cache"], s["table"], s["cu"], s["kv_len"], s["blocks"], s["counts"], s["q"], s["out"], s["case"]["dim"] ** -0.5, lse=s["lse"])
    return s["out"], s["lse"]


_OWN = dict(append=_own_append, attn=_own_attn, sparse=_own_sparse)


def _owners(cu, n):
    """The sequence of each packed token, and its place in it."""
    at = torch.arange(n, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), at.int(), right=True)
    return seq, at - cu[seq]


def _rows(s, seq, pos):
    """Pool rows of the positions."""
    page = s["case"]["page"]
    return s["table"][seq, pos // page].long() * page + pos % page


def _rotated(x, pos, rot):
    """The first `rot` values of each head: values i and i + rot / 2 turned by pos * BASE^(-2 i / rot)."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    angle = pos.double()[:, None] * BASE ** (-2.0 * i / rot)[None]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b, rest = x.float().split([rot // 2, rot // 2, x.shape[-1] - rot], -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_append(s):
    c = s["case"]
    seq, at = _owners(s["cu"], s["k"].shape[0])
    pos = s["kv_len"][seq] - (s["cu"][1:] - s["cu"][:-1])[seq] + at
    rows = _rows(s, seq, pos)
    s["q_out"].copy_(_rotated(s["q"], pos, c["rot"]))
    for x, y in (("K", _rotated(s["k"], pos, c["rot"])), ("V", s["v"])):
        if c["cache"] == "bf16":
            s[x][rows] = y.bfloat16()
        elif c["cache"] == "e4m3":
            code, s[x + "_exp"][rows] = _encode8(y)
            s[x].view(torch.uint8)[rows] = code.view(torch.uint8)
        else:
            s[x][rows], scale, s[x + "_exp"][rows] = _encode4(y)
            s[x + "_scale"].view(torch.uint8).view(-1, c["dim"] // GROUP)[_scale_places(s, rows)] = scale.view(torch.uint8)
    if c["cache"] == "e2m1":
        cell = s["cells"].long()
        there = cell < s["kv_len"][:, None]
        line = torch.arange(c["seqs"], device=DEV)[:, None].expand_as(cell)
        k, v = _values(s, _rows(s, line, torch.where(there, cell, 0)))
        s["K_out"].copy_(torch.where(there[..., None, None], k, s["K_out"]))
        s["V_out"].copy_(torch.where(there[..., None, None], v, s["V_out"]))
    return _appended(s)


def _values(s, rows):
    """Keys and values of pool rows, in 32 bits."""
    if s["case"]["cache"] == "bf16":
        return s["K"][rows].float(), s["V"][rows].float()
    if s["case"]["cache"] == "e4m3":
        return tuple(s[x].view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * _two_to(s[x + "_exp"][rows].int() - EXP_BIAS)[..., None] for x in ("K", "V"))
    at = _scale_places(s, rows)
    scale = lambda x: s[x + "_scale"].view(torch.uint8).view(-1, s["case"]["dim"] // GROUP)[at].view(torch.float8_e4m3fn)  # noqa: E731
    return tuple(_decode4(s[x][rows], scale(x), s[x + "_exp"][rows]) for x in ("K", "V"))


def _softmax_product(logits, seen, v):
    """softmax over the seen keys times v, and the logarithm of its sum."""
    logits.masked_fill_(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    weights = logits.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    return (weights @ v).div_(total), (top + total.log()).squeeze(-1)


def _plain_attn(s):
    c, long = s["case"], s["longest"]
    b, h, d, new, group = c["seqs"], c["heads"], c["dim"], s["max_q"], c["q_heads"] // c["heads"]
    cell = torch.arange(long, device=DEV)
    at = torch.minimum(cell[None], s["kv_len"][:, None] - 1)
    k, v = _values(s, _rows(s, torch.arange(b, device=DEV)[:, None].expand(b, long), at))
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)  # [b, h, long, d]
    seq, place = _owners(s["cu"], s["q"].shape[0])
    q = torch.zeros(b, new, h * group, d, device=DEV)
    q[seq, place] = s["q"].float()
    q = q.view(b, new, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * new, d)
    logits = (q @ k.transpose(-1, -2)).mul_(d ** -0.5)
    fresh = s["cu"][1:] - s["cu"][:-1]
    last = s["kv_len"][:, None] - fresh[:, None] + torch.arange(new, device=DEV)[None]  # position of each query
    seen = cell[None, None] <= last[:, :, None]
    seen = seen[:, None, None].expand(b, 1, group, new, long).reshape(b, 1, group * new, long)
    out, lse = _softmax_product(logits, seen, v)
    out = out.view(b, h, group, new, d).permute(0, 3, 1, 2, 4).reshape(b, new, h * group, d)
    lse = lse.view(b, h, group, new).permute(0, 3, 1, 2).reshape(b, new, h * group)
    s["out"].copy_(out[seq, place])
    s["lse"].copy_(lse[seq, place])
    return s["out"], s["lse"]


def _plain_sparse(s):
    c = s["case"]
    n, h, d, group = s["q"].shape[0], c["heads"], c["dim"], c["q_heads"] // c["heads"]
    seq, place = _owners(s["cu"], n)
    pos = s["kv_len"][seq] - (s["cu"][1:] - s["cu"][:-1])[seq] + place
    four = torch.arange(BLOCK, device=DEV)
    listed_ = torch.arange(c["blocks"], device=DEV)[None] < s["counts"][:, None]
    cells = torch.cat([(s["blocks"].long()[..., None] * BLOCK + four).flatten(1), ((pos + 1) // BLOCK * BLOCK)[:, None] + four], 1)
    seen = torch.cat([listed_[..., None].expand(n, c["blocks"], BLOCK).flatten(1), cells[:, -BLOCK:] <= pos[:, None]], 1)
    cells = torch.where(seen, cells, 0)
    k, v = _values(s, _rows(s, seq[:, None].expand_as(cells), cells))  # [n, cells, h, d]
    q = s["q"].float().view(n, h, group, d)
    out, lse = _softmax_product((q @ k.permute(0, 2, 3, 1)).mul_(d ** -0.5), seen[:, None, None], v.permute(0, 2, 1, 3))
    s["out"].copy_(out.reshape(n, h * group, d))
    s["lse"].copy_(lse.reshape(n, h * group))
    return s["out"], s["lse"]


_PLAIN = dict(append=_plain_append, attn=_plain_attn, sparse=_plain_sparse)


# ------------------------------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    """One token's keys or values in the cache."""
    h, d = case["heads"], case["dim"]
    return h * {"bf16": 2 * d, "e4m3": d + 1, "e2m1": d // 2 + d // GROUP + 1}[case["cache"]]


def work(case):
    h, hq, d, row = case["heads"], case["q_heads"], case["dim"], _row_bytes(case)
    lens, news = _lengths(case), _news(case)
    n = sum(news)
    if case["op"] == "append":
        size = 2 if case["src"] == "bf16" else 4
        back = n * 2 * (row + 2 * h * d) if case["cache"] == "e2m1" else 0
        return {"bytes": n * (2 * row + 2 * h * d * size + 2 * hq * d * size) + back, "flops": n * (3 * (hq + h) * case["rot"] + 4 * h * d)}
    if case["op"] == "attn":
        pairs = sum(x * m - x * (x - 1) // 2 for x, m in zip(news, lens))
        return {"bytes": 2 * sum(lens) * row + n * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    pairs = cells = 0
    for x, m in zip(news, lens):
        seen = [min(p + 1, BLOCK * case["blocks"] + (p + 1) % BLOCK) for p in range(m - x, m)]
        pairs += sum(seen)
        cells += min(m, sum(seen))  # (tokens that share cells need them once)
    return {"bytes": 2 * cells * row + n * (4 * case["blocks"] + hq * (4 * d + 4)), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------------ in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _grid8(x):
    """Values of the e4m3 grid nearest to x (ties to even), in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_exponent(top, most):
    e = torch.ceil(torch.log2(top / most)).clamp(EXP_MIN, EXP_MAX)
    e = torch.where(top > most * torch.exp2(e), e + 1, e)
    return torch.where((top <= most * torch.exp2(e - 1)) & (e > EXP_MIN), e - 1, e)


def _exact_stored(x, cache):
    """What a row of 64-bit values is in the cache: values, and the exponent byte (8 bits: values are the codes alone)."""
    if cache == "bf16":
        return x, None
    top = x.abs().amax(-1, keepdim=True)
    if cache == "e4m3":
        e = _exact_exponent(top, E4M3_MAX)
        return _grid8(x * torch.exp2(-e)), e.squeeze(-1).int() + EXP_BIAS
    e = _exact_exponent(top, E4M3_MAX * E2M1_MAX)
    y = (x * torch.exp2(-e)).unflatten(-1, (-1, GROUP))
    s = _grid8(y.abs().amax(-1, keepdim=True) / E2M1_MAX)
    a = torch.where(s > 0, y.abs() / s, 0.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=E2M1_MAX)
    return (a * torch.sign(y) * s).flatten(-2) * torch.exp2(e), None


def _exact_turn(x, pos, rot):
    """As complex numbers times e^(i angle)."""
    i = torch.arange(0, rot, 2, device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones_like(i).expand(len(pos), -1), pos.double()[:, None] * torch.exp(-math.log(BASE) * i / rot))
    y = x.double().clone()
    z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn[:, None]
    y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_slots(s, i, positions):
    page = s["case"]["page"]
    return s["table"][i].long()[positions // page] * page + positions % page


def _exact_cells(s, slots, name):
    """Values of pool rows in 64 bits, [n, heads, dim]."""
    c = s["case"]
    if c["cache"] == "bf16":
        return s[name][slots].double()
    scale = torch.exp2(s[name + "_exp"][slots].double() - EXP_BIAS)[..., None]
    if c["cache"] == "e4m3":
        return s[name].view(torch.uint8)[slots].view(torch.float8_e4m3fn).double() * scale
    byte = s[name][slots].long()
    code = torch.stack((byte % 16, byte // 16), -1).reshape(len(slots), c["heads"], -1)
    grid = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=DEV)
    by16 = s[name + "_scale"].view(torch.uint8)[slots // c["page"], :, slots % c["page"]].view(torch.float8_e4m3fn).double()
    return grid[code] * by16.repeat_interleave(GROUP, -1) * scale


def _exact_attend(q, k, v, hide):
    """q [m, hq, d] over k, v [n, h, d], hide [m, n]: the attention and the logarithm of its sum, in 64 bits."""
    m, hq, d = q.shape
    h = k.shape[1]
    out, lse = torch.empty(m, hq, d, dtype=torch.float64, device=DEV), torch.empty(m, hq, dtype=torch.float64, device=DEV)
    for j in range(hq):
        logit = torch.einsum("id,jd->ij", q[:, j].double(), k[:, j * h // hq]) / math.sqrt(d)
        logit = torch.where(hide, -math.inf, logit)
        lse[:, j] = torch.logsumexp(logit, -1)
        out[:, j] = torch.einsum("ij,jd->id", torch.exp(logit - lse[:, j, None]), v[:, j * h // hq])
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    places = [(i, cu[i], cu[i + 1] - cu[i], n) for i, n in enumerate(lens)]  # sequence, first new token, new tokens, length
    if case["op"] == "append":
        turned = {"K": _exact_turn(s["k"], s["pos"], case["rot"]), "V": s["v"].double()}
        q = _exact_turn(s["q"], s["pos"], case["rot"])
        got, exps = {}, {}
        for x, y in turned.items():
            value, byte = _exact_stored(y, case["cache"])
            if case["cache"] == "e2m1":
                got[x] = s[x + "_out"].double()
                for i, at, n, length in places:
                    got[x][i, :n] = value[at:at + n]
                continue
            got[x] = s[x].double()
            for i, at, n, length in places:
                got[x][_exact_slots(s, i, torch.arange(length - n, length, device=DEV))] = value[at:at + n]
            if byte is not None:
                exps[x] = None
        return [q, got["K"], got["V"]] + [None] * len(exps)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for i, at, n, length in places:
        if case["op"] == "attn":
            slots = _exact_slots(s, i, torch.arange(length, device=DEV))
            hide = torch.arange(length, device=DEV)[None] > torch.arange(length - n, length, device=DEV)[:, None]
            out[at:at + n], lse[at:at + n] = _exact_attend(s["q"][at:at + n], _exact_cells(s, slots, "K"), _exact_cells(s, slots, "V"), hide)
            continue
        for t in range(at, at + n):
            p = length - n + t - at
            mine = s["blocks"][t, :int(s["counts"][t])].long()
            cell = torch.cat([(mine[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(), torch.arange((p + 1) // BLOCK * BLOCK, p + 1, device=DEV)])
            slots = _exact_slots(s, i, cell)
            k, v = _exact_cells(s, slots, "K"), _exact_cells(s, slots, "V")
            qt = s["q"][t].double().unflatten(0, (case["heads"], -1))  # [h, group, d]
            logit = torch.einsum("hgd,nhd->hgn", qt, k) / math.sqrt(case["dim"])
            whole = torch.logsumexp(logit, -1)
            lse[t] = whole.flatten()
            out[t] = torch.einsum("hgn,nhd->hgd", torch.exp(logit - whole[..., None]), v).flatten(0, 1)
    return out, lse
