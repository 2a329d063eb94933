"""The serving operators around the sparse attention, as cases that can be timed and compared: the paged
key/value cache (written, quantised, read back), attention of new tokens over it, attention over whole packed
prompts, and the verification of drafted tokens.

``run`` computes the plain form (elementary torch operations in 32 bits, 64 at borders), or with ``own`` set the
library's calls, on what ``prepare`` made from the case and the seed.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
EXP_BIAS = 127  # stored exponent byte = e + 127
EXP_MIN, EXP_MAX = -100, 100


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token for each of 64 running sequences, appended to an 8-bit cache
        dict(name="write tokens e4m3", op="write", seqs=64, longest=8192, new=1, heads=4, dim=128, page=64, cache="e4m3", src="bf16"),
        # the keys and values of a batch of prompts, into an 8-bit cache
        dict(name="write prompts e4m3", op="write", seqs=6, longest=8192, new=0, heads=4, dim=128, page=64, cache="e4m3", src="bf16"),
        # the selected cells of a four-token step (512 blocks and the open one), read back for the sparse attention
        dict(name="read selected e4m3", op="read", seqs=4, longest=61789, cells=2051, heads=4, dim=128, page=64, cache="e4m3", out="bf16"),
        # whole sequences read back, as a swap to another cache does
        dict(name="read whole e4m3", op="read", seqs=3, longest=61789, cells=0, heads=4, dim=128, page=64, cache="e4m3", out="bf16"),
        # one sequence's token, a short context of the small shape: the latency of one call
        dict(name="attn 1x1 @2050", op="attn", seqs=1, longest=2050, new=1, q_heads=8, heads=2, dim=128, page=64, cache="bf16"),
        # one long sequence, one token: the split over the context
        dict(name="attn 1x1 @255181", op="attn", seqs=1, longest=255181, new=1, q_heads=32, heads=4, dim=128, page=64, cache="bf16"),
        # a running batch of ragged lengths on the 8-bit cache, a token and three drafts each
        dict(name="attn 48x4 @16384 e4m3", op="attn", seqs=48, longest=16384, new=4, q_heads=32, heads=4, dim=128, page=64, cache="e4m3"),
        # a prefill chunk at depth
        dict(name="attn 1x1024 @61789", op="attn", seqs=1, longest=61789, new=1024, q_heads=32, heads=4, dim=128, page=64, cache="bf16"),
        # one short prompt
        dict(name="prompt 777", op="prompt", lens="777", q_heads=8, heads=2, dim=128),
        # packed prompts of very different lengths, one token among them
        dict(name="prompt packed 16384", op="prompt", lens="8192,1,4501,2050,1607,33", q_heads=32, heads=4, dim=128),
        # one sequence's three drafts
        dict(name="verify 1x3", op="verify", seqs=1, drafts=3, vocab=50257, greedy=False),
        # a batch of drafts from a model with a large vocabulary
        dict(name="verify 64x4", op="verify", seqs=64, drafts=4, vocab=131072, greedy=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "prompt", "verify"])
    heads, page = rng.choice([1, 2, 4]), rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "write":
        seqs = _log(rng, 1, 64)
        new = rng.choice([0, 1, rng.randint(2, 9)])
        return dict(op=op, seqs=seqs, longest=_log(rng, 16, 40000 // seqs + 16), new=new, heads=heads, dim=128, page=page, cache=cache, src=rng.choice(["bf16", "f32"]))
    if op == "read":
        seqs = _log(rng, 1, 16)
        return dict(op=op, seqs=seqs, longest=_log(rng, 64, 100000 // seqs), cells=rng.choice([0, _log(rng, 16, 2051)]), heads=heads, dim=128, page=page, cache=cache,
                    out=rng.choice(["bf16", "f32"]))
    if op == "attn":
        kind = rng.choice(["token", "drafts", "chunk"])
        group = rng.choice([4, 8])
        if kind == "chunk":
            return dict(op=op, seqs=_log(rng, 1, 4), longest=_log(rng, 1000, 16000), new=_log(rng, 17, 700), q_heads=group * heads, heads=heads, dim=128, page=page, cache=cache)
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, longest=_log(rng, 64, 400000 // seqs), new=1 if kind == "token" else rng.randint(2, 4), q_heads=group * heads, heads=heads, dim=128, page=page, cache=cache)
    if op == "prompt":
        n = rng.randint(1, 6)
        lens = [_log(rng, 1, 12000 // n) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), q_heads=heads * rng.choice([1, 4, 8]), heads=heads, dim=128)
    return dict(op=op, seqs=_log(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 131072), greedy=rng.random() < 0.3)


def _lengths(case):
    """Context lengths of the case's sequences: the longest, then lengths spread evenly below it."""
    n, top = case["seqs"], case["longest"]
    least = min(top, max(1, case.get("new", 1)))
    return [top] + [least + int((top - least) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, n)]


def _news(case):
    """New tokens of each sequence: the same number for all, or whole sequences where it is 0."""
    return [case["new"] or n for n in _lengths(case)]


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


def _encode(x):
    """e4m3 codes of the rows' values and one exponent for each: the least e with max|x| <= 448 * 2^e."""
    x = x.float()
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(EXP_MIN, EXP_MAX)
    e = torch.where(top == 0, EXP_MIN, e)
    y = (x * _two_to(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    y = torch.where(fine, y, math.nan)
    return y.to(torch.float8_e4m3fn), (e + EXP_BIAS).to(torch.uint8)


def _decode(codes, exps):
    return codes.float() * _two_to(exps.int() - EXP_BIAS)[..., None]


def _pool(case, g, pages):
    """A pool of pages with keys and values of normalised layers: unit rows with a few large channels."""
    rows, h, d = pages * case["page"], case["heads"], case["dim"]
    wide = 1.0 + 3.0 * (torch.rand(h, d, device=DEV, generator=g) < 0.03)
    k = _normal(g, rows, h, d, dtype=torch.float32) * wide
    v = _normal(g, rows, h, d, dtype=torch.float32)
    if case["cache"] == "e4m3":
        (k, ke), (v, ve) = _encode(k), _encode(v)
        return dict(K=k, V=v, K_exp=ke, V_exp=ve)
    return dict(K=k.bfloat16(), V=v.bfloat16(), K_exp=None, V_exp=None)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "verify":
        n, d, v = case["seqs"], case["drafts"], case["vocab"]
        logits = 3.0 * torch.randn(n, d + 1, v, device=DEV, generator=g)
        s["target"] = torch.softmax(logits, -1)
        guess = logits[:, :d] + 0.7 * torch.randn(n, d, v, device=DEV, generator=g)
        del logits
        if case["greedy"]:
            s["draft"], s["tokens"] = None, guess.argmax(-1).int()
        else:
            s["draft"] = torch.softmax(guess, -1)
            noise = -torch.log(-torch.log(torch.rand(n, d, v, device=DEV, generator=g).clamp(1e-9, 1 - 1e-7)))
            s["tokens"] = (guess + noise).argmax(-1).int()
        s["u"] = torch.rand(n, d + 1, device=DEV, generator=g)
        s["n_draft"] = _i32([d - (i % 3 == 2) for i in range(n)])  # some sequences drafted one token fewer
        s["out"], s["accepted"] = torch.zeros(n, d + 1, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    elif op == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        s["cu"], n, d = _i32(_starts(lens)), sum(lens), case["dim"]
        s["q"] = _normal(g, n, case["q_heads"], d)
        s["k"], s["v"] = _normal(g, n, case["heads"], d), _normal(g, n, case["heads"], d)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(n, case["q_heads"], device=DEV)
    else:
        lens = _lengths(case)
        s["table"], pages = _pages(case, g)
        s["kv_len"] = _i32(lens)
        s["longest"] = max(lens)
        s |= _pool(case, g, pages)
        if op == "write":
            s["cu"] = _i32(_starts(_news(case)))
            n, t = sum(_news(case)), torch.bfloat16 if case["src"] == "bf16" else torch.float32
            s["k"], s["v"] = (_normal(g, n, case["heads"], case["dim"], dtype=t) for _ in range(2))
        elif op == "read":
            many = case["cells"] or s["longest"]
            s["n_cells"] = _i32([min(many, n) for n in lens])
            s["max_cells"] = many
            s["pos"] = None
            if case["cells"]:  # ascending cells, as a selection of blocks gives them
                s["pos"] = torch.full((len(lens), many), -1, dtype=torch.int32, device=DEV)
                for i, n in enumerate(lens):
                    c = min(many, n)
                    s["pos"][i, :c] = torch.randperm(n, device=DEV, generator=g)[:c].sort().values.int()
            t = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["K_out"], s["V_out"] = (torch.zeros(len(lens), many, case["heads"], case["dim"], dtype=t, device=DEV) for _ in range(2))
        else:
            news = _news(case)
            s["cu"], s["max_q"] = _i32(_starts(news)), max(news)
            s["q"] = _normal(g, sum(news), case["q_heads"], case["dim"])
            s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(sum(news), case["q_heads"], device=DEV)
    if own:  # the handle and the workspaces that a user's program keeps
        import gather_qsa_pool_gb300 as qsa

        s["qsa"] = qsa
        if op in ("write", "read", "attn"):
            s["cache"] = qsa.PagedCache(s["K"], s["V"], case["page"], K_exp=s["K_exp"], V_exp=s["V_exp"])
        size = 0
        if op == "attn":
            size = qsa.paged_attn_workspace_size(s["q"].shape[0], case["seqs"], s["max_q"], case["q_heads"], case["heads"], case["dim"])
        elif op == "prompt":
            size = qsa.prompt_attn_workspace_size(s["q"].shape[0], s["cu"].numel() - 1, case["q_heads"], case["heads"], case["dim"])
        s["workspace"] = torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ passes

def run(s):
    return _OWN[s["case"]["op"]](s) if own else _PLAIN[s["case"]["op"]](s)


def _cache_of(s):
    return [s[x] for x in ("K", "V", "K_exp", "V_exp") if s[x] is not None]


def _own_write(s):
    s["qsa"].paged_write(s["cache"], s["table"], s["cu"], s["kv_len"], s["k"], s["v"])
    return _cache_of(s)


def _own_read(s):
    s["qsa"].paged_read(s["cache"], s["table"], s["kv_len"], s["n_cells"], s["max_cells"], s["K_out"], s["V_out"], pos=s["pos"])
    return s["K_out"], s["V_out"]


def _own_attn(s):
    s["qsa"].paged_attn(s["cache"], s["table"], s["cu"], s["kv_len"], s["q"], s["out"], s["case"]["dim"] ** -0.5, s["max_q"], lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _own_prompt(s):
    s["qsa"].prompt_attn(s["q"], s["k"], s["v"], s["cu"], s["out"], s["case"]["dim"] ** -0.5, lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _own_verify(s):
    s["qsa"].draft_verify(s["target"], s["draft"], s["tokens"], s["u"], s["out"], s["accepted"], n_draft=s["n_draft"])
    return s["out"], s["accepted"]


_OWN = dict(write=_own_write, read=_own_read, attn=_own_attn, prompt=_own_prompt, verify=_own_verify)


def _owners(cu, n):
    """The sequence of each packed token, and its place in it."""
    at = torch.arange(n, device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), at.int(), right=True)
    return seq, at - cu[seq]


def _rows(s, seq, pos):
    """Pool rows of the positions."""
    page = s["case"]["page"]
    return s["table"][seq, pos // page].long() * page + pos % page


def _plain_write(s):
    seq, at = _owners(s["cu"], s["k"].shape[0])
    fresh = (s["cu"][1:] - s["cu"][:-1])[seq]
    rows = _rows(s, seq, s["kv_len"][seq] - fresh + at)
    if s["case"]["cache"] == "bf16":
        s["K"][rows], s["V"][rows] = s["k"].bfloat16(), s["v"].bfloat16()
        return _cache_of(s)
    (k, ke), (v, ve) = _encode(s["k"]), _encode(s["v"])
    s["K"].view(torch.uint8)[rows], s["V"].view(torch.uint8)[rows] = k.view(torch.uint8), v.view(torch.uint8)
    s["K_exp"][rows], s["V_exp"][rows] = ke, ve
    return _cache_of(s)


def _values(s, rows):
    """Keys and values of pool rows, in 32 bits."""
    if s["case"]["cache"] == "bf16":
        return s["K"][rows].float(), s["V"][rows].float()
    k, v = s["K"].view(torch.uint8)[rows].view(torch.float8_e4m3fn), s["V"].view(torch.uint8)[rows].view(torch.float8_e4m3fn)
    return _decode(k, s["K_exp"][rows]), _decode(v, s["V_exp"][rows])


def _plain_read(s):
    n, many = s["K_out"].shape[:2]
    seq = torch.arange(n, device=DEV)[:, None].expand(n, many)
    cell = torch.arange(many, device=DEV)[None].expand(n, many)
    there = cell < s["n_cells"][:, None]
    pos = torch.where(there, cell if s["pos"] is None else s["pos"], 0)
    k, v = _values(s, _rows(s, seq, pos))
    there = there[:, :, None, None]
    s["K_out"].copy_(torch.where(there, k, s["K_out"]))
    s["V_out"].copy_(torch.where(there, v, s["V_out"]))
    return s["K_out"], s["V_out"]


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


def _plain_prompt(s):
    c = s["case"]
    n, h, d, group = s["q"].shape[0], c["heads"], c["dim"], c["q_heads"] // c["heads"]
    q = s["q"].float().view(n, h, group, d).permute(1, 2, 0, 3)
    k, v = s["k"].float().permute(1, 0, 2)[:, None], s["v"].float().permute(1, 0, 2)[:, None]
    seq, place = _owners(s["cu"], n)
    seen = (seq[:, None] == seq[None]) & (place[:, None] >= place[None])
    out, lse = _softmax_product((q @ k.transpose(-1, -2)).mul_(d ** -0.5), seen, v)
    s["out"].copy_(out.permute(2, 0, 1, 3).reshape(n, h * group, d))
    s["lse"].copy_(lse.permute(2, 0, 1).reshape(n, h * group))
    return s["out"], s["lse"]


def _plain_verify(s):
    d, v = s["case"]["drafts"], s["case"]["vocab"]
    n = s["tokens"].shape[0]
    token = s["tokens"].long()[..., None]
    here = torch.arange(d + 1, device=DEV)[None]
    p = s["target"][:, :d].gather(-1, token).squeeze(-1).double()
    q = torch.ones_like(p) if s["draft"] is None else s["draft"].gather(-1, token).squeeze(-1).double()
    take = (s["u"][:, :d].double() * q < p) & (here[:, :d] < s["n_draft"][:, None])
    count = take.int().cumprod(-1).sum(-1)
    line = torch.arange(n, device=DEV)
    weights = s["target"][line, count].double()
    refused = (count < s["n_draft"])[:, None]
    at = count.clamp(max=d - 1)
    if s["draft"] is None:
        less = torch.zeros_like(weights).scatter_(1, token[line, at], weights.gather(1, token[line, at]))
    else:
        less = s["draft"][line, at].double()
    rest = (weights - less).clamp(min=0)
    weights = torch.where(refused & (rest.sum(-1, keepdim=True) > 0), rest, weights)
    sums = weights.cumsum(-1)
    last = torch.where(weights > 0, torch.arange(v, device=DEV), 0).amax(-1)
    drawn = (sums <= s["u"][:, d:].double() * sums[:, -1:]).sum(-1)
    drawn = torch.minimum(drawn, last)
    padded = torch.cat([s["tokens"], torch.zeros_like(s["tokens"][:, :1])], 1)
    s["out"].copy_(torch.where(here < count[:, None], padded, torch.where(here == count[:, None], drawn[:, None], -1)))
    s["accepted"].copy_(count)
    return s["out"], s["accepted"]


_PLAIN = dict(write=_plain_write, read=_plain_read, attn=_plain_attn, prompt=_plain_prompt, verify=_plain_verify)


# ------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "verify":
        rows = case["seqs"] * (1 if case["greedy"] else 2)
        return {"bytes": rows * case["vocab"] * 4 + case["seqs"] * case["drafts"] * 20, "flops": 3 * rows * case["vocab"]}
    h, d = case["heads"], case["dim"]
    if op == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        n, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
        return {"bytes": n * d * 2 * (2 * case["q_heads"] + 2 * h) + n * case["q_heads"] * 4, "flops": 4 * d * case["q_heads"] * pairs}
    row = h * d * 2 if case["cache"] == "bf16" else h * (d + 1)  # one of K and V, one token
    lens, news = _lengths(case), _news(case) if op != "read" else []
    if op == "write":
        return {"bytes": 2 * sum(news) * (row + h * d * (2 if case["src"] == "bf16" else 4)), "flops": 4 * sum(news) * h * d}
    if op == "read":
        cells = sum(min(case["cells"] or n, n) for n in lens)
        return {"bytes": 2 * cells * (row + h * d * (2 if case["out"] == "bf16" else 4)) + (4 * cells if case["cells"] else 0), "flops": 2 * cells * h * d}
    pairs = sum(x * n - x * (x - 1) // 2 for x, n in zip(news, lens))
    return {"bytes": 2 * sum(lens) * row + sum(news) * case["q_heads"] * (4 * d + 4), "flops": 4 * d * case["q_heads"] * pairs}


# ------------------------------------------------------------------------------------------ in 64 bits

def _grid(x):
    """Values of the e4m3 grid nearest to x (ties to even), in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_row_code(x):
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where((top <= E4M3_MAX * torch.exp2(e - 1)) & (e > EXP_MIN), e - 1, e)
    return _grid(x * torch.exp2(-e)), e.squeeze(-1).int() + EXP_BIAS


def _exact_places(s):
    """(sequence, first new token, new tokens, length) in plain numbers."""
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    return [(i, cu[i], cu[i + 1] - cu[i], n) for i, n in enumerate(lens)]


def _exact_slots(s, i, positions):
    page = s["case"]["page"]
    return s["table"][i].long()[positions // page] * page + positions % page


def _exact_cache(s, slots, name):
    x = s[name].view(torch.uint8)[slots].view(torch.float8_e4m3fn).double() if s["case"]["cache"] == "e4m3" else s[name][slots].double()
    return x * torch.exp2(s[name + "_exp"][slots].double() - EXP_BIAS)[..., None] if s["case"]["cache"] == "e4m3" else x


def _exact_attend(q, k, v, first):
    """q [m, hq, d] at positions first ... over k, v [n, h, d]: the attention and the logarithm of its sum, in 64 bits."""
    m, hq, d = q.shape
    n, h = k.shape[:2]
    out, lse = torch.empty(m, hq, d, dtype=torch.float64, device=DEV), torch.empty(m, hq, dtype=torch.float64, device=DEV)
    hide = torch.arange(n, device=DEV)[None] > torch.arange(first, first + m, device=DEV)[:, None]
    for j in range(hq):
        logit = torch.einsum("id,jd->ij", q[:, j].double(), k[:, j * h // hq].double()) / math.sqrt(d)
        logit = torch.where(hide, -math.inf, logit)
        lse[:, j] = torch.logsumexp(logit, -1)
        out[:, j] = torch.einsum("ij,jd->id", torch.exp(logit - lse[:, j, None]), v[:, j * h // hq].double())
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None  # whole numbers: equal or not
    if op == "write":
        e4m3 = case["cache"] == "e4m3"
        new = {x: s[x].double() for x in ("K", "V")}
        exps = {x: s[x + "_exp"].int() for x in ("K", "V")} if e4m3 else {}
        for i, at, n, length in _exact_places(s):
            slots = _exact_slots(s, i, torch.arange(length - n, length, device=DEV))
            for x, y in (("K", "k"), ("V", "v")):
                fresh = s[y][at:at + n]
                if e4m3:
                    new[x][slots], exps[x][slots] = _exact_row_code(fresh)
                else:
                    new[x][slots] = fresh.double()
        return [new["K"], new["V"]] + ([None, None] if e4m3 else [])
    if op == "read":
        out = {"K": s["K_out"].double(), "V": s["V_out"].double()}
        for i, n in enumerate(s["n_cells"].tolist()):
            at = torch.arange(n, device=DEV) if s["pos"] is None else s["pos"][i, :n].long()
            slots = _exact_slots(s, i, at)
            for x in out:
                out[x][i, :n] = _exact_cache(s, slots, x)
        return out["K"], out["V"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    if op == "prompt":
        cu = s["cu"].tolist()
        for a, b in zip(cu, cu[1:]):
            out[a:b], lse[a:b] = _exact_attend(s["q"][a:b], s["k"][a:b], s["v"][a:b], 0)
        return out, lse
    for i, at, n, length in _exact_places(s):
        slots = _exact_slots(s, i, torch.arange(length, device=DEV))
        out[at:at + n], lse[at:at + n] = _exact_attend(s["q"][at:at + n], _exact_cache(s, slots, "K"), _exact_cache(s, slots, "V"), length - n)
    return out, lse
