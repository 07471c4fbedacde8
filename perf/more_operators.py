"""A step of tree-drafted decoding over a paged key/value cache, and norms of queries and keys with the rotation.

Each case is one call of one operator.  ``own`` false computes it with elementary torch operations in fp32 (angles in
fp64), rounded once; ``own`` true calls the framework.  The operators: norms of queries and keys per head with the
rotary positions in the same pass, forward and backward (``norm``, ``grad``), and on the way to a paged cache
(``append``); page tables, slots, positions and ancestor masks of a step from the requests' lengths (``assign``); the
cache rows of an accepted path moved next to each other (``accept``); attention of a tree of drafted tokens over the
cache (``tree``).  Head counts, lengths and page sizes are generic ones around this repository's own workloads.

Layouts: rows of heads [tokens, heads, dim] (possibly slices of a wider row, as a fused projection leaves them); the
cache [pages, kv_heads, page_size, dim] for K and for V, bf16 or E4M3 with an fp32 scale per kv head; a page table
[seqs, max_pages].  A sequence's n new tokens are its last n keys; token i's parent in the tree is parents[i] < i, -1
for a child of the context's last token, and bit t of a token's mask (int64 words) says that it sees new token t.
"""

import math
import random

import torch

own = False

_THETA = 500000.0
_TRAINED = 8192.0  # the context that the frequencies were trained for, where they are stretched beyond it
_EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _norm(name, op, tokens, heads, kv_heads, dim, rot, interleaved, factor, far, wide, weight):
    return dict(name=name, op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, factor=factor, far=far, wide=wide, weight=weight)


def _append(name, seqs, tokens, heads, kv_heads, dim, rot, interleaved, factor, context, page, cache, weight):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, factor=factor, context=context, page=page, cache=cache, weight=weight)


def _assign(name, seqs, kind, new, context, page, spare):
    return dict(name=name, op="assign", seqs=seqs, kind=kind, new=new, context=context, page=page, spare=spare)


def _accept(name, seqs, new, context, kv_heads, dim, page, cache):
    return dict(name=name, op="accept", seqs=seqs, new=new, context=context, kv_heads=kv_heads, dim=dim, page=page,
                cache=cache)


def _tree(name, seqs, new, context, ragged, heads, kv_heads, dim, page, cache, window=0, softcap=0.0):
    return dict(name=name, op="tree", seqs=seqs, new=new, context=context, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, cache=cache, window=window, softcap=softcap)


def listed():
    return [
        # a long prompt's queries and keys, normalised and rotated out of a fused projection's rows
        _norm("norm_rope_prompt", "norm", 8191, 32, 8, 128, 128, False, 8.0, 131072, True, "bf16"),
        # the way back through it in a training step
        _norm("norm_rope_gradient", "grad", 8191, 32, 8, 128, 64, True, 1.0, 8192, True, "fp32"),
        # one decode step of 16 sequences: latency
        _append("norm_append_step", 16, 16, 16, 8, 128, 128, False, 1.0, 4096, 64, "bf16", "bf16"),
        # a prefill's tokens quantized into small pages
        _append("norm_append_prompt_e4m3", 3, 8191, 32, 8, 128, 128, False, 8.0, 20000, 16, "e4m3", "bf16"),
        # a verify step: trees of up to 31 drafted tokens for 16 requests
        _assign("assign_trees", 16, "tree", 31, 4096, 64, 17),
        # continuous batching: prompt pieces, single tokens, idle and finished requests
        _assign("assign_mixed", 256, "mixed", 1024, 8192, 16, 100),
        # one request's accepted path
        _accept("accept_one", 1, 15, 4096, 8, 128, 64, "bf16"),
        # a large batch's
        _accept("accept_batch_e4m3", 64, 64, 16000, 8, 128, 64, "e4m3"),
        # one sequence's verify block at a short context: latency
        _tree("tree_one", 1, 15, 999, "no", 16, 8, 128, 16, "bf16"),
        # a serving batch's trees over contexts from a few tokens to 16K
        _tree("tree_batch", 32, 32, 16383, "spread", 32, 8, 128, 64, "bf16"),
        # large trees over two very long conversations on a quantized cache
        _tree("tree_long_e4m3", 2, 63, 131008, "no", 64, 8, 128, 128, "e4m3"),
        # a sliding-window layer with wide heads and capped logits
        _tree("tree_window", 4, 21, 8177, "spread", 16, 8, 256, 32, "bf16", 1024, 50.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "grad", "append", "assign", "accept", "tree", "tree", "tree", "tree"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    factor = rng.choice([1.0, 4.0, 8.0])
    interleaved = rng.random() < 0.5
    weight = rng.choice(["bf16", "fp32"])
    if op in ("norm", "grad"):
        dim = rng.choice([dim, dim, 96])
        rot = rng.choice([dim, dim, dim // 2])
        tokens = _log_int(rng, 1, min(32768, (1 << 25) // (kv_heads * (group + 1) * dim)))
        c = _norm("", op, tokens, kv_heads * group, kv_heads, dim, rot, interleaved, factor,
                  _log_int(rng, 64, 1 << 20), rng.random() < 0.5, weight)
    elif op == "append":
        rot = rng.choice([dim, dim, dim // 2])
        tokens = _log_int(rng, 1, min(16384, (1 << 25) // (kv_heads * (group + 2) * dim)))
        c = _append("", rng.randint(1, min(tokens, 64)), tokens, kv_heads * group, kv_heads, dim, rot, interleaved,
                    factor, _log_int(rng, 1, 30000), page, cache, weight)
    elif op == "assign":
        kind = rng.choice(["one", "tree", "mixed"])
        c = _assign("", _log_int(rng, 1, 512), kind, {"one": 1, "tree": _log_int(rng, 2, 200),
                                                      "mixed": _log_int(rng, 2, 2048)}[kind],
                    _log_int(rng, 1, 30000) - 1, page, _log_int(rng, 1, 256) - 1)
    elif op == "accept":
        c = _accept("", _log_int(rng, 1, 64), _log_int(rng, 2, 200), _log_int(rng, 1, 16384) - 1, kv_heads, dim, page,
                    cache)
    else:
        while True:
            seqs, new = _log_int(rng, 1, 64), rng.choice([rng.randint(2, 16), _log_int(rng, 2, 200)])
            context = _log_int(rng, 1, 131072) - 1
            c = _tree("", seqs, new, context, rng.choice(["no", "spread"]), kv_heads * group, kv_heads, dim, page,
                      cache, rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]), rng.choice([0.0, 0.0, 50.0]))
            # the plain form keeps padded fp32 keys and scores
            if (seqs * kv_heads * group * new * (context + new) <= 1 << 30
                    and seqs * kv_heads * dim * (context + new) <= 64 * 16384 * 8 * 128
                    and work(c)["flops"] <= work(listed()[-2])["flops"]):
                break
    del c["name"]
    return c


def _rng(c):
    return random.Random(" ".join(str(c[k]) for k in sorted(c) if k != "name"))


def _parents(rng, n):
    """A drafted tree of n tokens: the likeliest chain first, then side branches off it, each a chain too."""
    main = max(1, min(n, rng.randint(n // 4, n // 2) + rng.randint(0, 2)))
    return [i - 1 if i < main else (rng.randint(-1, main // 2) if i == main or rng.random() < 0.3 else i - 1)
            for i in range(n)]


def _path_to(parents, i):
    """The tokens from the context to token i."""
    up = []
    while i >= 0:
        up.append(i)
        i = parents[i]
    return up[::-1]


def _accepted(rng, parents):
    """A path that a verify step may accept: the likeliest chain for a while, then a side branch, no longer than that
    chain.  So its rows move to places that it does not take any from, and the same call may be made again."""
    main = sum(all(parents[x] == x - 1 for x in range(i + 1)) for i in range(len(parents)))
    path = _path_to(parents, rng.randrange(min(main, len(parents) - 1), len(parents)))
    return path[:max(1, rng.randint(main // 2, main))]


def _trees(c):
    """(new tokens, kv length, parents) of each sequence of a tree or accept case: from the case alone."""
    rng = _rng(c)
    out = []
    for b in range(c["seqs"]):
        n, ctx = c["new"], c["context"]
        if b > 0 and c.get("ragged", "spread") != "no":
            n, ctx = _log_int(rng, 1, n), _log_int(rng, 1, ctx + 1) - 1
        out.append((n, n + ctx, _parents(rng, n)))
    return out


def _counts(c):
    """New tokens of each request of an assign case (-1: finished): from the case alone."""
    rng = _rng(c)
    if c["kind"] == "one":
        return [1] * c["seqs"]
    if c["kind"] == "tree":
        return [c["new"]] + [_log_int(rng, 1, c["new"]) for _ in range(c["seqs"] - 1)]
    return [c["new"]] + [rng.choice([1, 1, 1, 1, 0, -1, _log_int(rng, 1, c["new"]), _log_int(rng, 1, c["new"])])
                         for _ in range(c["seqs"] - 1)]


def _append_lengths(c):
    """(new tokens, kv length after them) of each sequence of an append."""
    rng = _rng(c)
    cuts = sorted(rng.sample(range(1, c["tokens"]), c["seqs"] - 1)) if c["seqs"] > 1 else []
    ends = [0] + cuts + [c["tokens"]]
    return [(b - a, b - a + rng.randint(0, c["context"])) for a, b in zip(ends, ends[1:])]


# ------------------------------------------------------------------ the inputs
def _inv_freq(rot, factor, dev):
    """Radians a position for each rotated pair, fp64.  factor > 1 stretches the pairs that turn fewer than 32 times
    over the trained context, wholly where they turn less than once."""
    w = _THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    if factor > 1.0:
        keep = ((_TRAINED * w / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        w = w * (keep + (1.0 - keep) / factor)
    return w


def _amplitude(factor):
    return 1.0 if factor <= 1.0 else 0.1 * math.log(factor) + 1.0


def _pages(c, lengths, gen, dev):
    """A page table that places each sequence's pages anywhere in the pool, and the number of pages of the pool."""
    counts = [-(-n // c["page"]) for n in lengths]
    total, most = sum(counts), max(1, max(counts))
    pool = total + 3
    order = torch.randperm(pool, generator=gen, device=dev)[:total].to(torch.int32)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32, device=dev)
    table[torch.arange(most, device=dev)[None, :] < torch.tensor(counts, device=dev)[:, None]] = order
    return table, pool


def _pool(c, pool, gen, dev):
    """One of the two pools [pages, kv_heads, page, dim] with values in all of it, and its scales."""
    shape = (pool, c["kv_heads"], c["page"], c["dim"])
    if c["cache"] == "bf16":
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen), None
    data = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, 50.0, generator=gen)
    scale = (0.01 + 0.02 * torch.rand(c["kv_heads"], generator=gen, device=dev)).float()
    return data.to(torch.float8_e4m3fn), scale


def _framework():
    from nvfp4_w4a16_moe_skinny_gb300 import binding
    return binding


def _int32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = case
    s = {"case": c}
    if own:
        s["lib"] = _framework().load()

    def rows(tokens, heads):
        return torch.empty(tokens, heads, c["dim"], dtype=torch.bfloat16, device=dev).normal_(generator=gen)

    if c["op"] in ("norm", "grad", "append"):
        kind = torch.bfloat16 if c["weight"] == "bf16" else torch.float32
        s["q_norm"], s["k_norm"] = ((1.0 + 0.2 * torch.randn(c["dim"], generator=gen, device=dev)).to(kind)
                                    for _ in range(2))
        s["inv_freq"], s["amplitude"] = _inv_freq(c["rot"], c["factor"], dev), _amplitude(c["factor"])
    if c["op"] in ("norm", "grad"):
        h, kv = c["heads"], c["kv_heads"]
        qkv = rows(c["tokens"], h + kv + (kv if c["wide"] else 0))  # a fused projection's rows
        qkv.mul_(0.5 + torch.rand(c["tokens"], 1, 1, generator=gen, device=dev))  # tokens of different sizes
        s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + kv]
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=gen, device=dev).to(torch.int32)
        if c["op"] == "grad":
            s["dq"], s["dk"] = rows(c["tokens"], h), rows(c["tokens"], kv)
        return s
    if c["op"] == "assign":
        return _prepare_assign(c, s, seed, gen, dev)
    if c["op"] == "append":
        lengths = _append_lengths(c)
        n = torch.tensor([a for a, _ in lengths], device=dev)
        kv_len = torch.tensor([b for _, b in lengths], device=dev)
        table, pool = _pages(c, [b for _, b in lengths], gen, dev)
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), n)
        pos = (kv_len - n.cumsum(0))[seq] + torch.arange(c["tokens"], device=dev)
        s["slots"] = table[seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
        s["positions"] = pos.to(torch.int32)
        h, kv = c["heads"], c["kv_heads"]
        qkv = rows(c["tokens"], h + 2 * kv)
        qkv.mul_(0.5 + torch.rand(c["tokens"], 1, 1, generator=gen, device=dev))
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    else:
        trees = _trees(c)
        s["kv_len"] = _int32([b for _, b, _ in trees], dev)
        cu = [0]
        for n, _, _ in trees:
            cu.append(cu[-1] + n)
        s["cu"] = _int32(cu, dev)
        s["table"], pool = _pages(c, [b for _, b, _ in trees], gen, dev)
        if c["op"] == "tree":
            s["q"] = rows(cu[-1], c["heads"])
            words = -(-c["new"] // 64)
            seen = torch.zeros(cu[-1], 64 * words, dtype=torch.bool)
            for first, (n, _, parents) in zip(cu, trees):
                for i, p in enumerate(parents):
                    if p >= 0:
                        seen[first + i] = seen[first + p]
                    seen[first + i, i] = True
            bit = torch.ones(64, dtype=torch.int64) << torch.arange(64)
            s["masks"] = (seen.view(-1, words, 64) * bit).sum(-1).to(dev)
        else:
            rng = _rng(c)
            paths = [_accepted(rng, parents) for _, _, parents in trees]
            most = max(len(p) for p in paths) + 2
            s["paths"] = _int32([p + [-1] * (most - len(p)) for p in paths], dev)
    s["k_cache"], s["k_scale"] = _pool(c, pool, gen, dev)
    s["v_cache"], s["v_scale"] = _pool(c, pool, gen, dev)
    if own:  # the handles that a serving program makes once for its pools and once a step for its batch
        binding = _framework()
        s["cache"] = binding.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] != "append":
            s["batch"] = binding.Batch(s["cu"], s["kv_len"], s["table"], c["new"])
    return s


def _prepare_assign(c, s, seed, gen, dev):
    """Requests in the middle of their lives: committed lengths, the pages that they hold (a rejected draft's among
    them), the free pages, and the new tokens of this step."""
    rng = random.Random(seed)
    counts, page = _counts(c), c["page"]
    s["new"] = _int32(counts, dev)
    lengths = [rng.randint(0, c["context"]) for _ in counts]
    s["kv_len"] = _int32(lengths, dev)
    held = [min(-(-n // page) + rng.choice([0, 0, 0, 1]), -(-(c["context"] + 1) // page)) for n in lengths]
    s["held"] = _int32(held, dev)
    most = -(-(c["context"] + c["new"]) // page) + 1
    pool = sum(-(-(c["context"] + max(1, m)) // page) for m in counts) + c["spare"]  # enough for the longest
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    s["table"] = torch.full((c["seqs"], most), -1, dtype=torch.int32, device=dev)
    s["table"][torch.arange(most, device=dev)[None, :] < s["held"][:, None]] = order[:sum(held)]
    s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=dev)
    s["free"][:pool - sum(held)] = order[sum(held):]
    s["free_count"] = _int32([pool - sum(held)], dev)
    s["tokens"] = sum(max(0, n) for n in counts) + c["spare"]  # a captured step's rows, some of them unused
    s["words"] = -(-c["new"] // 64) if c["kind"] == "tree" else 0
    s["parents"] = None
    if s["words"]:
        s["parents"] = _int32([p for n in counts for p in _parents(rng, n)] + [-1] * c["spare"], dev)
    if own:
        binding = _framework()
        s["pages"] = binding.PageTable(s["table"], s["held"], s["free"], s["free_count"], page)
        s["step"] = binding.Step(c["seqs"], s["tokens"], s["words"], dev)
    return s


# ------------------------------------------------------------------ one pass
def _turn(f, positions, inv_freq, interleaved, amplitude, back=False):
    """Rotary positions on the first 2 * len(inv_freq) values of each fp32 head, with fp64 angles."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    cos = (amplitude * angle.cos()).float()[:, None, :]
    sin = (amplitude * angle.sin()).float()[:, None, :]
    if back:
        sin = -sin
    r = f[..., :2 * half]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, f[..., 2 * half:]), -1)


def _root(f):
    return (f.square().mean(-1, keepdim=True) + _EPS).rsqrt()


def _normed(s, x, weight):
    f = x.float()
    return _turn(f * _root(f) * weight.float(), s["positions"], s["inv_freq"], s["case"]["interleaved"],
                 s["amplitude"])


def _plain_gradient(s, dy, x, weight):
    f = x.float()
    r = _root(f)
    unit = f * r
    u = _turn(dy.float(), s["positions"], s["inv_freq"], s["case"]["interleaved"], s["amplitude"], back=True)
    z = u * weight.float()
    dx = r * (z - unit * (z * unit).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (u * unit).sum((0, 1))


def _plain_append(s):
    c = s["case"]
    k, v = _normed(s, s["k"], s["k_norm"]), s["v"].float()
    q = _normed(s, s["q"], s["q_norm"]).to(torch.bfloat16)
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    if c["cache"] == "bf16":
        s["k_cache"][page, :, off] = k.to(torch.bfloat16)
        s["v_cache"][page, :, off] = v.to(torch.bfloat16)
    else:
        k = (k / s["k_scale"][:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        v = (v / s["v_scale"][:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["k_cache"].view(torch.uint8)[page, :, off] = k.view(torch.uint8)
        s["v_cache"].view(torch.uint8)[page, :, off] = v.view(torch.uint8)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_assign(s):
    c, dev = s["case"], s["new"].device
    page, rows = c["page"], s["tokens"]
    n, ctx, held = s["new"].long().clamp(min=0), s["kv_len"].long(), s["held"].long()
    done = s["new"] < 0
    cu = torch.zeros(c["seqs"] + 1, dtype=torch.int64, device=dev)
    cu[1:] = n.cumsum(0)
    kv_len = torch.where(done, 0, ctx + n)
    # pages from the top of the free list, in the order of the requests
    need = torch.where(done, 0, ((ctx + n + page - 1) // page - held).clamp(min=0))
    first = need.cumsum(0) - need
    col = torch.arange(s["table"].shape[1], device=dev)[None, :]
    rank = first[:, None] + col - held[:, None]
    is_new = (col >= held[:, None]) & (col < (held + need)[:, None])
    count = s["free_count"].long()
    taken = s["free"][(count - 1 - rank).clamp(0, s["free"].numel() - 1)]
    table = torch.where(is_new, taken, s["table"])
    # finished requests' pages go on top of what is left
    back = torch.where(done, held, 0)
    left = count - need.sum()
    place = left + (back.cumsum(0) - back)[:, None] + col
    gone = done[:, None] & (col < held[:, None])
    s["free"][place[gone]] = table[gone]
    s["table"].copy_(table)
    s["held"].copy_(torch.where(done, 0, held + need))
    s["free_count"].copy_(left + back.sum())
    t = torch.arange(rows, device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = t < cu[-1]
    seq = seq.clamp(max=c["seqs"] - 1)
    i = t - cu[seq]
    at = torch.where(live, ctx[seq] + i, 0)
    slots = torch.where(live, table[seq, at // page].long() * page + at % page, -1)
    positions, masks = at, torch.zeros(rows, s["words"], dtype=torch.int64, device=dev)
    if s["words"]:
        # reach[t, x]: token x of its sequence is an ancestor of t or t itself; doubled until the deepest is done
        width = 64 * s["words"]
        j = torch.arange(width, device=dev)
        up = torch.where(live & (s["parents"] >= 0), cu[seq] + s["parents"], rows)
        up = torch.cat((up, torch.tensor([rows], device=dev)))
        reach = torch.cat((live[:, None] & (j == i[:, None]), torch.zeros(1, width, dtype=torch.bool, device=dev)))
        for _ in range(max(1, (c["new"] - 1).bit_length())):
            reach = reach | reach[up]
            up = up[up]
        reach = reach[:rows]
        positions = torch.where(live, ctx[seq] + reach.sum(-1) - 1, 0)
        bit = torch.ones(64, dtype=torch.int64, device=dev) << torch.arange(64, device=dev)
        masks = (reach.view(rows, -1, 64) * bit).sum(-1)
    return {"slots": slots, "positions": positions.to(torch.int32), "cu_tokens": cu.to(torch.int32),
            "kv_len": kv_len.to(torch.int32), "masks": masks, "table": s["table"], "held": s["held"],
            "free": s["free"], "free_count": s["free_count"]}


def _plain_accept(s):
    c = s["case"]
    paths = s["paths"].long()
    ctx = s["kv_len"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    taken = paths >= 0
    seq, d = taken.nonzero(as_tuple=True)
    to, frm = ctx[seq] + d, ctx[seq] + paths[taken]
    p = c["page"]
    to_page, to_off = s["table"][seq, to // p].long(), to % p
    from_page, from_off = s["table"][seq, frm // p].long(), frm % p
    k = s["k_cache"].view(torch.uint8 if c["cache"] == "e4m3" else torch.bfloat16)
    v = s["v_cache"].view(k.dtype)
    k[to_page, :, to_off] = k[from_page, :, from_off]
    v[to_page, :, to_off] = v[from_page, :, from_off]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_len": (ctx + taken.sum(-1)).to(torch.int32)}


def _gathered(cache, scale, table):
    """[seqs, kv_heads, keys, dim] fp32: every sequence's pages in order (page 0 in the place of no page)."""
    b, p = table.shape
    x = cache.view(torch.uint8)[table.clamp(min=0).long()].view(cache.dtype).float()
    x = x.permute(0, 2, 1, 3, 4).reshape(b, cache.shape[1], p * cache.shape[2], cache.shape[3])
    return x if scale is None else x * scale[:, None, None]


def _plain_tree(s):
    c = s["case"]
    h, kv, d = c["heads"], c["kv_heads"], c["dim"]
    g, b, n = h // kv, c["seqs"], c["new"]
    dev = s["q"].device
    cu, kv_len, tokens = s["cu"].long(), s["kv_len"].long(), s["q"].shape[0]
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    q = s["q"].float()[at].view(b, n, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * n, d)
    k = _gathered(s["k_cache"], s["k_scale"], s["table"])
    v = _gathered(s["v_cache"], s["v_scale"], s["table"])
    scores = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    if c["softcap"] > 0:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    # the new tokens that each one sees, and the first key of the context
    seen = (s["masks"][at][..., i // 64] >> (i % 64)) & 1                       # [b, token, new token]
    low = torch.zeros(b, n, dtype=torch.int64, device=dev)
    ctx = kv_len - count
    if c["window"] > 0:
        low = ctx[:, None] + seen.sum(-1) - c["window"]
        seen = seen * (seen.flip(-1).cumsum(-1).flip(-1) <= c["window"])
    j = torch.arange(scores.shape[-1], device=dev)
    new = (j - ctx[:, None]).clamp(0, n - 1)
    tail = torch.gather(seen, 2, new[:, None, :].expand(-1, n, -1)) > 0
    tail &= ((j >= ctx[:, None]) & (j < kv_len[:, None]))[:, None]
    sees = ((j < ctx[:, None, None]) & (j >= low[..., None])) | tail
    scores = scores.view(b, kv, g, n, -1).masked_fill_(~sees[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, kv, g * n, -1) @ v).view(b, kv, g, n, d) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=dev), right=True)
    idx = torch.arange(tokens, device=dev) - cu[seq]
    out = out.permute(0, 3, 1, 2, 4)[seq, idx].reshape(tokens, h, d).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[seq, idx].reshape(tokens, h)}


def run(state):
    s = state
    c = s["case"]
    if c["op"] == "norm":
        if own:
            q, k = s["lib"].qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_norm"], s["k_norm"],
                                         eps=_EPS, interleaved=c["interleaved"], amplitude=s["amplitude"])
            return {"q": q, "k": k}
        return {"q": _normed(s, s["q"], s["q_norm"]).to(torch.bfloat16),
                "k": _normed(s, s["k"], s["k_norm"]).to(torch.bfloat16)}
    if c["op"] == "grad":
        if own:
            dq, dk, dqn, dkn = s["lib"].qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"],
                                                              s["inv_freq"], s["q_norm"], s["k_norm"], eps=_EPS,
                                                              interleaved=c["interleaved"], amplitude=s["amplitude"])
        else:
            dq, dqn = _plain_gradient(s, s["dq"], s["q"], s["q_norm"])
            dk, dkn = _plain_gradient(s, s["dk"], s["k"], s["k_norm"])
        return {"dq": dq, "dk": dk, "dq_norm": dqn, "dk_norm": dkn}
    if c["op"] == "append":
        if own:
            q = s["lib"].kv_append(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"],
                                   inv_freq=s["inv_freq"], interleaved=c["interleaved"], amplitude=s["amplitude"],
                                   q=s["q"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=_EPS)
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        return _plain_append(s)
    if c["op"] == "assign":
        if own:
            t = s["lib"].kv_assign(s["pages"], s["kv_len"], s["new"], s["step"], parents=s["parents"])
            return {"slots": t.slots, "positions": t.positions, "cu_tokens": t.cu_tokens, "kv_len": t.kv_len,
                    "masks": t.masks, "table": s["table"], "held": s["held"], "free": s["free"],
                    "free_count": s["free_count"]}
        return _plain_assign(s)
    if c["op"] == "accept":
        if own:
            kv_len = s["lib"].kv_accept(s["cache"], s["batch"], s["paths"])
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_len": kv_len}
        return _plain_accept(s)
    if own:
        out, lse = s["lib"].tree_attention(s["q"], s["cache"], s["batch"], s["masks"], window=c["window"],
                                           softcap=c["softcap"], with_lse=True)
        return {"out": out, "lse": lse}
    return _plain_tree(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("norm", "grad", "append"):
        weight = 2 if c["weight"] == "bf16" else 4
        q, k = c["tokens"] * c["heads"] * c["dim"], c["tokens"] * c["kv_heads"] * c["dim"]
        turned = 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot"]
        fixed = 4 * c["tokens"] + 4 * c["rot"] + 2 * weight * c["dim"]
        if c["op"] == "norm":
            return {"bytes": 4 * (q + k) + fixed, "flops": 4 * (q + k) + turned}
        if c["op"] == "grad":
            return {"bytes": 6 * (q + k) + fixed + 8 * c["dim"], "flops": 12 * (q + k) + turned}
        size = 2 if c["cache"] == "bf16" else 1
        return {"bytes": 4 * q + 2 * k * (2 + size) + fixed + 8 * c["tokens"], "flops": 4 * (q + k) + turned}
    if c["op"] == "assign":
        tokens = sum(max(0, n) for n in _counts(c)) + c["spare"]
        words = -(-c["new"] // 64) if c["kind"] == "tree" else 0
        # lengths, new tokens, pages held (in and out), ends and lengths out; a page id for each page that is written to
        pages = sum(-(-max(0, n) // c["page"]) for n in _counts(c))
        return {"bytes": 24 * c["seqs"] + 4 * pages + (12 + 8 * words + (4 if words else 0)) * tokens,
                "flops": 4 * tokens}
    trees = _trees(c)
    size = 2 if c["cache"] == "bf16" else 1
    if c["op"] == "accept":
        rng = _rng(c)
        moved = sum(d != i for _, _, parents in trees for d, i in enumerate(_accepted(rng, parents)))
        return {"bytes": 4 * moved * c["kv_heads"] * c["dim"] * size + 24 * c["seqs"] + 12 * moved, "flops": 0}
    tokens = keys = pairs = 0
    w = c["window"] or (1 << 60)
    for n, length, parents in trees:
        tokens += n
        ctx = length - n
        depth = [0] * n
        for i, p in enumerate(parents):
            depth[i] = 1 + (depth[p] if p >= 0 else 0)
        keys += n + min(ctx, w - 1)  # seen by some token
        pairs += sum(min(w, ctx + e) for e in depth)
    rows = tokens * c["heads"]
    return {"bytes": rows * c["dim"] * 4 + rows * 4 + keys * c["kv_heads"] * c["dim"] * 2 * size
            + 4 * (-(-keys // c["page"]) + 2 * c["seqs"] + 1) + 8 * tokens * -(-c["new"] // 64),
            "flops": 4 * c["dim"] * c["heads"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _turned64(x, s, sign=1.0):
    """The rotation as a product of complex numbers."""
    interleaved, r = s["case"]["interleaved"], 2 * s["inv_freq"].numel()
    z = x[..., :r].unflatten(-1, (-1, 2)) if interleaved else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous())
    angle = sign * torch.outer(s["positions"].double(), s["inv_freq"])[:, None, :]
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, s["amplitude"]), angle))
    y = x.clone()
    y[..., :r] = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return y


def _unit64(x):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS)


def _gradient64(s, dy, x, weight):
    """dx is what is left of weight * u beside x's direction, shrunk by the norm."""
    x, u = x.double(), _turned64(dy.double(), s, -1.0)
    size = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS)
    z = u * weight.double()
    along = (z * x).sum(-1, keepdim=True) / (x.shape[-1] * size * size)
    return (z - along * x) / size, (u * x / size).flatten(0, 1).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        return {"q": _turned64(_unit64(s["q"]) * s["q_norm"].double(), s),
                "k": _turned64(_unit64(s["k"]) * s["k_norm"].double(), s)}
    if c["op"] == "grad":
        dq, dqn = _gradient64(s, s["dq"], s["q"], s["q_norm"])
        dk, dkn = _gradient64(s, s["dk"], s["k"], s["k_norm"])
        return {"dq": dq, "dk": dk, "dq_norm": dqn, "dk_norm": dkn}
    if c["op"] == "append":
        out = {"q": _turned64(_unit64(s["q"]) * s["q_norm"].double(), s)}
        for name, rows in (("k", _turned64(_unit64(s["k"]) * s["k_norm"].double(), s)), ("v", s["v"].double())):
            pool = s[name + "_cache"].double()
            if c["cache"] == "e4m3":
                rows = (rows / s[name + "_scale"].double()[:, None]).clamp(-448.0, 448.0)
            flat = pool.transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])
            flat[s["slots"]] = rows
            out[name + "_cache"] = flat.view(-1, c["page"], c["kv_heads"], c["dim"]).transpose(1, 2).contiguous()
        return out
    if c["op"] == "assign":
        return _exact_assign(c, s)
    if c["op"] == "accept":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        kv_len, table = s["kv_len"].tolist(), s["table"].tolist()
        for b, (path, (n, length, _)) in enumerate(zip(s["paths"].tolist(), _trees(c))):
            path = [i for i in path if i >= 0]
            places = [divmod(length - n + d, c["page"]) for d in range(n)]
            for x in (k, v):
                old = [x[table[b][at], :, off].clone() for at, off in (places[i] for i in path)]
                for (at, off), value in zip(places, old):
                    x[table[b][at], :, off] = value
            kv_len[b] = length - n + len(path)
        return {"k_cache": k, "v_cache": v, "kv_len": _int32(kv_len, k.device)}
    h, kv, d = c["heads"], c["kv_heads"], c["dim"]
    g = h // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    at = 0
    for b, (n, length, parents) in enumerate(_trees(c)):
        pages = s["table"][b, :-(-length // c["page"])].long()
        hidden = torch.zeros(n, length, dtype=torch.bool)
        for i in range(n):
            mine = _path_to(parents, i)
            hidden[i, length - n:] = True
            hidden[i, [length - n + t for t in mine]] = False
            if c["window"]:
                keys = list(range(max(0, length - n - c["window"]), length - n)) + [length - n + t for t in mine]
                hidden[i] = True
                hidden[i, keys[-c["window"]:]] = False
        hidden = hidden.to(out.device)
        for e in range(kv):
            keys = s["k_cache"][pages, e].double().reshape(-1, d)[:length]
            values = s["v_cache"][pages, e].double().reshape(-1, d)[:length]
            if c["cache"] == "e4m3":
                keys, values = keys * s["k_scale"][e].double(), values * s["v_scale"][e].double()
            for r in range(e * g, (e + 1) * g):
                x = s["q"][at:at + n, r].double() @ keys.T / math.sqrt(d)
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                x[hidden] = float("-inf")
                z = torch.logsumexp(x, -1)
                lse[at:at + n, r] = z
                out[at:at + n, r] = torch.exp(x - z[:, None]) @ values
        at += n
    return {"out": out, "lse": lse}


def _exact_assign(c, s):
    """One request after the other."""
    table, held, free = s["table"].tolist(), s["held"].tolist(), s["free"].tolist()
    count, page, rows = int(s["free_count"]), c["page"], s["tokens"]
    parents = s["parents"].tolist() if s["words"] else None
    slots, positions, masks = [-1] * rows, [0] * rows, [[0] * s["words"] for _ in range(rows)]
    cu, kv_len, gone = [0], [], []
    for b, (n, ctx) in enumerate(zip(s["new"].tolist(), s["kv_len"].tolist())):
        if n < 0:
            gone += table[b][:held[b]]
            held[b] = 0
            kv_len.append(0)
            cu.append(cu[-1])
            continue
        while held[b] * page < ctx + n:
            count -= 1
            table[b][held[b]] = free[count]
            held[b] += 1
        for i in range(n):
            t = cu[-1] + i
            slots[t] = table[b][(ctx + i) // page] * page + (ctx + i) % page
            positions[t] = ctx + i
            if parents:
                path = _path_to(parents[cu[-1]:cu[-1] + n], i)
                positions[t] = ctx + len(path) - 1
                for w in range(s["words"]):
                    value = sum(1 << (x - 64 * w) for x in path if x // 64 == w)
                    masks[t][w] = value - (1 << 64) if value >> 63 else value
        cu.append(cu[-1] + n)
        kv_len.append(ctx + n)
    free[count:count + len(gone)] = gone
    dev = s["table"].device
    return {"slots": torch.tensor(slots, device=dev), "positions": _int32(positions, dev), "cu_tokens": _int32(cu, dev),
            "kv_len": _int32(kv_len, dev),
            "masks": torch.tensor(masks, dtype=torch.int64, device=dev).view(rows, s["words"]),
            "table": _int32(table, dev), "held": _int32(held, dev), "free": _int32(free, dev),
            "free_count": _int32([count + len(gone)], dev)}
