"""The attention side of a decode step: rotary positions, the append to a paged key/value cache, and attention over it.

Each case is one call of one operator.  ``own`` false computes it with elementary torch operations in fp32
(angles in fp64), rounded once; ``own`` true calls the framework.  Head counts, lengths and page sizes are generic
ones around this repository's own workloads (a verify block of 15 tokens, a prefill chunk of 512, 64K contexts and
beyond); the cache is bf16 or E4M3 with an fp32 scale per kv head.

Layouts: rows of heads [tokens, heads, dim] (possibly slices of a wider row, as a fused projection leaves them);
the cache [pages, kv_heads, page_size, dim] for K and for V; a page table [seqs, max_pages] with -1 past a
sequence's last page.  Token i of a sequence's n new tokens is at position kv_len - n + i and sees the keys at or
before it (the last ``window`` of them, where a window is set).
"""

import math
import random

import torch

own = False

_THETA = 500000.0
_TRAINED = 8192.0  # the context that the frequencies were trained for, where they are stretched beyond it


# ------------------------------------------------------------------ the cases
def _rope(name, tokens, heads, dim, rot, interleaved, factor, far, wide):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, dim=dim, rot=rot, interleaved=interleaved,
                factor=factor, far=far, wide=wide)


def _append(name, seqs, tokens, heads, kv_heads, dim, rot, interleaved, factor, context, page, cache):
    return dict(name=name, op="append", seqs=seqs, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, factor=factor, context=context, page=page, cache=cache)


def _attention(name, seqs, new, context, ragged, heads, kv_heads, dim, page, cache, window=0, softcap=0.0):
    return dict(name=name, op="attention", seqs=seqs, new=new, context=context, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, cache=cache, window=window, softcap=softcap)


def listed():
    return [
        # the queries of one verify block: a launch's latency
        _rope("rope_verify_block", 15, 16, 128, 128, False, 1.0, 8192, False),
        # a long prompt's queries in a fused projection's rows, half of the head rotated, stretched frequencies
        _rope("rope_long_prompt", 16381, 32, 128, 64, True, 8.0, 131072, True),
        # one decode step of 16 sequences: q and k rotated, k and v written to their pages
        _append("append_step", 16, 16, 16, 8, 128, 128, False, 1.0, 4096, 64, "bf16"),
        # a prefill's tokens quantized into small pages
        _append("append_prompt_e4m3", 3, 8191, 32, 8, 128, 128, False, 8.0, 20000, 16, "e4m3"),
        # one sequence's decode step at a short context: latency
        _attention("attention_one", 1, 1, 999, "no", 16, 8, 128, 16, "bf16"),
        # a serving batch's decode step, contexts from a few tokens to 16K
        _attention("attention_batch", 64, 1, 16383, "spread", 32, 8, 128, 64, "bf16"),
        # two very long conversations on a quantized cache
        _attention("attention_long_e4m3", 2, 1, 131070, "no", 64, 8, 128, 128, "e4m3"),
        # verify blocks of 15 tokens in a sliding-window layer with wide heads and capped logits
        _attention("attention_verify_window", 4, 15, 8177, "spread", 16, 8, 256, 32, "bf16", 1024, 50.0),
        # a prefill chunk of 512 tokens in such a layer
        _attention("attention_chunk_window", 1, 512, 7680, "no", 16, 8, 256, 32, "bf16", 1024, 0.0),
        # continuous batching: prompt pieces of odd lengths and single tokens in one call, seven heads to a kv head
        _attention("attention_mixed_e4m3", 12, 1501, 4500, "mixed", 28, 4, 64, 16, "e4m3"),
        # a whole prompt at once
        _attention("attention_prompt", 1, 4096, 0, "no", 32, 8, 128, 64, "bf16"),
        # the last chunk of a long prompt
        _attention("attention_chunk_long", 1, 2048, 30720, "no", 32, 8, 128, 64, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    factor = rng.choice([1.0, 4.0, 8.0])
    interleaved = rng.random() < 0.5
    if op == "rope":
        heads = kv_heads * group
        tokens = _log_int(rng, 1, min(32768, (1 << 26) // (heads * dim)))
        c = _rope("", tokens, heads, dim, rot, interleaved, factor, _log_int(rng, 64, 1 << 20), rng.random() < 0.5)
    elif op == "append":
        tokens = _log_int(rng, 1, min(16384, (1 << 25) // (kv_heads * group * dim)))
        seqs = rng.randint(1, min(tokens, 64))
        c = _append("", seqs, tokens, kv_heads * group, kv_heads, dim, rot, interleaved, factor,
                    _log_int(rng, 1, 30000), page, cache)
    else:
        while True:
            seqs = _log_int(rng, 1, 96)
            new = rng.choice([1, 1, rng.randint(2, 16), _log_int(rng, 17, 4096)])
            context = _log_int(rng, 1, 131072) - 1
            ragged = rng.choice(["no", "spread", "mixed" if new > 1 else "spread"])
            window = rng.choice([0, 0, 0, _log_int(rng, 64, 4096)])
            softcap = rng.choice([0.0, 0.0, 50.0])
            c = _attention("", seqs, new, context, ragged, kv_heads * group, kv_heads, dim, page, cache, window,
                           softcap)
            # the plain form keeps padded fp32 keys and scores
            if (seqs * kv_heads * group * new * (context + new) <= 32 * 2048 * 32768
                    and seqs * kv_heads * dim * (context + new) <= 64 * 16384 * 8 * 128
                    and work(c)["flops"] <= work(listed()[-1])["flops"]):
                break
    del c["name"]
    return c


def _lengths(c):
    """(new tokens, kv length) of each sequence: from the case alone."""
    rng = random.Random("%d %d %d" % (c["seqs"], c["new"], c["context"]))
    out = []
    for b in range(c["seqs"]):
        n, ctx = c["new"], c["context"]
        if b > 0 and c["ragged"] != "no":
            ctx = _log_int(rng, 1, ctx + 1) - 1
        if b > 0 and c["ragged"] == "mixed":
            n = 1 if b % 2 else _log_int(rng, max(1, n // 8), n)
        out.append((n, n + ctx))
    return out


def _append_lengths(c):
    """(new tokens, kv length after them) of each sequence of an append."""
    rng = random.Random("%d %d %d" % (c["seqs"], c["tokens"], c["context"]))
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
    counts = [-(-n // c["page"]) for _, n in lengths]
    total, most = sum(counts), max(1, max(counts))
    pool = total + 3
    order = torch.randperm(pool, generator=gen, device=dev)[:total].to(torch.int32)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32, device=dev)
    fill = torch.arange(most, device=dev)[None, :] < torch.tensor(counts, device=dev)[:, None]
    table[fill] = order
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


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c = case
    s = {"case": c}

    def rows(tokens, heads):
        return torch.empty(tokens, heads, c["dim"], dtype=torch.bfloat16, device=dev).normal_(generator=gen)

    if c["op"] == "rope":
        extra = 2 * max(1, c["heads"] // 4) if c["wide"] else 0  # k and v heads after the queries in a fused row
        s["x"] = rows(c["tokens"], c["heads"] + extra)[:, :c["heads"]]
        s["positions"] = torch.randint(0, c["far"], (c["tokens"],), generator=gen, device=dev).to(torch.int32)
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"], dev)
        s["amplitude"] = _amplitude(c["factor"])
        if own:
            s["lib"] = _framework().load()
        return s
    lengths = _append_lengths(c) if c["op"] == "append" else _lengths(c)
    n = torch.tensor([a for a, _ in lengths], device=dev)
    kv_len = torch.tensor([b for _, b in lengths], device=dev)
    cu = torch.zeros(len(lengths) + 1, dtype=torch.int64, device=dev)
    cu[1:] = n.cumsum(0)
    tokens = sum(a for a, _ in lengths)
    table, pool = _pages(c, lengths, gen, dev)
    s["k_cache"], s["k_scale"] = _pool(c, pool, gen, dev)
    s["v_cache"], s["v_scale"] = _pool(c, pool, gen, dev)
    if c["op"] == "append":
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), n)
        pos = kv_len[seq] - n[seq] + torch.arange(tokens, device=dev) - cu[seq]
        s["slots"] = table[seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
        s["positions"] = pos.to(torch.int32)
        h, kv = c["heads"], c["kv_heads"]
        qkv = rows(tokens, h + 2 * kv)  # a fused projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        s["inv_freq"] = _inv_freq(c["rot"], c["factor"], dev)
        s["amplitude"] = _amplitude(c["factor"])
    else:
        s["q"] = rows(tokens, c["heads"])
        s["cu"], s["kv_len"], s["table"] = cu.to(torch.int32), kv_len.to(torch.int32), table
    if own:  # the handles that a serving program makes once for its pools and once a step for its batch
        binding = _framework()
        s["lib"] = binding.load()
        s["cache"] = binding.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "attention":
            s["batch"] = binding.Batch(s["cu"], s["kv_len"], s["table"], c["new"])
    return s


# ------------------------------------------------------------------ one pass
def _rotate(x, positions, inv_freq, interleaved, amplitude):
    """Rotary positions on the first 2 * len(inv_freq) values of each head, in fp32 with fp64 angles."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    cos = (amplitude * angle.cos()).float()[:, None, :]
    sin = (amplitude * angle.sin()).float()[:, None, :]
    f = x.float()
    r = f[..., :2 * half]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, f[..., 2 * half:]), -1)


def _plain_append(s):
    c = s["case"]
    k = _rotate(s["k"], s["positions"], s["inv_freq"], c["interleaved"], s["amplitude"])
    v = s["v"].float()
    q = _rotate(s["q"], s["positions"], s["inv_freq"], c["interleaved"], s["amplitude"]).to(torch.bfloat16)
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


def _gathered(cache, scale, table):
    """[seqs, kv_heads, keys, dim] fp32: every sequence's pages in order (page 0 in the place of no page)."""
    b, p = table.shape
    x = cache.view(torch.uint8)[table.clamp(min=0).long()].view(cache.dtype).float()
    x = x.permute(0, 2, 1, 3, 4).reshape(b, cache.shape[1], p * cache.shape[2], cache.shape[3])
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
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
    pos = (kv_len - count)[:, None] + i
    j = torch.arange(scores.shape[-1], device=dev)
    sees = (j <= pos[..., None]) & (j < kv_len[:, None, None])
    if c["window"] > 0:
        sees = sees & (j > pos[..., None] - c["window"])
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
    if c["op"] == "rope":
        if own:
            return s["lib"].rope_apply(s["x"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                                       amplitude=s["amplitude"])
        return _rotate(s["x"], s["positions"], s["inv_freq"], c["interleaved"], s["amplitude"]).to(torch.bfloat16)
    if c["op"] == "append":
        if own:
            q = s["lib"].kv_append(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"],
                                   inv_freq=s["inv_freq"], interleaved=c["interleaved"], amplitude=s["amplitude"],
                                   q=s["q"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        return _plain_append(s)
    if own:
        out, lse = s["lib"].paged_attention(s["q"], s["cache"], s["batch"], window=c["window"], softcap=c["softcap"],
                                            with_lse=True)
        return {"out": out, "lse": lse}
    return _plain_attention(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        values = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * values + 4 * c["tokens"] + 4 * c["rot"],
                "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    size = 2 if c["cache"] == "bf16" else 1
    if c["op"] == "append":
        q, k = c["tokens"] * c["heads"] * c["dim"], c["tokens"] * c["kv_heads"] * c["dim"]
        return {"bytes": 4 * q + 2 * k * (2 + size) + 12 * c["tokens"] + 4 * c["rot"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot"]}
    tokens = keys = pairs = 0
    w = c["window"] or (1 << 60)
    for n, length in _lengths(c):
        tokens += n
        ctx = length - n
        keys += length - max(0, ctx - w + 1)  # seen by some token
        full = max(0, min(n, w - ctx))  # tokens whose window reaches back to the first key
        pairs += full * ctx + full * (full + 1) // 2 + (n - full) * w if c["window"] else n * ctx + n * (n + 1) // 2
    rows = tokens * c["heads"]
    return {"bytes": rows * c["dim"] * 4 + rows * 4 + keys * c["kv_heads"] * c["dim"] * 2 * size
            + 4 * (-(-keys // c["page"]) + 2 * c["seqs"] + 1),
            "flops": 4 * c["dim"] * c["heads"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _turned64(x, positions, inv_freq, interleaved, amplitude):
    """The rotation as a product of complex numbers."""
    r = 2 * inv_freq.numel()
    x = x.double()
    z = x[..., :r].unflatten(-1, (-1, 2)) if interleaved else x[..., :r].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous())
    angle = torch.outer(positions.double(), inv_freq)[:, None, :]
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, amplitude), angle))
    y = x.clone()
    y[..., :r] = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _turned64(s["x"], s["positions"], s["inv_freq"], c["interleaved"], s["amplitude"])
    if c["op"] == "append":
        turn = lambda x: _turned64(x, s["positions"], s["inv_freq"], c["interleaved"], s["amplitude"])  # noqa: E731
        out = {"q": turn(s["q"])}
        for name, rows in (("k", turn(s["k"])), ("v", s["v"].double())):
            pool = s[name + "_cache"].double()
            if c["cache"] == "e4m3":
                rows = (rows / s[name + "_scale"].double()[:, None]).clamp(-448.0, 448.0)
            flat = pool.transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])
            flat[s["slots"]] = rows
            out[name + "_cache"] = flat.view(-1, c["page"], c["kv_heads"], c["dim"]).transpose(1, 2).contiguous()
        return out
    h, kv, d = c["heads"], c["kv_heads"], c["dim"]
    g = h // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=out.device)
    at = 0
    for b, (n, length) in enumerate(_lengths(c)):
        pages = s["table"][b, :-(-length // c["page"])].long()
        qpos = torch.arange(length - n, length, device=out.device)
        for e in range(kv):
            keys = s["k_cache"][pages, e].double().reshape(-1, d)[:length]
            values = s["v_cache"][pages, e].double().reshape(-1, d)[:length]
            if c["cache"] == "e4m3":
                keys, values = keys * s["k_scale"][e].double(), values * s["v_scale"][e].double()
            step = max(1, (1 << 27) // length)  # tokens at a time
            for t in range(0, n, step):
                here = qpos[t:t + step]
                hidden = torch.arange(length, device=out.device) > here[:, None]
                if c["window"]:
                    hidden |= here[:, None] - torch.arange(length, device=out.device) >= c["window"]
                for r in range(e * g, (e + 1) * g):
                    x = s["q"][at + t:at + t + here.numel(), r].double() @ keys.T / math.sqrt(d)
                    if c["softcap"]:
                        x = torch.tanh(x / c["softcap"]) * c["softcap"]
                    x[hidden] = float("-inf")
                    z = torch.logsumexp(x, -1)
                    lse[at + t:at + t + here.numel(), r] = z
                    out[at + t:at + t + here.numel(), r] = torch.exp(x - z[:, None]) @ values
        at += n
    return {"out": out, "lse": lse}
