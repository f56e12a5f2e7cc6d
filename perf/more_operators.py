"""Serving a latent cache that is held in 8 bits, shared between sequences and searched by beams: operators and the
cases they are timed on.

Four things a serving step needs around the paged latent cache (a row of 512 latent values and 64 rotary ones per token):

  append8   new rows, quantised as they are written (512 e4m3 values, a power-of-two scale for each 32 of them, 64
            rotary values of 16 bits: 656 bytes in place of 1152), the queries' rotary part, and the new rows read back
  read8     whole contexts of an 8-bit cache as 16-bit rows, one sequence behind the other
  decode8   absorbed attention of single or chained tokens over an 8-bit cache
  shared    absorbed attention of a batch whose groups of sequences share a long prefix, attended once for a group
  select    beam search: the best continuations over all beams and the vocabulary
  reorder   beam search: the cache rows and block tables of the chosen beams

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the library's calls (``serve.Serve``).
"""
import math
import random

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
GROUP = 32                                   # latent values that share a scale
ROW8 = LATENT + 2 * ROPE + LATENT // GROUP   # bytes: e4m3 values, rotary values, scales
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LEAST = {"bf16": -110, "f16": -15}           # the smallest scale's exponent: every value is one of the 16-bit type


def listed():
    return [
        # One decode step of 64 sequences: their rows into the cache and 64 heads' rotary queries; latency counts.
        dict(name="append8_64", op="append8", type="bf16", seqs=64, nodes=1, heads=64, short=1, long=12000, mix=1, page=64, interleaved=True),
        # Prompt chunks of 512 tokens of 16 sequences, read back for their expanded attention: bandwidth counts.
        dict(name="append8_8192", op="append8", type="f16", seqs=16, nodes=512, heads=64, short=512, long=8000, mix=2, page=64, interleaved=False),
        # The earlier context of eight prompts whose next chunk goes through expanded attention.
        dict(name="read8_8x_ragged", op="read8", type="bf16", seqs=8, short=33, long=1023, mix=3, page=16),
        # Sixteen long contexts: bound by bandwidth.
        dict(name="read8_16x32k", op="read8", type="f16", seqs=16, short=8000, long=32767, mix=4, page=64),
        # One sequence at a 4096-token context, one token: where splitting the context counts.
        dict(name="decode8_1x4k", op="decode8", type="bf16", heads=64, seqs=1, nodes=1, short=4096, long=4096, mix=1, page=64),
        # 64 sequences of 600 to 12000 tokens, one token each: the ordinary serving batch, bound by the cache's bytes.
        dict(name="decode8_64x12k", op="decode8", type="f16", heads=64, seqs=64, nodes=1, short=600, long=12000, mix=2, page=64),
        # Eight beams of one prompt, 16 heads, over an 8-bit cache: the smallest call that shares.
        dict(name="shared_1x8_4k", op="shared", type="bf16", bits=8, heads=16, groups=1, seqs=8, nodes=1, prefix=4096, short=1, long=63, mix=5, page=64),
        # 64 requests behind one 32,000-token document, 16 heads, over a 16-bit cache.
        dict(name="shared_1x64_32k", op="shared", type="f16", bits=16, heads=16, groups=1, seqs=64, nodes=1, prefix=32000, short=20, long=2000, mix=6, page=64),
        # One prompt's four beams.
        dict(name="select_1x4", op="select", type="f32", groups=1, beams=4, vocab=32000, keep=8),
        # 32 prompts of eight beams over a large odd vocabulary: bound by the logits' bytes.
        dict(name="select_32x8", op="select", type="f32", groups=32, beams=8, vocab=151643, keep=16),
        # One prompt's four beams, one layer's cache of 16 bits.
        dict(name="reorder_1x4", op="reorder", type="bf16", bits=16, groups=1, beams=4, layers=1, short=1000, long=1000, mix=9, page=16),
        # 32 prompts of eight beams, twelve layers' caches of 8 bits.
        dict(name="reorder_32x8x12", op="reorder", type="bf16", bits=8, groups=32, beams=8, layers=12, short=40, long=900, mix=10, page=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["append8", "read8", "decode8", "decode8", "shared", "shared", "select", "reorder"])
    half, mix, page = rng.choice(["bf16", "f16"]), rng.randrange(1000), rng.choice([1, 16, 32, 64, 256])
    if op == "append8":
        seqs = log(1, 64)
        nodes = log(1, 8192 // seqs)
        return dict(op=op, type=half, seqs=seqs, nodes=nodes, heads=rng.choice([1, 5, 16, 32, 64]), short=nodes, long=log(nodes, max(nodes, 260000 // seqs if seqs > 8 else 32000)), mix=mix, page=page,
                    interleaved=rng.random() < 0.5)
    if op == "read8":
        seqs = log(1, 64)
        long = log(1, min(32767, 260000 // seqs))
        return dict(op=op, type=half, seqs=seqs, short=max(1, long // rng.choice([1, 4, 30])), long=long, mix=mix, page=page)
    if op == "decode8":
        heads, nodes, seqs = rng.choice([1, 6, 16, 32, 64, 128]), rng.choice([1, 1, 2, 4, 7]), log(1, 64)
        most = min(131071, 500000 // seqs, int(4.9e7 / (heads * nodes * seqs)))
        long = log(max(nodes + 1, 70), max(nodes + 2, 71, most))
        return dict(op=op, type=half, heads=heads, seqs=seqs, nodes=nodes, short=max(nodes, long // rng.choice([1, 3, 20])), long=long, mix=mix, page=max(page, 16))
    if op == "shared":
        heads, nodes, groups = rng.choice([1, 6, 16, 32, 64]), rng.choice([1, 1, 1, 3]), log(1, 8)
        seqs = log(2, 64 // groups)
        rows = heads * nodes * groups * seqs
        prefix = log(64, min(32000, 250000 // groups, int(3.2e7 / rows)))
        long = log(nodes, max(nodes, min(2000, int(1e7 / rows))))
        return dict(op=op, type=half, bits=rng.choice([8, 16]), heads=heads, groups=groups, seqs=seqs, nodes=nodes, prefix=prefix, short=max(nodes, long // rng.choice([1, 10])), long=long, mix=mix,
                    page=max(page, 16))
    if op == "select":
        beams = rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), groups=log(1, 32), beams=beams, vocab=log(1000, 151643), keep=rng.choice([beams, 2 * beams, 2 * beams + 1]))
    return dict(op=op, type=half, bits=rng.choice([8, 16]), groups=log(1, 32), beams=rng.choice([2, 3, 4, 8]), layers=log(1, 6), short=rng.choice([20, 64]), long=log(64, 900), mix=mix,
                page=rng.choice([16, 64]))


# ---- sizes that a case fixes ---------------------------------------------

def count(case):
    """Sequences of a case."""
    return case.get("groups", 1) * case.get("beams", case.get("seqs", 1))


def lengths(case):
    """One length per sequence, spread over the logarithm of short..long; the first is the longest.  Of a shared case: what
    lies behind the prefix.  The beams of a prompt are of one length."""
    r, lo, hi = random.Random(case["mix"]), case["short"], case["long"]
    n = case["groups"] if case["op"] == "reorder" else count(case)
    got = [hi] + [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(n - 1)]
    return [x for x in got for _ in range(case["beams"])] if case["op"] == "reorder" else got


def parents_of(case):
    """The beam that each place of a group continues: good ones are continued by several, others by none."""
    r = random.Random(case["mix"] + 1)
    return np.array([[r.randrange(case["beams"]) for _ in range(case["beams"])] for _ in range(case["groups"])])


def ceil_div(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "append8":
        t, h = case["seqs"] * case["nodes"], case["heads"]
        return {"bytes": t * (ROW * 2 + ROW8 + ROW * 2) + 2 * t * h * ROPE * 2 + t * (12 + 2 * ROPE * 4 // 2) + LATENT * 2, "flops": t * (8 * LATENT + 3 * ROPE * (h + 1))}
    if op == "read8":
        return {"bytes": sum(lengths(case)) * (ROW8 + ROW * 2), "flops": sum(lengths(case)) * LATENT}
    if op == "decode8":
        n, h = case["nodes"], case["heads"]
        seen = sum(n * (ln - n) + n * (n + 1) // 2 for ln in lengths(case))
        rows = case["seqs"] * n * h
        return {"bytes": sum(lengths(case)) * ROW8 + rows * (ROW + LATENT) * 2 + rows * 4, "flops": 2 * h * seen * (ROW + LATENT)}
    if op == "shared":
        n, h, own_rows = case["nodes"], case["heads"], sum(lengths(case))
        seen = sum(n * (case["prefix"] + ln - n) + n * (n + 1) // 2 for ln in lengths(case))
        rows = count(case) * n * h
        return {"bytes": (case["groups"] * case["prefix"] + own_rows) * (ROW8 if case["bits"] == 8 else ROW * 2) + rows * (ROW + LATENT) * 2 + rows * 4, "flops": 2 * h * seen * (ROW + LATENT)}
    if op == "select":
        rows = case["groups"] * case["beams"]
        return {"bytes": rows * case["vocab"] * (4 if case["type"] == "f32" else 2) + rows * 4 + case["groups"] * case["keep"] * 12, "flops": rows * case["vocab"] * 4}
    ln, w, page = lengths(case), case["beams"], case["page"]
    moved = sum((w - len(set(p))) * (ln[i * w] % page) for i, p in enumerate(parents_of(case).tolist()))
    table = count(case) * ceil_div(case["long"] + 1, page) * 4 * 2
    return {"bytes": 2 * moved * case["layers"] * (ROW8 if case["bits"] == 8 else ROW * 2) + table, "flops": 0}


# ---- inputs ---------------------------------------------------------------

def prepare(case, seed):
    dev, dt = "cuda:0", TYPES[case["type"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def ints(a, kind=torch.int32):
        return torch.as_tensor(np.ascontiguousarray(a)).to(dev, kind)

    def paged(each):
        """A block table of so many pages a sequence, which lie anywhere, and the pages in all."""
        order, at = r.permutation(sum(each) + 2), 0
        table = np.full((len(each), max(each)), -1)
        for i, e in enumerate(each):
            table[i, :e] = order[at:at + e]
            at += e
        return table, len(order)

    def rows(*lead, bits=8):
        """Cached rows of normed latents: values of about one."""
        if bits == 16:
            return normal(*lead, ROW)
        return packed(torch.randn(*lead, LATENT, generator=g, device=dev), normal(*lead, ROPE), case["type"])

    s = dict(case)
    op, page = case["op"], case.get("page")
    if op == "select":
        b, w, vocab = case["groups"], case["beams"], case["vocab"]
        s.update(logits=(3 * torch.randn(b * w, vocab, generator=g, device=dev)).to(dt),
                 scores=-3 * torch.randn(b, w, generator=g, device=dev).abs())    # of beams that are near each other
        if own:
            s["serve"] = handle(case, b * w, b * w)
        return s
    ln = lengths(case)
    b = count(case)
    if op == "append8":
        n, most = case["nodes"], 32768
        table, pages = paged([ceil_div(x, page) for x in ln])
        pos = np.concatenate([np.arange(x - n, x) for x in ln])
        seq = np.repeat(np.arange(b), n)
        angle = torch.arange(most, device=dev, dtype=torch.float32)[:, None] * (10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float32) / ROPE))
        s.update(c=normal(b * n, ROW), weight=(1 + 0.1 * torch.randn(LATENT, generator=g, device=dev)).to(dt), cos=angle.cos(), sin=angle.sin(), q_pe=normal(b * n, case["heads"], ROPE),
                 positions=ints(pos), slots=ints(table[seq, pos // page] * page + pos % page, torch.int64), block_table=ints(table), first=ints(np.array(ln) - n),
                 k_start=ints(np.arange(b + 1) * n), cache=torch.zeros(pages, page, ROW8, device=dev, dtype=torch.uint8))
        if own:
            s["serve"] = handle(case, b * n, b)
    elif op == "read8":
        table, pages = paged([ceil_div(x, page) for x in ln])
        s.update(cache=rows(pages, page), block_table=ints(table), k_start=ints(np.concatenate([[0], np.cumsum(ln)])), total=sum(ln))
        if own:
            s["serve"] = handle(case, 1, b)
    elif op == "decode8":
        n = case["nodes"]
        table, pages = paged([ceil_div(x, page) for x in ln])
        s.update(cache=rows(pages, page), block_table=ints(table), q_start=ints(np.arange(b + 1) * n), kv_len=ints(ln), q_lat=normal(b * n, case["heads"], LATENT),
                 q_pe=normal(b * n, case["heads"], ROPE), scale=1 / 16.0)
        if own:
            s["serve"] = handle(case, b * n, b)
            s["serve"].plan(s["q_start"], s["kv_len"])
    elif op == "shared":
        n, w, prefix = case["nodes"], case["seqs"], case["prefix"]
        whole, part = prefix // page, prefix % page
        every = [ceil_div(prefix + x, page) for x in ln]
        mine, pages = paged([e if i % w == 0 else e - whole for i, e in enumerate(every)])
        table = np.full((b, max(every)), -1)
        for i, e in enumerate(every):        # the first of a group holds the prefix's whole pages for all of it
            first = i - i % w
            table[i, :whole] = mine[first, :whole]
            table[i, whole:e] = mine[i, whole:e] if i == first else mine[i, :e - whole]
        cache = rows(pages, page, bits=case["bits"])
        if part:                             # the page that the prefix ends in is each sequence's own
            at = ints(table[:, whole], torch.int64)
            cache[at, :part] = cache[at.view(-1, w)[:, :1].expand(-1, w).reshape(-1), :part]
        s.update(cache=cache, block_table=ints(table), q_start=ints(np.arange(b + 1) * n), kv_len=ints(np.array(ln) + prefix), group_start=ints(np.arange(case["groups"] + 1) * w),
                 prefix_len=ints(np.full(case["groups"], prefix)), q_lat=normal(b * n, case["heads"], LATENT), q_pe=normal(b * n, case["heads"], ROPE), scale=1 / 16.0)
        if own:
            s["serve"] = handle(case, b * n, b)
            s["serve"].plan(s["q_start"], s["kv_len"], group_start=s["group_start"], prefix_len=s["prefix_len"])
    else:
        w = case["beams"]
        every = [ceil_div(x + 1, page) for x in ln]           # room for the next token
        mine, pages = paged([e if i % w == 0 else e - x // page for i, (e, x) in enumerate(zip(every, ln))])
        table = np.full((b, max(every)), -1)
        for i, (e, x) in enumerate(zip(every, ln)):           # the whole pages of a prompt are those of all its beams
            first, whole = i - i % w, x // page
            table[i, :whole] = mine[first, :whole]
            table[i, whole:e] = mine[i, whole:e] if i == first else mine[i, :e - whole]
        s.update(cache=rows(case["layers"], pages, page, bits=case["bits"]), block_table=ints(table), kv_len=ints(ln), parents=ints(parents_of(case)))
        if own:
            s["serve"] = handle(case, b, b)
    return s


def handle(case, tokens, seqs):
    """The library's handle, as a program makes it once for its batches."""
    from int4_routed_expert_layer_amd.serve import Serve

    return Serve(n_heads=case.get("heads", 64), max_tokens=tokens, max_seqs=seqs, page_size=case.get("page", 64), dtype=case["type"] if case["type"] != "f32" else "bf16")


# ---- rows of 8 bits --------------------------------------------------------

def two_to(k):
    """2^k in fp32, of whole numbers."""
    return ((k + 127) << 23).view(torch.float32)


def packed(latent, rope, kind):
    """Rows of bytes: the smallest power of two that brings a group's values to 448 or below is its scale."""
    y = latent.float().unflatten(-1, (LATENT // GROUP, GROUP))
    most = y.abs().amax(-1).view(torch.int32)
    k = ((most >> 23) - 127 - 8 + ((most & 0x7FFFFF) > 0x600000).int()).clamp(min=LEAST[kind])   # 448 is 1.75 times 2^8
    q = (y * two_to(-k)[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return torch.cat([q.view(torch.uint8), rope.view(torch.uint8), (k + 127).to(torch.uint8)], -1)


def unpacked(rows, dt):
    """Rows of bytes as 576 values in 32 bits."""
    q = rows[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (LATENT // GROUP, GROUP))
    by = two_to(rows[..., LATENT + 2 * ROPE:].int() - 127)
    return torch.cat([(q * by[..., None]).flatten(-2), rows[..., LATENT:LATENT + 2 * ROPE].contiguous().view(dt).float()], -1)


def values(rows, dt):
    return unpacked(rows, dt) if rows.dtype == torch.uint8 else rows.float()


# ---- one pass -------------------------------------------------------------

def run(s):
    return (OWN if own else PLAIN)[s["op"]](s)


def own_append8(s):
    q = s["serve"].append(s["c"], s["weight"], 1e-6, s["cos"], s["sin"], s["positions"], s["slots"], s["cache"], q_pe=s["q_pe"], interleaved=s["interleaved"])
    return {"rows": s["serve"].read(s["cache"], s["block_table"], s["k_start"], n_rows=s["c"].shape[0], first=s["first"]), "q_pe": q}


def own_read8(s):
    return {"rows": s["serve"].read(s["cache"], s["block_table"], s["k_start"], n_rows=s["total"])}


def own_decode(s):
    out, lse = s["serve"].decode(s["q_lat"], s["q_pe"], s["cache"], s["block_table"], s["scale"], return_lse=True)
    return {"out": out, "lse": lse}


def own_select(s):
    scores, parents, tokens = s["serve"].beam_select(s["logits"], s["scores"], s["keep"])
    return {"scores": scores, "parents": parents, "tokens": tokens}


def own_reorder(s):
    return {"table": s["serve"].beam_reorder(s["cache"], s["block_table"], s["kv_len"], s["parents"]), "cache": s["cache"]}


def plain_append8(s):
    c, dt = s["c"].float(), s["c"].dtype
    lat = c[:, :LATENT]
    lat = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    cache = s["cache"].view(-1, ROW8)
    cache[s["slots"]] = packed(lat, rotate(c[:, LATENT:], cos, sin, s["interleaved"]).to(dt), s["type"])
    return {"rows": unpacked(cache[rows_of(s, s["first"])], dt).to(dt), "q_pe": rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(dt)}


def rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def rows_of(s, first, total=None):
    """The cache rows of positions first[b] .. of each sequence, one sequence behind the other."""
    start = s["k_start"].long()
    t = torch.arange(s["c"].shape[0] if total is None else total, device=start.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    pos = t - start[seq] + (0 if first is None else first.long()[seq])
    return s["block_table"].long()[seq, pos // s["page"]] * s["page"] + pos % s["page"]


def plain_read8(s):
    dt = TYPES[s["type"]]
    return {"rows": unpacked(s["cache"].view(-1, ROW8)[rows_of(s, None, s["total"])], dt).to(dt)}


def gathered(s, table, first, many):
    """Values of positions first .. first + many - 1 of every row of the table."""
    at = first + torch.arange(many, device=table.device)
    pages = table.long()[:, (at // s["page"]).clamp(max=table.shape[1] - 1)].clamp(min=0)
    return values(s["cache"].flatten(0, 1)[pages * s["page"] + at % s["page"]], s["q_lat"].dtype)


def plain_decode8(s):
    return attend(s, None, 0, s["long"], s["kv_len"].long())


def plain_shared(s):
    """The prefix's scores of all of a group's rows are one product, and its values summed by another."""
    prefix = gathered(s, s["block_table"][::s["seqs"]], 0, s["prefix"])
    return attend(s, prefix, s["prefix"], s["long"], s["kv_len"].long() - s["prefix"])


def attend(s, prefix, first, most, length):
    n, h, dt = s["nodes"], s["heads"], s["q_lat"].dtype
    b = s["block_table"].shape[0]
    kv = gathered(s, s["block_table"], first, most)
    q = torch.cat([s["q_lat"], s["q_pe"]], -1).float().view(b, n * h, ROW)
    score = torch.matmul(q, kv.transpose(1, 2).contiguous()).mul_(s["scale"]).view(b, n, h, most)
    at = torch.arange(most, device=q.device)
    node = at[None, None] - (length - n)[:, None, None]
    score.masked_fill_(~(node <= torch.arange(n, device=q.device)[None, :, None])[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if prefix is not None:
        g = s["groups"]
        before = torch.matmul(q.view(g, -1, ROW), prefix.transpose(1, 2).contiguous()).mul_(s["scale"])
        top = torch.maximum(top, before.amax(-1).view(b, n, h, 1))
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, n * h, most), kv[:, :, :LATENT].contiguous()).view(b, n, h, LATENT)
    if prefix is not None:
        p = before.sub_(top.view(g, -1, 1)).exp_()
        total = total + p.sum(-1).view(b, n, h, 1)
        out = out + torch.matmul(p, prefix[:, :, :LATENT].contiguous()).view(b, n, h, LATENT)
    return {"out": (out / total).view(b * n, h, LATENT).to(dt), "lse": (top + total.log()).view(b * n, h)}


def plain_select(s):
    """In 64 bits, where two beams' candidates are told apart; the lower beam, then the lower token, of equal ones."""
    b, w, vocab = s["groups"], s["beams"], s["vocab"]
    x = s["logits"].double()
    top = x.amax(1, keepdim=True)
    total = x - (top + (x - top).exp().sum(1, keepdim=True).log()) + s["scores"].double().view(-1, 1)
    best, at = torch.sort(total.view(b, w * vocab), dim=1, descending=True, stable=True)
    at = at[:, :s["keep"]]
    return {"scores": best[:, :s["keep"]].float(), "parents": (at // vocab).int(), "tokens": (at % vocab).int()}


def plain_reorder(s):
    """The first place that continues a beam keeps its last page; further ones get those of beams that nobody continues."""
    b, w, page = s["groups"], s["beams"], s["page"]
    parents, table = s["parents"].long(), s["block_table"].view(b, w, -1)
    here = torch.arange(w, device=table.device)
    same = parents[:, :, None] == parents[:, None]
    extra = (same & (here[None, :] < here[:, None])).any(2)                     # an earlier place has the same parent
    unused = ~(parents[:, :, None] == here).any(1)
    rank = extra.long().cumsum(1) - 1
    left = torch.argsort((~unused).long(), dim=1, stable=True)                  # the beams that nobody continues come first
    donor = torch.where(extra, left.gather(1, rank.clamp(min=0)), parents)
    whole = (s["kv_len"].view(b, w)[:, :1].long() // page)[:, :, None]
    cols = torch.arange(table.shape[2], device=table.device)
    group = torch.arange(b, device=table.device)[:, None]
    new = torch.where(cols < whole, table[group, parents], table[group, donor])
    last = whole.expand(b, w, 1).clamp(max=table.shape[2] - 1)
    src, dst = table[group, parents].gather(2, last)[..., 0].long(), table[group, donor].gather(2, last)[..., 0].long()
    part = (s["kv_len"].view(b, w) % page)[..., None]
    row = torch.arange(page, device=table.device)
    moved = extra[..., None] & (row < part)
    flat = s["cache"].view(s["layers"], -1, s["cache"].shape[-1])
    flat[:, (dst[..., None] * page + row)[moved]] = flat[:, (src[..., None] * page + row)[moved]]
    return {"table": new.reshape(b * w, -1), "cache": s["cache"]}


OWN = dict(append8=own_append8, read8=own_read8, decode8=own_decode, shared=own_decode, select=own_select, reorder=own_reorder)
PLAIN = dict(append8=plain_append8, read8=plain_read8, decode8=plain_decode8, shared=plain_shared, select=plain_select, reorder=plain_reorder)


# ---- the definitions in 64 bits -------------------------------------------

def e4m3_values():
    """The value of each byte: a sign, four bits of exponent (bias 7) and three of fraction; two bytes are NaN."""
    byte = np.arange(256)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((byte & 127) == 127, np.nan, v)
    return np.where(byte >= 128, -v, v)


def stored(cache, kind):
    """Rows of a cache as 64-bit values."""
    if cache.dtype != torch.uint8:
        return cache.double()
    table = torch.as_tensor(e4m3_values(), device=cache.device)
    by = torch.ldexp(torch.ones((), dtype=torch.float64, device=cache.device), cache[..., LATENT + 2 * ROPE:].int() - 127)
    latent = table[cache[..., :LATENT].long()] * by.repeat_interleave(GROUP, -1)
    return torch.cat([latent, cache[..., LATENT:LATENT + 2 * ROPE].contiguous().view(TYPES[kind]).double()], -1)


def quantised(x, kind):
    """Values of groups of 32 as the cache holds them: to the nearest multiple of an eighth of their own power of two, ties to
    even, in units of the group's scale; no finer than 2^-9 of it."""
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    fraction, exponent = torch.frexp(y.abs().amax(-1, keepdim=True))
    k = (exponent - 9 + (fraction > 0.875).to(exponent.dtype)).clamp(min=LEAST[kind])
    scale = torch.ldexp(torch.ones_like(fraction), k)
    z = y / scale
    step = torch.ldexp(torch.ones_like(z), (torch.frexp(z)[1] - 1).clamp(min=-6) - 3)
    return ((z / step).round() * step * scale).reshape(x.shape)


def exact(case, seed):
    global own
    own, was = False, own
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, kind = case["op"], case["type"]
    if op == "append8":
        c = s["c"].double()
        norm = c[:, :LATENT] / (c[:, :LATENT].square().mean(1, keepdim=True) + 1e-6).sqrt() * s["weight"].double()
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()]

        def turned(x, by):
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], ROPE // 2, 2).contiguous()) * by).flatten(-2)
            y = torch.complex(x[..., :ROPE // 2], x[..., ROPE // 2:]) * by
            return torch.cat([y.real, y.imag], -1)

        # every token is in the cache at its own slot, and read back in the order it came in
        return {"rows": torch.cat([quantised(norm, kind), turned(c[:, LATENT:].contiguous(), turn)], 1), "q_pe": turned(s["q_pe"].double(), turn[:, None])}
    if op == "read8":
        parts = []
        for i, ln in enumerate(lengths(case)):
            pages = s["block_table"][i, :ceil_div(ln, case["page"])].long()
            parts.append(stored(s["cache"][pages].reshape(-1, ROW8)[:ln], kind))
        return {"rows": torch.cat(parts)}
    if op == "select":
        x = s["logits"].double()
        logp = x - torch.logsumexp(x, 1, keepdim=True)
        total = (s["scores"].double()[..., None] + logp.view(case["groups"], case["beams"], -1)).flatten(1)
        return {"scores": torch.topk(total, case["keep"], dim=1).values, "parents": None, "tokens": None}
    if op == "reorder":
        if case["bits"] == 8:                # whole numbers alone
            return None
        cache, w, page = s["cache"].clone(), case["beams"], case["page"]
        for i, chosen in enumerate(parents_of(case).tolist()):
            ln, table = lengths(case)[i * w], s["block_table"][i * w:(i + 1) * w].tolist()
            left = [j for j in range(w) if j not in chosen]
            for j, p in enumerate(chosen):
                if p in chosen[:j]:
                    to = left.pop(0)
                    if ln % page:
                        cache[:, table[to][ln // page], :ln % page] = s["cache"][:, table[p][ln // page], :ln % page]
        return {"table": None, "cache": cache}
    outs, lses = [], []
    n, page, h, scale = case["nodes"], case["page"], case["heads"], s["scale"]
    for i, ln in enumerate(lengths(case)):
        ln += case.get("prefix", 0)
        kv = stored(s["cache"][s["block_table"][i, :ceil_div(ln, page)].long()].flatten(0, 1)[:ln], kind)
        q = torch.cat([s["q_lat"], s["q_pe"]], -1)[i * n:(i + 1) * n].double()
        see = torch.ones(n, ln, dtype=torch.bool, device=q.device).tril(ln - n)
        score = torch.where(see[:, None], (q.reshape(n * h, ROW) @ kv.t()).view(n, h, ln) * scale, -math.inf)
        lse = torch.logsumexp(score, -1)
        outs.append(((score - lse[..., None]).exp().view(n * h, ln) @ kv[:, :LATENT]).view(n, h, LATENT))
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
