"""What the attention operators of this package are measured on: causal attention over whole prompts with
its gradient, appending to a paged cache with the rotation of positions, and one token's attention over that
cache.

``run`` computes each case in its plain form (elementary torch operations in 32 bits, angles in 64, rounded
once at the end), or, where ``own`` is set, through ``state_space_sequence_m3_amd.m3attn``.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


def _io(case):
    return torch.bfloat16 if case["io"] == BF16 else torch.float32


def _es(case):
    return 2 if case["io"] == BF16 else 4


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt of a 4096 wide layer: launch latency
        dict(name="prompt b1 l64", op="prompt", io=BF16, batch=1, seqlen=64, heads=32, kv=8, dim=128, packed=0,
             fused=True),
        # prompts at the layer core's ordinary prefill and training shape
        dict(name="prompt b8 l2048", op="prompt", io=BF16, batch=8, seqlen=2048, heads=32, kv=8, dim=128, packed=0,
             fused=True),
        # one long prompt, heads of 64
        dict(name="prompt b1 l8192", op="prompt", io=BF16, batch=1, seqlen=8192, heads=32, kv=4, dim=64, packed=0,
             fused=False),
        # a packed batch of prompts of very different lengths (one empty, one of one token), odd head width
        dict(name="prompt packed f32", op="prompt", io=F32, batch=13, seqlen=701, heads=6, kv=2, dim=80, packed=5,
             fused=False),
        # a training step (forward and backward) at the ordinary shape
        dict(name="train b8 l2048", op="train", io=BF16, batch=8, seqlen=2048, heads=32, kv=8, dim=128, packed=0,
             fused=True),
        # the same over packed documents in fp32
        dict(name="train packed f32", op="train", io=F32, batch=9, seqlen=1100, heads=12, kv=4, dim=96, packed=3,
             fused=True),
        # decoding: one new token for each of 64 sequences
        dict(name="append b64", op="append", io=BF16, batch=64, seqlen=1, heads=32, kv=8, dim=128, packed=0, rot=128,
             halves=False, page=64, past=1000),
        # prompts enter the cache
        dict(name="append b8 l2048", op="append", io=BF16, batch=8, seqlen=2048, heads=32, kv=8, dim=128, packed=0,
             rot=128, halves=True, page=64, past=0),
        # packed chunks of prompts behind what is cached already; a part of each head is rotated, odd pages
        dict(name="append packed f32", op="append", io=F32, batch=9, seqlen=300, heads=6, kv=2, dim=80, packed=4, rot=32,
             halves=False, page=24, past=20000),
        # decoding one sequence behind a long context
        dict(name="step b1 l32768", op="step", io=BF16, batch=1, longest=32768, heads=32, kv=8, dim=128, page=64, mix=0),
        # decoding a batch of contexts of very different lengths
        dict(name="step b64 l8192", op="step", io=BF16, batch=64, longest=8192, heads=32, kv=8, dim=128, page=64, mix=7),
        # few heads to a group, odd widths and pages
        dict(name="step f32 b5", op="step", io=F32, batch=5, longest=1501, heads=6, kv=2, dim=80, page=24, mix=3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "append", "step", "step"])
    io = rng.choice([BF16, BF16, F32])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 64, 128, 32, 40, 72, 80, 96, 112])
    if op in ("prompt", "train"):
        seqlen = _spread(rng, 1, 8192)
        # rows times keys of all heads: what the scores of the plain form take
        most = (400_000_000 if op == "train" else 800_000_000) // (2 if io == F32 else 1)
        while heads * seqlen * seqlen > most:
            seqlen = seqlen * 2 // 3
        batch = max(1, min(_spread(rng, 1, 32), most // (heads * seqlen * seqlen), 60_000_000 // (heads * seqlen * dim)))
        return dict(op=op, io=io, batch=batch, seqlen=seqlen, heads=heads, kv=kv, dim=dim,
                    packed=rng.randrange(1, 1000) if rng.random() < 0.5 else 0, fused=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128, 256, 1, 24, 100])
    if op == "append":
        seqlen = rng.choice([1, _spread(rng, 1, 4096)])
        batch = max(1, min(_spread(rng, 1, 128), 15_000_000 // (heads * seqlen * dim)))
        past = _spread(rng, 1, 30000)
        past = min(past, 60_000_000 // (batch * kv * dim))
        return dict(op=op, io=io, batch=batch, seqlen=seqlen, heads=heads, kv=kv, dim=dim,
                    packed=rng.randrange(1, 1000) if rng.random() < 0.4 and seqlen > 1 else 0,
                    rot=rng.choice([dim, dim, dim, 32, 0]), halves=rng.random() < 0.5, page=page, past=past)
    longest = _spread(rng, 1, 60000)
    batch = max(1, min(_spread(rng, 1, 128), 110_000_000 // (longest * kv * dim)))
    return dict(op=op, io=io, batch=batch, longest=longest, heads=heads, kv=kv, dim=dim, page=page,
                mix=rng.randrange(0, 1000))


# ---------------------------------------------------------------------------------------- sizes

def _lens(case):
    """Tokens of each sequence: equal ones, or (packed) anything from none up to seqlen."""
    b, longest = case["batch"], case["seqlen"]
    if not case["packed"]:
        return [longest] * b
    rng = random.Random(case["packed"])
    lens = [rng.randint(0, longest) for _ in range(b)]
    if b >= 4:
        lens[1], lens[b - 2], lens[b - 1] = 0, 1, longest
    lens[0] = max(1, lens[0])
    return lens


def _contexts(case):
    """Cached tokens of each sequence of a decoding batch: equal ones (mix 0), or anything up to the longest."""
    b, longest = case["batch"], case["longest"]
    if not case["mix"]:
        return [longest] * b
    rng = random.Random(case["mix"])
    lens = [rng.randint(1, longest) for _ in range(b)]
    lens[-1] = longest
    if b >= 4:
        lens[1] = 0
    return lens


def _pasts(case):
    """Tokens cached before the new ones."""
    rng = random.Random(case["past"] + 1)
    return [rng.randint(case["past"] // 2, case["past"]) for _ in range(case["batch"])]


# ---------------------------------------------------------------------------------------- inputs

def _cache(case, totals, g):
    """Caches whose pages lie in no order, and the table of them."""
    page, dev = case["page"], "cuda"
    need = [-(-n // page) for n in totals]
    pages = max(1, sum(need))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(totals), max(1, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (pages, case["kv"], page, case["dim"])
    k = torch.randn(shape, generator=g, device=dev).to(_io(case))
    v = torch.randn(shape, generator=g, device=dev).to(_io(case))
    return k, v, table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, io = case["op"], _io(case)
    hq, hk, d = case["heads"], case["kv"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(io)

    if op == "step":
        lens = _contexts(case)
        k, v, table = _cache(case, lens, g)
        return {"case": case, "q": normal(len(lens), hq, d), "k_cache": k, "v_cache": v, "table": table,
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    lens = _lens(case)
    t, b, longest = sum(lens), len(lens), max(lens)
    # queries, keys and values are slices of one projection, or tensors of their own
    proj = normal(t, hq + 2 * hk, d)
    q, k, v = proj.split([hq, hk, hk], 1)
    if op == "append" or not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    length = torch.tensor(lens)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), length.cumsum(0)])
    s = {"case": case}
    if op == "append":
        totals = [p + n for p, n in zip(_pasts(case), lens)]
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, totals, g)
        s["lens"] = torch.tensor(totals, dtype=torch.int32, device="cuda")
        rot = case["rot"]
        s["inv_freq"] = None
        if rot:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
        # the sequence and the place in it of every token
        s["seq"] = torch.repeat_interleave(torch.arange(b), length).cuda()
        s["place"] = (torch.arange(t) - cu[:-1].repeat_interleave(length)).cuda()
        s["new"] = length.cuda()
    else:
        # rows of the batch padded to [b, longest], and back
        place = torch.arange(longest).unsqueeze(0)
        s["real"] = (place < length.unsqueeze(1)).reshape(-1).nonzero().squeeze(1).cuda() if case["packed"] else None
        s["scale"], s["b"], s["longest"] = 1.0 / math.sqrt(d), b, longest
        if op == "train":
            s["do"] = normal(t, hq, d)
            if not case["packed"]:
                s["do"] = s["do"].unflatten(0, (b, longest))
    if not case["packed"]:
        q, k, v = (x.unflatten(0, (b, longest)) for x in (q, k, v))
    s.update(q=q, k=k, v=v, cu=cu.to(torch.int32).cuda() if case["packed"] else None)
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _padded(s, x):
    """[b, H, L, D] in 32 bits of rows of heads, zero behind each sequence's end."""
    h, d = x.shape[-2:]
    x = x.float()
    if s["real"] is not None:
        rows = torch.zeros(s["b"] * s["longest"], h, d, device=x.device)
        rows[s["real"]] = x
        x = rows.view(s["b"], s["longest"], h, d)
    return x.transpose(1, 2)


def _rows(s, x, like):
    """The way back, rounded."""
    x = x.transpose(1, 2)
    if s["real"] is not None:
        x = x.reshape(-1, *x.shape[2:])[s["real"]]
    return x.to(like.dtype).contiguous()


def _plain_prompt(s, train):
    b, n, scale = s["b"], s["longest"], s["scale"]
    hq, hk, d = s["case"]["heads"], s["case"]["kv"], s["case"]["dim"]
    group = hq // hk
    # the rows of a group's query heads, one head after the other, meet the keys of their shared head
    q = _padded(s, s["q"]).reshape(b, hk, group * n, d)
    k, v = _padded(s, s["k"]), _padded(s, s["v"])
    row = torch.arange(n, device=q.device)
    hidden = (row.unsqueeze(0) > row.unsqueeze(1)).repeat(group, 1)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(scale).masked_fill_(hidden, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p, v)
    out = {"o": _rows(s, o.view(b, hq, n, d), s["q"])}
    if not train:
        return out
    do = _padded(s, s["do"]).reshape(b, hk, group * n, d)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    out["dq"] = _rows(s, torch.matmul(ds, k).view(b, hq, n, d), s["q"])
    out["dk"] = _rows(s, torch.matmul(ds.transpose(2, 3), q), s["k"])
    out["dv"] = _rows(s, torch.matmul(p.transpose(2, 3), do), s["v"])
    return out


def _turned(x, cos, sin, halves):
    """x [T, H, D] with its first pairs rotated."""
    rot = 2 * cos.shape[-1]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    y = x.float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if halves else (y[..., 0:rot:2], y[..., 1:rot:2])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    q, k, v = s["q"], s["k"], s["v"]
    shape = q.shape
    q, k, v = (x.reshape(-1, *x.shape[-2:]) for x in (q, k, v))
    at = s["lens"][s["seq"]] - s["new"][s["seq"]] + s["place"]
    if s["inv_freq"] is not None:
        angle = at.double().unsqueeze(1) * s["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        q, k = _turned(q, cos, sin, c["halves"]), _turned(k, cos, sin, c["halves"])
    to = s["table"][s["seq"], at // page].long()
    s["k_cache"][to, :, at % page] = k
    s["v_cache"][to, :, at % page] = v
    return {"q": q.view(shape), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_step(s):
    c, q = s["case"], s["q"]
    b, hq, d = q.shape
    hk, page, table = c["kv"], c["page"], s["table"]
    n = table.shape[1] * page
    # [b, kv, n, D]: each sequence's pages one after another
    k = s["k_cache"][table.long()].transpose(1, 2).reshape(b, hk, n, d).float()
    v = s["v_cache"][table.long()].transpose(1, 2).reshape(b, hk, n, d).float()
    gone = torch.arange(n, device=q.device) >= s["lens"].unsqueeze(1)
    p = torch.matmul(q.float().view(b, hk, hq // hk, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    p = p.masked_fill_(gone[:, None, None, :], -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = (p - top).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"o": o.view(b, hq, d).to(q.dtype)}


# ---------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "append":
        return _plain_append(s)
    return _plain_step(s) if op == "step" else _plain_prompt(s, op == "train")


def _own(s, op):
    from state_space_sequence_m3_amd import m3attn
    if op == "step":
        return {"o": m3attn.m3_attention_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])}
    if op == "append":
        q = m3attn.m3_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], q=s["q"],
                                   inv_freq=s["inv_freq"], halves=s["case"]["halves"], cu_seqlens=s["cu"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "prompt":
        return {"o": m3attn.m3_attention(s["q"], s["k"], s["v"], s["cu"])}
    o, lse = m3attn.m3_attention(s["q"], s["k"], s["v"], s["cu"], save_lse=True)
    d = m3attn.m3_attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu"])
    return {"o": o, "dq": d["q"], "dk": d["k"], "dv": d["v"]}


# ---------------------------------------------------------------------------------------- floors

def work(case):
    """Inputs read once, outputs written once, and the products that a causal mask leaves."""
    op, es, hq, hk, d = case["op"], _es(case), case["heads"], case["kv"], case["dim"]
    if op == "step":
        n, b = sum(_contexts(case)), case["batch"]
        return {"bytes": es * d * (2 * n * hk + 2 * b * hq), "flops": 4 * n * hq * d}
    lens = _lens(case)
    t = sum(lens)
    if op == "append":
        return {"bytes": es * t * d * 2 * (hq + 2 * hk), "flops": 3 * t * d * (hq + hk)}
    pairs = sum(n * (n + 1) // 2 for n in lens)
    if op == "prompt":
        return {"bytes": es * t * d * (2 * hq + 2 * hk), "flops": 4 * pairs * hq * d}
    return {"bytes": es * t * d * (4 * hq + 4 * hk), "flops": 14 * pairs * hq * d}


# ---------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    op, hq, hk, d = case["op"], case["heads"], case["kv"], case["dim"]
    group, scale = hq // hk, d ** -0.5
    if op == "step":
        o = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device="cuda")
        for i, n in enumerate(_contexts(case)):
            if n == 0:
                continue
            pages = s["table"][i, :-(-n // case["page"])].long()
            k = s["k_cache"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double()
            v = s["v_cache"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double()
            for h in range(hq):
                w = torch.softmax((k[h // group] @ s["q"][i, h].double()) * scale, 0)
                o[i, h] = w @ v[h // group]
        return {"o": o}
    lens = _lens(case)
    starts = [sum(lens[:i]) for i in range(len(lens))]
    q, k, v = (s[x].flatten(0, -3).double() for x in "qkv")
    if op == "append":
        return _exact_append(case, s, lens, starts, q, k, v)
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = s["do"].flatten(0, -3).double() if op == "train" else None
    for a, n in zip(starts, lens):
        part = slice(a, a + n)
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(hq):
            j = h // group
            z = (q[part, h] @ k[part, j].T) * scale
            w = torch.softmax(torch.where(seen, z, -math.inf), 1)
            o[part, h] = w @ v[part, j]
            if op == "train":
                dw = do[part, h] @ v[part, j].T
                dz = w * (dw - (w * dw).sum(1, keepdim=True))
                dv[part, j] += w.T @ do[part, h]
                dq[part, h] = scale * (dz @ k[part, j])
                dk[part, j] += scale * (dz.T @ q[part, h])
    out = {"o": o.view(s["q"].shape)}
    if op == "train":
        out.update(dq=dq.view(s["q"].shape), dk=dk.view(s["k"].shape), dv=dv.view(s["v"].shape))
    return out


def _exact_append(case, s, lens, starts, q, k, v):
    """Pairs as complex numbers, turned by e^(i angle)."""
    page, rot = case["page"], case["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    totals = s["lens"].tolist()
    for i, (a, n) in enumerate(zip(starts, lens)):
        if n == 0:
            continue
        at = torch.arange(totals[i] - n, totals[i], device="cuda")
        if rot:
            angle = torch.outer(at.double(), s["inv_freq"].double())
            turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
            for x in (q, k):
                y = x[a:a + n, :, :rot]
                pairs = y.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["halves"] else y.unflatten(-1, (rot // 2, 2))
                z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                x[a:a + n, :, :rot] = (z.transpose(-1, -2) if case["halves"] else z).flatten(-2)
        to = s["table"][i].long()[at // page]
        kc[to, :, at % page] = k[a:a + n]
        vc[to, :, at % page] = v[a:a + n]
    return {"q": q.view(s["q"].shape), "k_cache": kc, "v_cache": vc}
