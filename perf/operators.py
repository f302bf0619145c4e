"""What the 8-bit key/value cache's operators are measured on: the appending of keys and values
(with the position rotation) and the attention that reads them.

Each case is one pass of one operator.  `run` computes it either in its plain form (torch
operations in 32 bits, rounded once at the end) or, where `own` is true, through the package's
public functions.  `exact` computes it in 64 bits from the definition.

The cache holds, for every page, head and block of 32 tokens, one record of 64 * dim + 16 bytes:
the 32 x dim int8 key codes, the 32 x dim int8 value codes, the f32 key scale, the f32 value scale
and 8 reserved bytes.  A code c stands for the value c * scale.
"""
import math

import torch

own = False

BLOCK = 32  # tokens that share one scale per head


# ---------------------------------------------------------------------------------------- cases
def listed():
    """Head counts and sizes are those of the 7B GQA layer of this repository (28 query heads, 4
    key/value heads of 128, 3584 wide) unless a comment says otherwise."""
    return [
        # one user's next token, a short conversation, f32 as the quantized projections give it:
        # the smallest call, where latency counts
        dict(name="decode_one", op="attend", dtype="f32", seqs=1, new_lo=1, new_hi=1, len_lo=777, len_hi=777,
             heads=28, kv_heads=4, dim=128, page=64, window=0),
        # one user's next token at the far end of a very long document: one row of work per head,
        # so the long axis has to be shared out
        dict(name="decode_long", op="attend", dtype="bf16", seqs=1, new_lo=1, new_hi=1, len_lo=131069, len_hi=131069,
             heads=28, kv_heads=4, dim=128, page=64, window=0),
        # a full serving batch of ragged conversations (8 key/value heads): the largest decode
        dict(name="decode_full", op="attend", dtype="f16", seqs=64, new_lo=1, new_hi=1, len_lo=1000, len_hi=8191,
             heads=32, kv_heads=8, dim=128, page=128, window=0),
        # heads of 64 without sharing, a sliding window that leaves most of the cache unread
        dict(name="decode_window", op="attend", dtype="bf16", seqs=48, new_lo=1, new_hi=1, len_lo=90, len_hi=4001,
             heads=16, kv_heads=16, dim=64, page=32, window=1024),
        # drafted tokens checked together, a few rows per sequence
        dict(name="verify_draft", op="attend", dtype="bf16", seqs=8, new_lo=2, new_hi=5, len_lo=517, len_hi=3001,
             heads=28, kv_heads=4, dim=128, page=64, window=0),
        # a prompt of 2048 tokens, all new
        dict(name="prefill_prompt", op="attend", dtype="bf16", seqs=1, new_lo=2048, new_hi=2048, len_lo=2048,
             len_hi=2048, heads=28, kv_heads=4, dim=128, page=64, window=0),
        # prompts of odd lengths after shared beginnings, f32 as the quantized projections give them
        dict(name="prefill_f32", op="attend", dtype="f32", seqs=3, new_lo=131, new_hi=699, len_lo=700, len_hi=1501,
             heads=28, kv_heads=4, dim=128, page=64, window=0),
        # a chunk of a long document's prompt on top of what the cache holds: the largest
        dict(name="prefill_chunk", op="attend", dtype="f16", seqs=1, new_lo=1024, new_hi=1024, len_lo=32768,
             len_hi=32768, heads=32, kv_heads=8, dim=128, page=128, window=0),
        # one user's next token joins its block
        dict(name="append_one", op="append", dtype="f32", seqs=1, new_lo=1, new_hi=1, len_lo=778, len_hi=778, heads=28,
             kv_heads=4, dim=128, page=64, rotary=128, interleaved=False),
        # the next tokens of a full serving batch
        dict(name="append_batch", op="append", dtype="bf16", seqs=64, new_lo=1, new_hi=1, len_lo=1001, len_hi=8192,
             heads=32, kv_heads=8, dim=128, page=128, rotary=128, interleaved=False),
        # a prompt of 8192 tokens
        dict(name="append_prompt", op="append", dtype="bf16", seqs=1, new_lo=8192, new_hi=8192, len_lo=8192,
             len_hi=8192, heads=28, kv_heads=4, dim=128, page=64, rotary=128, interleaved=False),
        # prompts of odd lengths that begin inside a block, half of each head rotated, in adjacent pairs
        dict(name="append_ragged", op="append", dtype="f32", seqs=5, new_lo=33, new_hi=997, len_lo=1013, len_hi=3001,
             heads=16, kv_heads=16, dim=64, page=32, rotary=32, interleaved=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: decode, drafted tokens, prompts and appends over the ranges of the listed ones."""
    kind = rng.choice(["decode", "decode", "draft", "prompt", "prompt", "append", "append_prompt"])
    kv_heads, group = rng.choice([(4, 7), (8, 4), (16, 1), (2, 8), (1, 8), (4, 2), (6, 3)])
    c = dict(op="append" if kind.startswith("append") else "attend", dtype=rng.choice(["f32", "bf16", "f16"]),
             heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice([64, 128, 128, 128, 256]),
             page=rng.choice([32, 64, 128]))
    if kind in ("decode", "draft", "append"):
        c["seqs"] = _log(rng, 1, 64)
        # at most the largest listed batch's cache
        most = min(131072, 64 * 4600 * 8 * 128 // (c["seqs"] * c["kv_heads"] * c["dim"]))
        hi = _log(rng, 64, most)
        lo = max(16, int(hi * rng.uniform(0.1, 1.0)))
        new = 1 if kind != "draft" else rng.randint(2, 8)
        c.update(new_lo=1, new_hi=new, len_lo=lo, len_hi=hi)
    else:
        new = _log(rng, 16, 2048)
        c["seqs"] = rng.choice([1, 1, 2, 4])
        # new * len * heads * dim stays below the largest listed case's
        most = 1024 * 32768 * 32 * 128 // (new * c["heads"] * c["dim"] * c["seqs"])
        hi = new if rng.random() < 0.4 else new + _log(rng, 1, max(2, min(16384, most - new)))
        hi = max(new, min(hi, most))
        lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
        c.update(new_lo=max(1, int(new * rng.uniform(0.3, 1.0))), new_hi=new, len_lo=lo, len_hi=hi)
    if c["op"] == "append":
        c.update(rotary=rng.choice([c["dim"], c["dim"], c["dim"] // 2]), interleaved=rng.random() < 0.4)
    else:
        c["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    return c


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _spread(lo, hi, n, shift):
    """n whole numbers from lo to hi, hi the first of them, the others spread without an order."""
    return [hi] + [lo + int((hi - lo) * ((i * 0.6180339887 + shift) % 1.0)) for i in range(1, n)]


def _lengths(c):
    """(length with the new tokens, new tokens) of each sequence, from the case alone."""
    lens = _spread(c["len_lo"], c["len_hi"], c["seqs"], 0.31)
    news = _spread(c["new_lo"], c["new_hi"], c["seqs"], 0.77)
    return lens, [min(n, m) for n, m in zip(news, lens)]


def _first_key(pos, window):
    return max(0, pos - window + 1) if window else 0


def work(case):
    lens, news = _lengths(case)
    e = 4 if case["dtype"] == "f32" else 2
    H, KH, D = case["heads"], case["kv_heads"], case["dim"]
    T = sum(news)
    tables = 4 * (2 * len(lens) + sum((n + case["page"] - 1) // case["page"] for n in lens))
    if case["op"] == "append":
        old = sum((n - m) % BLOCK for n, m in zip(lens, news))  # older tokens of the blocks written to
        # keys, values and queries in, queries out, rotation tables; codes written, the older ones
        # read, the values of all of them out
        io = T * (2 * KH + 2 * H) * D * e + T * case["rotary"] * 4 + 2 * (T + old) * KH * D + (T + old) * 2 * KH * D * e
        return {"bytes": io + tables, "flops": 6 * T * (H + KH) * D}
    W = case["window"]
    keys = blocks = 0
    for n, m in zip(lens, news):
        first = _first_key(n - m, W)
        blocks += (n + BLOCK - 1) // BLOCK - first // BLOCK
        if W:
            keys += sum(min(p + 1, W) for p in range(n - m, n))
        else:
            keys += m * (n - m) + m * (m + 1) // 2
    return {"bytes": 2 * T * H * D * e + blocks * KH * (2 * BLOCK * D + 16) + tables, "flops": 4 * keys * H * D}


# ---------------------------------------------------------------------------------------- inputs
def _fill_codes(rec, dim, gen):
    """Codes as blocks of normal values have them: their largest value, near four deviations, at
    the last code."""
    flat = rec.view(-1, rec.shape[-1])
    step = max(1, (1 << 27) // (64 * dim))
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        x = torch.randn((part.shape[0], 64 * dim), device=rec.device, generator=gen)
        part[:, :64 * dim] = x.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    s = torch.rand((flat.shape[0], 2), device=rec.device, generator=gen).mul_(1.0).add_(0.5).mul_(1.0 / 32.0)
    flat[:, 64 * dim:64 * dim + 8] = s.view(torch.uint8)
    flat[:, 64 * dim + 8:] = 0


def _rotation(rows, rotary, device):
    """cos and sin of position * 10000^(-2i / rotary), f32 [rows, rotary / 2]."""
    freq = torch.pow(10000.0, -torch.arange(0, rotary, 2, device=device, dtype=torch.float64) / rotary)
    a = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * freq[None]
    return a.cos().float(), a.sin().float()


def _int32(v, device):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    """The cache with what earlier tokens left in it, the batch's tables, and the new rows."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    lens, news = _lengths(case)
    B, T, page = len(lens), sum(news), case["page"]
    H, KH, D, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32)  # pages lie anywhere
    table = torch.zeros((B, max(need)), dtype=torch.int32, device=dev)
    for b, at in enumerate(_starts(need)[:-1]):
        table[b, :need[b]] = order[at:at + need[b]]
    data = torch.empty((pages, KH, page // BLOCK, 64 * D + 16), dtype=torch.uint8, device=dev)
    _fill_codes(data, D, gen)
    s = dict(case=case, data=data, table=table, lens=_int32(lens, dev), starts=_int32(_starts(news), dev), tokens=T,
             max_new=max(news), scale=1.0 / math.sqrt(D))
    # the rows as slices of one joint projection of queries, keys and values
    qkv = torch.randn((T, (H + 2 * KH) * D), device=dev, generator=gen).to(dt)
    s["q"] = qkv[:, :H * D].view(T, H, D)
    s["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(news, device=dev))
    s["nth"] = torch.arange(T, device=dev) - s["starts"].long()[s["seq"]]
    if case["op"] == "append":
        s["k"] = qkv[:, H * D:(H + KH) * D].view(T, KH, D)
        s["v"] = qkv[:, (H + KH) * D:].view(T, KH, D)
        s["cos"], s["sin"] = _rotation(max(need) * page, case["rotary"], dev)
        # the blocks that the new tokens fall into, and the same batch counted from their beginnings
        hit = [(b, j) for b, (n, m) in enumerate(zip(lens, news)) for j in range((n - m) // BLOCK, (n + BLOCK - 1) // BLOCK)]
        s["hit_seq"] = torch.tensor([b for b, _ in hit], device=dev)
        s["hit_block"] = torch.tensor([j for _, j in hit], device=dev)
        back = [m + (n - m) % BLOCK for n, m in zip(lens, news)]
        s["back_starts"], s["back_tokens"], s["back_max"] = _int32(_starts(back), dev), sum(back), max(back)
        s["back_hit"] = torch.tensor([i for i, (b, j) in enumerate(hit) for _ in range(min(BLOCK, lens[b] - j * BLOCK))],
                                     device=dev)
        s["back_at"] = torch.tensor([p for b, j in hit for p in range(min(BLOCK, lens[b] - j * BLOCK))], device=dev)
    if own:  # the handles that a program keeps beside its tensors
        import block_quantized_int8_mmq_gb300 as mmq
        s["cache"] = mmq.KVCache(data)
        s["batch"] = mmq.KVBatch(s["starts"], s["lens"], table, T, s["max_new"])
        if case["op"] == "append":
            s["rope"] = mmq.Rope(s["cos"], s["sin"], interleaved=case["interleaved"])
            s["back"] = mmq.KVBatch(s["back_starts"], s["lens"], table, s["back_tokens"], s["back_max"])
    return s


# ----------------------------------------------------------------------------------- plain forms
def _codes(rec, which, D):
    """The key (0) or value (1) codes of records [..., 64 * D + 16] as f32 [..., 32, D], and their scales."""
    c = rec[..., 32 * D * which:32 * D * (which + 1)].contiguous().view(torch.int8)
    sc = rec[..., 64 * D + 4 * which:64 * D + 4 * which + 4].contiguous().view(torch.float32)
    return c.view(*c.shape[:-1], BLOCK, D).float(), sc[..., None]


def _attend_plain(s):
    c = s["case"]
    H, KH, D, W = c["heads"], c["kv_heads"], c["dim"], c["window"]
    G, B, N = H // KH, s["lens"].shape[0], s["max_new"]
    rec = s["data"][s["table"].long()]  # [B, pages, KH, blocks, bytes]
    rec = rec.transpose(1, 2).reshape(B, KH, -1, rec.shape[-1])
    kc, ks = _codes(rec, 0, D)
    vc, vs = _codes(rec, 1, D)
    del rec
    k = (kc * ks).view(B, KH, -1, D)
    v = (vc * vs).view(B, KH, -1, D)
    del kc, vc
    q = torch.zeros((B, N, H, D), device=k.device)
    q[s["seq"], s["nth"]] = s["q"].float()
    q = q.view(B, N, KH, G, D).transpose(1, 2).reshape(B, KH, N * G, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, KH, N, G, -1)
    lens, news = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    pos = (lens - news)[:, None] + torch.arange(N, device=k.device)[None]  # [B, N]
    key = torch.arange(k.shape[2], device=k.device)
    out_of = (key > pos[..., None]) | (key >= lens[:, None, None])
    if W:
        out_of = out_of | (key <= pos[..., None] - W)
    p.masked_fill_(out_of[:, None, :, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, KH, N * G, -1), v).view(B, KH, N, G, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.transpose(1, 2).reshape(B, N, H, D)[s["seq"], s["nth"]]
    return o.to(s["q"].dtype)


def _rotate(x, cos, sin, R, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _join(codes, old_scale, x, is_new, is_old):
    """One scale for a block's old and new tokens: [hits, KH, 32, D] codes and f32 values."""
    scale = torch.where(is_new[:, None, :, None], x, torch.zeros_like(x)).abs().amax((2, 3), keepdim=True)
    scale = scale / torch.full_like(scale, 127.0)
    had = is_old.any(-1)[:, None, None, None]
    scale = torch.where(had, torch.maximum(scale, old_scale), scale)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    new = (x / safe).round().clamp(-127, 127)
    old = torch.where(old_scale == scale, codes, (codes * (old_scale / safe)).round().clamp(-127, 127))
    codes = torch.where(is_new[:, None, :, None], new, torch.where(is_old[:, None, :, None], old, codes))
    return codes, scale


def _append_plain(s):
    c = s["case"]
    KH, D, R, page, data = c["kv_heads"], c["dim"], c["rotary"], c["page"], s["data"]
    lens, news = s["lens"].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    pos = (lens - news)[s["seq"]] + s["nth"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotate(s["q"], cos, sin, R, c["interleaved"])
    k = _rotate(s["k"], cos, sin, R, c["interleaved"])
    b, j = s["hit_seq"], s["hit_block"]
    at = j[:, None] * BLOCK + torch.arange(BLOCK, device=data.device)  # [hits, 32] positions
    first = (lens - news)[b][:, None]
    is_new, is_old = (at >= first) & (at < lens[b][:, None]), at < first
    row = (s["starts"].long()[b][:, None] + at - first).clamp(0, s["tokens"] - 1)
    where = s["table"].long()[b, j * BLOCK // page], j % (page // BLOCK)
    rec = data[where[0], :, where[1]]  # [hits, KH, bytes]
    kc, ks = _codes(rec, 0, D)
    vc, vs = _codes(rec, 1, D)
    kc, ks = _join(kc, ks, k[row].transpose(1, 2), is_new, is_old)
    vc, vs = _join(vc, vs, s["v"].float()[row].transpose(1, 2), is_new, is_old)
    put = torch.cat((kc.flatten(2).to(torch.int8).view(torch.uint8), vc.flatten(2).to(torch.int8).view(torch.uint8),
                     ks.flatten(2).contiguous().view(torch.uint8), vs.flatten(2).contiguous().view(torch.uint8),
                     rec[..., 64 * D + 8:]), -1)
    data[where[0], :, where[1]] = put
    # what the written blocks stand for, up to each sequence's end
    pick = s["back_hit"], slice(None), s["back_at"]
    dt = s["q"].dtype
    return {"q": q.to(dt), "k": (kc * ks)[pick].to(dt), "v": (vc * vs)[pick].to(dt)}


def run(state):
    s = state
    if own:
        import block_quantized_int8_mmq_gb300 as mmq
        if s["case"]["op"] == "attend":
            return mmq.mmq_kv_attend(s["cache"], s["batch"], s["q"], scale=s["scale"], window=s["case"]["window"])
        q = mmq.mmq_kv_append(s["cache"], s["batch"], s["k"], s["v"], q=s["q"], rope=s["rope"])
        k, v = mmq.mmq_kv_read(s["cache"], s["back"], dtype=s["q"].dtype)
        return {"q": q, "k": k, "v": v}
    return _attend_plain(s) if s["case"]["op"] == "attend" else _append_plain(s)


# ------------------------------------------------------------------------------------- 64 bits
def _values64(s, b, n):
    """Sequence b's first n tokens as the cache holds them: keys, values f64 [n, KH, D]."""
    D, page = s["case"]["dim"], s["case"]["page"]
    rec = s["data"][s["table"][b, :(n + page - 1) // page].long()].cpu()  # [pages, KH, blocks, bytes]
    got = []
    for w in (0, 1):
        codes = rec[..., w * 32 * D:(w + 1) * 32 * D].contiguous().view(torch.int8).to("cuda").double()
        sc = rec[..., 64 * D + 4 * w:64 * D + 4 * w + 4].contiguous().view(torch.float32).to("cuda").double()
        x = codes.unflatten(-1, (BLOCK, D)) * sc[..., None]
        got.append(x.permute(0, 2, 3, 1, 4).flatten(0, 2)[:n])
    return got


def _exact_attend(s):
    c = s["case"]
    H, KH, D, W = c["heads"], c["kv_heads"], c["dim"], c["window"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = torch.zeros((s["tokens"], H, D), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        m = starts[b + 1] - starts[b]
        k, v = _values64(s, b, n)
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        seen = (key <= pos) & (key > pos - W) if W else key <= pos
        for h in range(H):
            q = s["q"][starts[b]:starts[b + 1], h].double()
            x = (q @ k[:, h * KH // H].T * s["scale"]).masked_fill(~seen, -math.inf)
            out[starts[b]:starts[b + 1], h] = torch.softmax(x, -1) @ v[:, h * KH // H]
    return out


def _turn64(x, pos, s):
    R = s["case"]["rotary"]
    z = x[..., :R].double()
    w = (s["cos"].double() + 1j * s["sin"].double())[pos][:, None]  # the tables as given
    if s["case"]["interleaved"]:
        z = torch.view_as_real(torch.view_as_complex(z.reshape(*z.shape[:-1], R // 2, 2).contiguous()) * w).flatten(-2)
    else:
        z = torch.complex(z[..., :R // 2].contiguous(), z[..., R // 2:].contiguous()) * w
        z = torch.cat((z.real, z.imag), -1)
    return torch.cat((z, x[..., R:].double()), -1)


def _exact_append(s):
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = {"q": [], "k": [], "v": []}
    for b, n in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        m = starts[b + 1] - starts[b]
        pos = torch.arange(n - m, n, device="cuda")
        out["q"].append(_turn64(s["q"][rows], pos, s))
        had = _values64(s, b, n)
        for name, old, new in (("k", had[0], _turn64(s["k"][rows], pos, s)), ("v", had[1], s["v"][rows].double())):
            first = (n - m) // BLOCK * BLOCK
            x = torch.cat((old[first:n - m], new))  # the tokens of the blocks written to
            kept = n - m - first
            pad = -x.shape[0] % BLOCK
            x = torch.cat((x, x.new_zeros((pad, *x.shape[1:])))).unflatten(0, (-1, BLOCK))
            fresh = x.clone()
            if kept:
                fresh[0, :kept] = 0
            scale = fresh.abs().amax((1, 3), keepdim=True) / 127
            if kept:  # the scale that the block had, from its record
                blk, page, D = first // BLOCK, s["case"]["page"], s["case"]["dim"]
                at = 64 * D + (0 if name == "k" else 4)
                rec = s["data"][int(s["table"][b, first // page]), :, blk % (page // BLOCK), at:at + 4]
                had_scale = rec.contiguous().view(torch.float32).double()[None, :, :]
                scale[0] = torch.maximum(scale[0], had_scale)
            x = torch.where(scale > 0, (x / torch.where(scale > 0, scale, torch.ones_like(scale))).round(), torch.zeros_like(x))
            out[name].append((x.clamp(-127, 127) * scale).flatten(0, 1)[:kept + m])
    return {name: torch.cat(v) for name, v in out.items()}


def exact(case, seed):
    """What run returns, in 64 bits from the definition (float64 on the GPU, a sequence and a head
    at a time)."""
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend" else _exact_append(s)
