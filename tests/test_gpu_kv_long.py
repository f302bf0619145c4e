"""Attention over long runs of records on the GPU: every worker of the stream goes many times round its ring,
over the ends of pages, heads and sequences; sums of tens of thousands of terms.  The reference is 64-bit torch
on the same GPU."""
import math

import pytest
import torch

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def make_records(pages, heads, page, dim, gen, lowest):
    """Records of normal keys, values of codes lowest .. 127, and what they stand for: f64 [heads, tokens, dim]
    of page after page."""
    n = page // 32
    data = torch.zeros((pages, heads, n, 64 * dim + 16), dtype=torch.uint8, device="cuda")
    kc = torch.randn((pages, heads, n, 32 * dim), device="cuda", generator=gen).mul_(32).round_().clamp_(-127, 127)
    vc = torch.randint(lowest, 128, (pages, heads, n, 32 * dim), device="cuda", generator=gen)
    scales = torch.full((pages, heads, n, 2), 0.03, device="cuda")
    if lowest < 0:
        scales *= torch.rand(scales.shape, device="cuda", generator=gen) + 0.5
    data[..., :32 * dim] = kc.to(torch.int8).view(torch.uint8)
    data[..., 32 * dim:64 * dim] = vc.to(torch.int8).view(torch.uint8)
    data[..., 64 * dim:64 * dim + 8] = scales.view(torch.uint8)

    def values(codes, which):
        x = codes.double() * scales[..., which:which + 1].double()
        return x.view(pages, heads, n, 32, dim).transpose(0, 1)  # [heads, pages, n, 32, dim]

    return data, values(kc, 0), values(vc, 1)


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs,new", [(356, 1), (356, 4), (356, 6), (40, 130)])
def test_f32_sums_of_long_runs(dim, seqs, new):
    """f32 rows over 65500 tokens each (shared pages), values of one sign and of nearly one size: what is lost
    in adding them up shows.  Bound, of |out|:
      2^-19 (4 + S) spread  the weights' own errors (as in the other tests), which move the output by what the
                            values differ from it: spread = (127 - 96) / 96
      2^-22                 weights as two f16 terms
      2^-20                 a record's products (256 keys of the tiles) in the tensor cores, which round
                            towards zero
      2 * 6 sqrt(n / 3) 2^-23 / sqrt(12)   six deviations of n additions rounded to nearest, the sum of the
                            values and that of the weights, growing evenly; n: two a record of a unit at most"""
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    length, page, group = 65500, 256, 4
    pages = -(-length // page)
    data, k, v = make_records(pages, 1, page, dim, gen, 96)
    k, v = (x[0].reshape(-1, dim) for x in (k, v))
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].repeat(seqs, 1)
    batch = mmq.KVBatch(int32([new * i for i in range(seqs + 1)]), int32([length] * seqs), table, seqs * new, new)
    q = torch.randn((seqs * new, group, dim), device="cuda", generator=gen) * 0.3
    out = mmq.mmq_kv_attend(mmq.KVCache(data), batch, q, scale=1 / math.sqrt(dim))
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == 0
    n = 2 * -(-length // 32)
    for b in range(0, seqs, max(1, seqs // 9)):
        for t in {0, new // 2, new - 1}:
            end, x = length - new + t + 1, q[b * new + t].double()
            s = x @ k[:end].T / math.sqrt(dim)
            want = s.softmax(-1) @ v[:end]
            big = float((x.abs() @ k[:end].abs().T).max()) / math.sqrt(dim)
            bound = 2.0 ** -19 * (4 + big) * (127 - 96) / 96 + 2.0 ** -22 + 2.0 ** -20 + \
                12 * math.sqrt(n / 3) * 2.0 ** -23 / math.sqrt(12) + UNIT["f32"]
            off = float(((out[b * new + t].double() - want) / want).abs().max())
            assert off <= bound, f"2^{math.log2(off):.1f} off, 2^{math.log2(bound):.1f} allowed"


def stream_shape(dim, rows, dtype):
    """Of the attention stream with at most `rows` query rows a sequence and head: rows of a unit, workers on this
    GPU, records that a worker has in flight."""
    unit = 8 if dim == 256 or rows <= 8 else 16 if rows <= 16 or (dim == 128 and dtype == "f32") else 24
    warps = 6 if dim == 256 else 12 if unit == 8 else 8
    stages = 4 if dim == 64 else 3 if dim == 128 and unit > 8 else 2
    return unit, warps * torch.cuda.get_device_properties(0).multi_processor_count, stages


# (query heads a key/value head, new tokens): units of 8, 16 and 24 rows, one or several of them a sequence and head
ROWS = {64: [(4, 1), (4, 4), (8, 3), (4, 11)], 128: [(7, 1), (4, 4), (8, 3), (8, 5)], 256: [(4, 2), (8, 2)]}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,group,new", [(d, g, n) for d in ROWS for g, n in ROWS[d]])
@pytest.mark.parametrize("heads,page,window", [(4, 32, 0), (3, 256, 0), (4, 96, 700)])
def test_workers_go_many_times_round_their_rings(dtype, dim, group, new, heads, page, window):
    """Ragged sequences with idle slots between them: at least twelve records and three ring turns a worker,
    ranges that hold whole units, ends of units, pages and windows of the page table.  All rows against 64 bits,
    with the bound of the other attention tests."""
    gen = torch.Generator(device="cuda").manual_seed(dim + group + new + page)
    unit, workers, stages = stream_shape(dim, group * new, dtype)
    lens, news, records = [], [], 0
    while records < workers * max(12, 3 * stages):
        i = len(lens)
        n = 40 + int(4300 * ((i * 0.6180339887 + 0.1) % 1.0) ** 1.5)
        m = 0 if i % 7 == 3 else new if i % 3 else 1 + i % new
        first = max(0, n - m - window + 1) if window else 0
        records += heads * -(-m * group // unit) * (-(-n // 32) - first // 32)
        lens.append(n)
        news.append(m)
    need = [-(-n // page) for n in lens]
    data, k, v = make_records(sum(need) + 1, heads, page, dim, gen, -127)
    order = torch.randperm(sum(need) + 1, device="cuda", generator=gen)
    table = torch.full((len(lens), max(need)), -3, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for m in news:
        starts.append(starts[-1] + m)
    T, H = starts[-1], heads * group
    batch = mmq.KVBatch(int32(starts), int32(lens), table, T, new)
    q = torch.randn((T, H, dim), device="cuda", generator=gen).to(DT[dtype])
    scale = 1 / math.sqrt(dim)
    out, lse = torch.full_like(q, float("nan")), torch.full((T, H), float("nan"), device="cuda")
    mmq.mmq_profile_read(reset=True)
    before = mmq.mmq_profile_enable(True)
    mmq.mmq_kv_attend(mmq.KVCache(data), batch, q, scale=scale, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    mmq.mmq_profile_enable(before)
    assert "k_kv_attend_stream" in mmq.mmq_profile_read(reset=True)
    assert mmq.mmq_get_device_error() == 0
    e = 2.0 ** -22 if dtype == "f32" else 2.0 ** -11
    for b, (n, m) in enumerate(zip(lens, news)):
        if m == 0:
            continue
        pages = table[b, :need[b]].long()
        kk, vv = (x[:, pages].reshape(heads, -1, dim)[:, :n] for x in (k, v))
        rows = slice(starts[b], starts[b + 1])
        x = q[rows].double().view(m, heads, group, dim).transpose(0, 1).reshape(heads, m * group, dim)
        pos = torch.arange(n - m, n, device="cuda").repeat_interleave(group)[:, None]
        key = torch.arange(n, device="cuda")[None]
        seen = (key <= pos) & (key > pos - window) if window else key <= pos
        s = (x @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
        big = (x.abs() @ kk.abs().transpose(1, 2) * scale).masked_fill(~seen, 0).amax(-1)
        w = s.softmax(-1)

        def back(t):
            return t.view(heads, m, group, -1).transpose(0, 1).reshape(m, H, -1)

        want, size, f = back(w @ vv), back(w @ vv.abs()), 2.0 ** -19 * (4 + back(big))
        bound = UNIT[dtype] * want.abs() + (2.0 ** -25 if dtype == "f16" else 0) + (e + f) * size + \
            2.0 ** -31 * n * float(vv.abs().max())
        off = (out[rows].double() - want).abs()
        assert bool((off <= bound).all()), f"sequence {b}: {float((off / bound).max())} of the bound"
        ref = back(s.logsumexp(-1)[..., None])[..., 0]
        assert bool(((lse[rows].double() - ref).abs() <= 2 * f[..., 0] + 2.0 ** -22 * ref.abs()).all())
