"""The 8-bit key/value cache on the GPU against its definition (tests/kv_ref.py): the cache's bytes
and the rotated queries bit for bit, attention against 64 bits.

Bounds of the attention tests, per element of out = sum_j w_j v_j:
  u |out|            one rounding to the output type (u = 2^-8 bf16, of 8 significant bits, 2^-11 f16, 2^-24 f32;
                     + 2^-25, f16's smallest half step)
  (e + f) sum w|v|   e: weights rounded to f16 (2^-11), or split into two f16 terms (f32 rows: 2^-22);
                     f = 2^-19 (4 + S): the scores' f32 sums and the exponential, S = max sum |q k| scale
                     (dim products and their sum in f32: well below 2^-19 S; the exponential's argument
                     and its own error: below 2^-19 * 4)
  2^-31 n max|v|     weights below the smallest f16 step are dropped (2^-32 of the largest, n tokens)
"""
import numpy as np
import pytest
import torch

import kv_ref

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
MMQ_ERR_RANGE = -11


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), device="cuda") if dtype is None else torch.as_tensor(x, device="cuda").to(dtype)


def clean():
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == 0


class Case:
    """A cache whose pages lie in no order, its unused parts full of what must not matter."""

    def __init__(self, seed, lens, news, heads, kv_heads, dim, page, dtype, pad_rows=0, spare=3):
        r = self.r = np.random.default_rng(seed)
        self.lens, self.news, self.H, self.KH, self.D, self.page, self.dt = lens, news, heads, kv_heads, dim, page, dtype
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.T = int(self.starts[-1]) + pad_rows
        need = [-(-n // page) for n in lens]
        mp = max(need + [1]) + 1
        ids = r.permutation(sum(need) + spare)
        self.pages = len(ids)
        self.table = np.full((len(lens), mp), -5, np.int32)  # past a length: never a page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.data = r.integers(0, 256, (self.pages, kv_heads, page // 32, kv_ref.rec_bytes(dim))).astype(np.uint8)
        scales = self.data[..., 64 * dim:64 * dim + 8].copy().view(np.float32)
        scales[:] = np.nan
        for b, n in enumerate(lens):
            for blk in range(-(-n // 32)):
                pg, i = self.table[b, blk // (page // 32)], blk % (page // 32)
                scales[pg, :, i] = r.uniform(0.004, 0.03, (kv_heads, 2))
                codes = self.data[pg, :, i, :64 * dim].view(np.int8)
                codes[:] = np.clip(np.rint(r.normal(0, 32, codes.shape)), -127, 127)
        self.data[..., 64 * dim:64 * dim + 8] = scales.view(np.uint8)

    def rows(self, heads, scale=1.0):
        x = torch.from_numpy(self.r.normal(0, scale, (self.T, heads, self.D)).astype(np.float32))
        return x.to(DT[self.dt])

    def upload(self):
        self.cache = mmq.KVCache(dev(self.data))
        self.batch = mmq.KVBatch(dev(self.starts), dev(np.asarray(self.lens, np.int32)), dev(self.table), self.T,
                                 max(list(self.news) + [0]))
        return self.cache, self.batch

    def real(self):
        """Which rows are tokens of a sequence."""
        at = np.full(self.T, -1)
        for b, n in enumerate(self.news):
            at[self.starts[b]:self.starts[b + 1]] = self.lens[b] - n + np.arange(n)
        return at >= 0


def tables(rows, rotary, seed=0):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rotary, 2) / rotary)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def check_append(c, rope=None, want_q=True, k=None, v=None, strided=False):
    """Appends on the GPU and in the reference, compares the whole cache and the queries."""
    k = c.rows(c.KH) if k is None else k
    v = c.rows(c.KH) if v is None else v
    q = c.rows(c.H)
    cache, batch = c.upload()
    if strided:  # slices of one joint projection
        joint = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).cuda()
        n, m = c.H * c.D, c.KH * c.D
        gq, gk, gv = (joint[:, a:a + w].view(c.T, -1, c.D) for a, w in ((0, n), (n, m), (n + m, m)))
        assert not gk.is_contiguous()
    else:
        gq, gk, gv = q.cuda(), k.cuda(), v.cuda()
    gr = None if rope is None else mmq.Rope(dev(rope[0]), dev(rope[1]), interleaved=rope[2])
    fill = torch.full((c.T, c.H, c.D), 7.0, dtype=DT[c.dt], device="cuda")
    got = mmq.mmq_kv_append(cache, batch, gk, gv, q=gq if want_q else None, rope=gr, q_out=fill if want_q else None)
    clean()
    ref = c.data.copy()
    kv_ref.append(ref, c.starts, c.lens, c.table, k.float().numpy(), v.float().numpy(), c.D, rope)
    assert np.array_equal(cache.data.cpu().numpy(), ref)
    if want_q:
        pos = np.full(c.T, -1)
        for b, n in enumerate(c.news):
            pos[c.starts[b]:c.starts[b + 1]] = c.lens[b] - n + np.arange(n)
        x = q.float().numpy()
        want = np.full(x.shape, 7.0, np.float32)
        for t in range(c.T):
            if pos[t] >= 0:
                for h in range(c.H):
                    want[t, h] = kv_ref.rotate(x[t, h], pos[t], *rope) if rope else x[t, h]
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(DT[c.dt]))
    else:
        assert got is None
    return cache, batch, ref


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,rotary,interleaved", [(128, 128, False), (64, 32, True), (256, 256, True), (64, 64, False),
                                                    (128, 40, False), (256, 8, False)])
def test_append_bits(dtype, dim, rotary, interleaved):
    lens, news = [70, 1, 33, 160, 64, 31], [70, 1, 2, 97, 32, 1]
    c = Case(dim + rotary, lens, news, 6, 2, dim, 64, dtype)
    check_append(c, (*tables(192, rotary), interleaved))


@pytest.mark.parametrize("page", [32, 96, 256])
def test_append_pages_and_strides(page):
    c = Case(page, [300, 5, 97], [201, 5, 64], 4, 4, 64, page, "f32")
    check_append(c, (*tables(512, 64), False), strided=True)


@pytest.mark.parametrize("news,lens", [([0, 3, 0], [10, 3, 0]), ([1, 1, 1], [1, 0, 40]), ([4, 2], [2, 2]), ([5], [0]),
                                       ([1] * 40, list(range(1, 41)))])
def test_append_empty_padding_and_many(news, lens):
    c = Case(len(news) + sum(lens), lens, news, 4, 2, 64, 32, "bf16", pad_rows=3)
    check_append(c, (*tables(64, 64), True))
    check_append(Case(5, lens, news, 4, 2, 128, 64, "f32"), None, want_q=False)


def test_append_more_sequences_than_threads():
    r = np.random.default_rng(1)
    news = r.integers(0, 4, 700)
    lens = news + r.integers(0, 80, 700)
    check_append(Case(3, lens.tolist(), news.tolist(), 1, 1, 64, 32, "f32"), (*tables(96, 64), False))


def test_append_scales():
    """Growing, equal and all-zero scales, codes at ties, values below the smallest scale."""
    c = Case(9, [40, 40, 40, 40, 33], [8, 8, 8, 8, 33], 2, 1, 64, 32, "f32")
    k, v = c.rows(1, 0.01), c.rows(1, 50.0)  # keys keep the older scale, values outgrow it
    k[8:16], v[8:16] = 0, 0                  # nothing but zeros beside older tokens
    k[16:24], v[16:24] = 1e-33, 1e-29        # below and above 127 * 2^-100 beside larger ones
    k[24:32] = torch.arange(-32, 32).float()[None, None] * 0.5
    v[24:32] = 3.0
    k[32:], v[32:] = 0, 1e-32                # a whole new block of zeros, and one that counts as zero
    cache, batch, ref = check_append(c, None, k=k, v=v)
    _, _, d = kv_ref.split(kv_ref.record(ref, c.table, 4, 0, 0), 64)
    assert d.tolist() == [0.0, 0.0]


def test_append_token_by_token():
    """A sequence grown one token at a time: every step's bytes are the reference's."""
    c = Case(11, [70], [1], 2, 2, 64, 32, "f32")
    rope = (*tables(96, 64), False)
    cache, batch = c.upload()
    gr = mmq.Rope(dev(rope[0]), dev(rope[1]))
    ref = c.data.copy()
    for n in range(1, 71):
        batch.lens.fill_(n)
        k, v = c.rows(2, 1.0 + n % 5), c.rows(2)
        mmq.mmq_kv_append(cache, batch, k.cuda(), v.cuda(), rope=gr)
        kv_ref.append(ref, [0, 1], [n], c.table, k.numpy(), v.numpy(), 64, rope)
    clean()
    assert np.array_equal(cache.data.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64), (256, 96)])
def test_read_bits(dtype, dim, page):
    lens, news = [100, 31, 1, 65, 0], [100, 2, 1, 33, 2]
    c = Case(dim, lens, news, 2, 2, dim, page, dtype, pad_rows=1)
    cache, batch = c.upload()
    out = [torch.full((c.T, 2, dim), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    got = mmq.mmq_kv_read(cache, batch, dtype=DT[dtype], k_out=out[0], v_out=out[1])
    clean()
    for w in (0, 1):
        want = torch.full((c.T, 2, dim), 7.0)
        for b, n in enumerate(news):
            if lens[b]:
                x = kv_ref.values(c.data, c.table, b, lens[b], dim, w, np.float32)[lens[b] - n:]
                want[c.starts[b]:c.starts[b + 1]] = torch.from_numpy(x)
        assert torch.equal(got[w].cpu(), want.to(DT[dtype]))


# ------------------------------------------------------------------------------------ attention
def compare_attend(c, got, lse, q, scale, window=0, data=None):
    out, ref_lse, absum, big = kv_ref.attend(c.data if data is None else data, c.starts, c.lens, c.table,
                                             q.float().numpy(), c.D, scale, window)
    rows = ~np.isnan(out[..., 0])
    e = 2.0 ** -22 if c.dt == "f32" else 2.0 ** -11
    f = 2.0 ** -19 * (4 + big)
    vmax = absum.max() if absum.size else 0.0
    bound = UNIT[c.dt] * np.abs(out) + (2.0 ** -25 if c.dt == "f16" else 0) + (e + f)[..., None] * absum + \
        2.0 ** -31 * max(list(c.lens) + [1]) * vmax * 4
    err = np.abs(got.cpu().double().numpy() - out)
    assert np.all(err[rows] <= bound[rows]), f"{np.nanmax(err[rows] / bound[rows])} of the bound"
    if lse is not None:
        x, y = lse.cpu().double().numpy()[rows], ref_lse[rows]
        empty = np.isneginf(y)
        assert np.array_equal(np.isneginf(x), empty)
        x, y = x[~empty], y[~empty]
        assert np.all(np.abs(x - y) <= 2 * f[rows][~empty] + 2.0 ** -22 * np.abs(y))


def check_attend(c, window=0, scale=None, qscale=1.0, q=None):
    q = c.rows(c.H, qscale) if q is None else q
    cache, batch = c.upload()
    scale = 1 / np.sqrt(c.D) if scale is None else scale
    out = torch.full((c.T, c.H, c.D), float("nan"), dtype=DT[c.dt], device="cuda")
    lse = torch.full((c.T, c.H), float("nan"), device="cuda")
    mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=scale, window=window, out=out, lse=lse)
    clean()
    compare_attend(c, out, lse, q, scale, window)
    again = mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=scale, window=window)
    rows = np.zeros(c.T, bool)
    rows[c.starts[0]:c.starts[-1]] = True
    assert torch.equal(out[rows], again[rows])
    assert np.array_equal(cache.data.cpu().numpy(), c.data)  # only read
    if not rows.all():  # rows of no sequence are left alone
        assert out[~rows].isnan().all() and lse[~rows].isnan().all()
    return out, lse


HEADS = [(7, 1), (4, 4), (16, 2), (6, 2), (32, 2), (5, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_attend_decode(dtype, dim, heads):
    """One new token a sequence: lengths around block and page ends, one, and an idle slot."""
    lens = [1, 31, 32, 33, 0, 64, 95, 200, 257, 2]
    check_attend(Case(dim, lens, [1] * len(lens), *heads, dim, 64, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(7, 1), (4, 4), (16, 2)])
def test_attend_prompts(dtype, dim, heads):
    """Ragged prompts: tiles that end inside a page, rows past a tile's end, padding rows."""
    c = Case(7 * dim, [150, 40, 129, 3, 0], [150, 3, 64, 5, 2], *heads, dim, 32, dtype, pad_rows=2)
    check_attend(c)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("news", [[2, 5, 0, 3], [8, 1, 7, 4], [33, 17, 0, 1]])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_attend_few_rows(dtype, news, window):
    check_attend(Case(13, [90, 300, 77, 129], news, 8, 2, 128, 64, dtype), window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news,group", [([4, 0, 1, 3], 4), ([3, 3, 2, 1], 7), ([6, 1, 5, 0], 4), ([12, 0, 7, 9], 4),
                                        ([48, 17, 1, 25], 1), ([2, 1, 2, 2], 24)])
@pytest.mark.parametrize("window", [0, 45])
def test_attend_row_groups(dtype, dim, news, group, window):
    """Sequences whose 9 to 48 rows are several units of the same records, beside some with one."""
    c = Case(dim + group, [90, 700, 77, 129], news, 2 * group, 2, dim, 64, dtype, pad_rows=1)
    check_attend(c, window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 1 << 30, 1 << 40])
def test_attend_window(dtype, window):
    check_attend(Case(window % 1000, [1, 40, 333, 96], [1] * 4, 4, 2, 64, 32, dtype), window=window)
    check_attend(Case(window % 999, [140, 40, 333], [140, 9, 200], 4, 2, 64, 32, dtype), window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_attend_sharp_and_flat(dtype, new):
    """Softmax with one token far above the rest, in turn late and early, and with all alike."""
    for qs, scale in ((8.0, 0.3), (1e-6, 0.1), (1.0, 4.0)):
        check_attend(Case(17, [300, 90], [new] * 2, 4, 2, 64, 32, dtype), scale=scale, qscale=qs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_attend_scales_of_every_size(dtype, new):
    """Blocks of zeros, of tiny and of large values beside each other, keys that are all zero."""
    c = Case(19, [320, 64], [new] * 2, 4, 2, 64, 32, dtype)
    for i, (a, b) in enumerate([(0.01, 0.0), (0.0, 0.02), (0.02, 1e-6), (0.01, 300.0), (0.0, 0.0), (0.01, 1e-25),
                                (1e-20, 0.01), (0.01, 2.0), (0.03, 1e-31), (0.01, 0.01)]):
        for h in range(2):
            kc, vc, d = kv_ref.split(kv_ref.record(c.data, c.table, 0, i, h), 64)
            d[:] = (a, b if b > 2.0 ** -100 else 0)
            if d[0] == 0:
                kc[:] = 0
            if d[1] == 0:
                vc[:] = 0
    for blk in range(2):  # a sequence of nothing but zero values
        for h in range(2):
            _, vc, d = kv_ref.split(kv_ref.record(c.data, c.table, 1, blk, h), 64)
            d[1], vc[:] = 0, 0
    out, _ = check_attend(c)
    assert (out[c.starts[1]:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("new", [1, 5, 300])
def test_attend_longer(dtype, new):
    """Lengths that are shared out over many workers and joined, beside short ones."""
    check_attend(Case(23, [5000, 300, 2049, 1000], [min(new, 300), 1, new, new], 4, 1, 128, 128, dtype))


@pytest.mark.parametrize("new", [1, 2])
def test_attend_many_sequences(new):
    r = np.random.default_rng(2)
    lens = r.integers(0, 70, 600).tolist()
    check_attend(Case(29, lens, [new] * 600, 2, 1, 64, 32, "bf16"))


@pytest.mark.parametrize("dtype,window", [("bf16", 0), ("f16", 300), ("f32", 0)])
@pytest.mark.parametrize("lens,news", [([1400], [1400]), ([1100, 640, 33, 900, 257], [800, 640, 33, 400, 256])])
def test_attend_more_units_than_sms(dtype, window, lens, news):
    """Units of many lengths, several a CTA, whole or cut."""
    check_attend(Case(sum(lens), lens, news, 32, 8, 64, 64, dtype), window=window)


def test_attend_more_sequences_than_threads():
    lens = [30 + 7 * i % 50 for i in range(400)]
    check_attend(Case(61, lens, [30] * 400, 4, 2, 64, 32, "bf16"))


@pytest.mark.parametrize("dtype,length,dim", [("bf16", 20000, 64), ("f32", 20000, 128), ("f16", 9000, 256),
                                              ("bf16", 140000, 64)])
@pytest.mark.parametrize("new", [1, 3])
def test_attend_many_parts(dtype, length, dim, new):
    """One long sequence of one key/value head: its parts are joined in one, two and three steps."""
    c = Case(length, [length], [new], 8, 1, dim, 256, dtype)
    check_attend(c)


@pytest.mark.parametrize("seed", range(24))
def test_attend_drawn(seed):
    """Shapes, types, windows and lengths drawn with a fixed seed."""
    r = np.random.default_rng(1000 + seed)
    kh, group = [(1, 7), (2, 4), (4, 1), (1, 8), (3, 2), (1, 16)][r.integers(6)]
    dim, page = int(r.choice([64, 128, 256])), int(r.choice([32, 64, 96, 256]))
    seqs = int(r.integers(1, 7))
    news = np.exp(r.uniform(0, np.log(150), seqs)).astype(int) if seed % 2 else r.integers(1, 5, seqs)
    lens = news + (np.exp(r.uniform(0, np.log(700), seqs)).astype(int) - 1) * (r.random(seqs) < 0.8)
    c = Case(seed, lens.tolist(), news.tolist(), kh * group, kh, dim, page, ["f32", "bf16", "f16"][seed % 3])
    check_attend(c, window=int(r.choice([0, 0, 50, 200])), qscale=float(r.choice([0.3, 1.0, 3.0])))


def test_attend_query_range():
    """Rows of very different sizes, a row of zeros, elements far below their row's largest."""
    for dtype in ("f32", "bf16", "f16"):
        for new in (6, 40):
            c = Case(31, [200, 77], [new, 1], 4, 2, 128, 64, dtype)
            q = c.rows(4).float()
            q[0], q[1] = 0, q[1] * 1e-4
            q[2, :, ::2] *= 1e-3
            q[3] *= 6.0
            q[4, 0], q[4, 1] = q[4, 0] * (1e-30 if dtype != "f16" else 1e-5), 0
            check_attend(c, q=q.to(DT[dtype]))


def test_attend_strided_queries_and_outputs():
    c = Case(37, [100, 50], [3, 40], 4, 2, 64, 32, "bf16")
    q = c.rows(4)
    cache, batch = c.upload()
    wide = torch.zeros((c.T, 9, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 1::2] = q.cuda()
    out = mmq.mmq_kv_attend(cache, batch, wide[:, 1::2])
    clean()
    compare_attend(c, out, None, q, 1 / 8.0)
    with pytest.raises(ValueError):
        mmq.mmq_kv_attend(cache, batch, wide.transpose(1, 2)[:, :4])
    with pytest.raises(mmq.MMQError):
        odd = torch.zeros((c.T, 4 * 64 + 4), dtype=torch.bfloat16, device="cuda")[:, :256].view(c.T, 4, 64)
        mmq.mmq_kv_attend(cache, batch, odd)


def test_page_numbers_far_apart():
    """Records past 2^32 bytes, a table with a stride of its own."""
    dim, page, kh = 128, 256, 8
    rec = kv_ref.rec_bytes(dim)
    pages = (5 << 30) // (kh * page // 32 * rec)
    c = Case(41, [300, 290], [1, 40], 8, kh, dim, page, "bf16")
    data = torch.zeros((pages, kh, page // 32, rec), dtype=torch.uint8, device="cuda")
    new = {int(old): pages - 1 - 3 * i for i, old in enumerate(np.unique(c.table[c.table >= 0]))}
    table = c.table.copy()
    for old, to in new.items():
        data[to] = dev(c.data[old])
        table[c.table == old] = to
    cache = mmq.KVCache(data)
    wide = torch.full((2, 7), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = dev(table)
    batch = mmq.KVBatch(dev(c.starts), dev(np.asarray(c.lens, np.int32)), wide[:, :table.shape[1]], c.T, 40)
    q, k, v = c.rows(8), c.rows(kh), c.rows(kh)
    mmq.mmq_kv_append(cache, batch, k.cuda(), v.cuda())
    out = mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=0.1)
    clean()
    kv_ref.append(c.data, c.starts, c.lens, c.table, k.float().numpy(), v.float().numpy(), dim)
    for old, to in new.items():
        assert np.array_equal(data[to].cpu().numpy(), c.data[old])
    compare_attend(c, out, None, q, 0.1)


@pytest.mark.parametrize("new", [1, 4, 60])
def test_other_stream_and_graph(new):
    """On a side stream, then captured once and replayed with other lengths and other rows."""
    c = Case(43, [200, 200], [new] * 2, 4, 2, 64, 32, "f32")  # the pages that the longest replay needs
    cache, batch = c.upload()
    q, k, v = (c.rows(h).cuda() for h in (4, 2, 2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = mmq.mmq_kv_attend(cache, batch, q, scale=0.2, stream=side)
    side.synchronize()
    compare_attend(c, out, None, q.cpu(), 0.2)
    rope = (*tables(256, 64), False)
    gr = mmq.Rope(dev(rope[0]), dev(rope[1]))
    ws = torch.zeros(mmq.mmq_kv_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    turned, got = torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mmq.mmq_kv_append(cache, batch, k, v, q=q, rope=gr, q_out=turned)
        mmq.mmq_kv_attend(cache, batch, turned, scale=0.2, out=got, workspace=ws)
    for lens in ([200, 130], [61, 197], [64, 60]):
        c.lens = lens
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(c.rows(4))
        k.copy_(c.rows(2))
        v.copy_(c.rows(2))
        cache.data.copy_(dev(c.data))
        graph.replay()
        clean()
        ref = c.data.copy()
        kv_ref.append(ref, c.starts, lens, c.table, k.cpu().numpy(), v.cpu().numpy(), 64, rope)
        assert np.array_equal(cache.data.cpu().numpy(), ref)
        compare_attend(c, got, None, turned.cpu(), 0.2, data=ref)
    assert (ws[:16384] == 0).all()


def test_graphs_without_a_workspace():
    """Two captures on a stream that no call has run on, replayed in the other order, then a call on it."""
    c = Case(53, [900, 2100], [1, 2], 8, 2, 128, 64, "bf16")
    cache, batch = c.upload()
    q = c.rows(8)
    qd, side, graphs, outs = q.cuda(), torch.cuda.Stream(), [], []
    for _ in range(2):
        out = torch.zeros_like(qd)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(2):  # two calls of one graph
                mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, out=out)
        graphs.append(graph)
        outs.append(out)
    for i in (1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        clean()
        compare_attend(c, outs[i], None, q, 0.1)
    with torch.cuda.stream(side):
        out = mmq.mmq_kv_attend(cache, batch, qd, scale=0.1)
    clean()
    compare_attend(c, out, None, q, 0.1)


def test_package_workspaces_are_zeroed_after_a_timeout(monkeypatch):
    """The error word's status is a stand-in: no wait runs out."""
    from block_quantized_int8_mmq_gb300 import kv
    c = Case(59, [900], [1], 8, 2, 128, 64, "bf16")
    cache, batch = c.upload()
    q = c.rows(8)
    mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=0.1)
    clean()
    for ws in kv._workspaces.values():
        ws[:16384] = 1

    class Lib:
        def mmq_get_device_error(self, stream):
            return -7

    monkeypatch.setattr(mmq, "_lib", Lib())
    assert mmq.mmq_get_device_error() == -7
    monkeypatch.undo()
    assert all((ws[:16384] == 0).all() for ws in kv._workspaces.values())
    out = mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=0.1)
    clean()
    compare_attend(c, out, None, q, 0.1)


def test_workspace_is_left_clean_and_shared():
    """Calls of other shapes follow one another on one workspace."""
    ws = torch.zeros(mmq.mmq_kv_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    for seed, (lens, news) in enumerate([([3000], [1]), ([900, 20, 4000], [1, 1, 1]), ([700, 900], [300, 17]), ([31], [1]),
                                         ([2500], [9]), ([2600, 5], [1, 2])]):
        c = Case(47 + seed, lens, news, 7, 1, 128, 64, "bf16")
        cache, batch = c.upload()
        q = c.rows(7)
        out = mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=0.1, workspace=ws)
        clean()
        compare_attend(c, out, None, q, 0.1)
        assert (ws[:16384] == 0).all()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what", ["page", "length", "negative", "starts", "past tokens", "max_new"])
def test_values_out_of_range_are_not_followed(what, new):
    """Sequence 1 of three is wrong in device memory: the error word says so, nothing else changes."""
    c = Case(53, [90, 80, 70], [new] * 3, 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    q, k, v = (c.rows(h).cuda() for h in (4, 2, 2))
    good = mmq.mmq_kv_attend(cache, batch, q)
    clean()
    if what == "page":
        batch.table[1, 2] = c.pages
    elif what == "length":
        batch.lens[1] = c.table.shape[1] * 32 + 1
    elif what == "negative":
        batch.lens[1] = -1
    elif what == "starts":
        batch.starts[1] = 3 * new + 5
    elif what == "past tokens":
        batch.starts[3] = 3 * new + 1
    else:
        batch._c.max_new = new - 1
        if new == 1:
            batch._c.max_new = 1
            batch.starts[1] = 0  # sequence 1 then has two new tokens
    out = torch.full_like(q, 9.0)
    mmq.mmq_kv_attend(cache, batch, q, out=out)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE
    assert mmq.mmq_get_device_error() == 0
    if what in ("page", "length", "negative"):  # the other sequences' rows are right
        rest = out.clone()
        rest[new:2 * new] = good[new:2 * new]
        compare_attend(c, rest, None, q.cpu(), 1 / 8.0)
    if what in ("length", "negative"):
        assert (out[new:2 * new] == 9.0).all()
    mmq.mmq_kv_append(cache, batch, k, v, q=q, rope=None)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE
    if what in ("length", "negative"):  # the other sequences' records, and only theirs, are written
        ref = c.data.copy()
        for b in (0, 2):
            kv_ref.append(ref, [c.starts[b], c.starts[b + 1]], [c.lens[b]], c.table[b:b + 1], k.cpu().numpy(),
                          v.cpu().numpy(), 64)
        assert np.array_equal(cache.data.cpu().numpy(), ref)
    mmq.mmq_kv_read(cache, batch)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE


def test_position_past_the_rotation_tables():
    c = Case(59, [90], [1], 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    cos, sin = tables(89, 64)
    mmq.mmq_kv_append(cache, batch, c.rows(2).cuda(), c.rows(2).cuda(), rope=mmq.Rope(dev(cos), dev(sin)))
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE


def test_python_refusals():
    c = Case(61, [40], [2], 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    q, k = c.rows(4).cuda(), c.rows(2).cuda()
    for bad in (q[:1], q.half()[:, :, :32], q.double(), q.cpu()):
        with pytest.raises(ValueError):
            mmq.mmq_kv_attend(cache, batch, bad)
    with pytest.raises(ValueError):
        mmq.mmq_kv_append(cache, batch, k, k.half())
    with pytest.raises(ValueError):
        mmq.mmq_kv_append(cache, batch, k[:, :1], k[:, :1])
    with pytest.raises(ValueError):
        mmq.mmq_kv_attend(cache, batch, q, out=torch.empty_like(q, dtype=torch.float16))
    with pytest.raises(ValueError):
        mmq.mmq_kv_read(cache, batch, dtype=torch.float64)
    with pytest.raises(mmq.MMQError) as e:
        mmq.mmq_kv_attend(cache, batch, q, workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -1
    with pytest.raises(mmq.MMQError):
        mmq.mmq_kv_attend(cache, batch, q[:, :3])
    with pytest.raises(mmq.MMQError):
        mmq.mmq_kv_attend(cache, batch, q, scale=-1.0)


def test_no_rows():
    c = Case(67, [40, 3], [0, 0], 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    q, k = (torch.empty((0, h, 64), device="cuda") for h in (4, 2))
    assert mmq.mmq_kv_append(cache, batch, k, k, q=q).shape == (0, 4, 64)
    assert mmq.mmq_kv_attend(cache, batch, q).shape == (0, 4, 64)
    assert mmq.mmq_kv_read(cache, batch)[0].shape == (0, 2, 64)
    clean()


def test_profiler_names():
    c = Case(71, [40], [2], 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    mmq.mmq_profile_read(reset=True)
    prev = mmq.mmq_profile_enable(True)
    try:
        q = mmq.mmq_kv_append(cache, batch, c.rows(2).cuda(), c.rows(2).cuda(), q=c.rows(4).cuda())
        mmq.mmq_kv_attend(cache, batch, q)
        mmq.mmq_kv_read(cache, batch)
        names = mmq.mmq_profile_read(reset=True)
    finally:
        mmq.mmq_profile_enable(prev)
    assert {"k_kv_append", "k_kv_read"} <= set(names) and any(n.startswith("k_kv_attend") for n in names)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_k"])
def test_attention_layer_example(fmt):
    """Projections, append and attention together: prompts, then captured single-token steps. The
    bound is the f32 one of the tests above for scores up to S = 60 or so: 2^-19 (4 + S) < 1.3e-4."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.run(fmt, prompts=(90, 33, 5), steps=5, page=32, quiet=True, hidden=512, heads=8, kv_heads=2, dim=64) < 1.3e-4


def test_a_capture_on_a_stream_in_use_has_its_own_workspace():
    """Two graphs captured on a stream that has already run a call share nothing with it or each other: what
    a call leaves in the stream's workspace does not reach the replays."""
    from block_quantized_int8_mmq_gb300 import kv
    c = Case(73, [900, 2100], [1, 2], 8, 2, 128, 64, "bf16")
    cache, batch = c.upload()
    q = c.rows(8)
    qd, side = q.cuda(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mmq.mmq_kv_attend(cache, batch, qd, scale=0.1)
    side.synchronize()
    kept = kv._workspaces[(0, side.cuda_stream, 128)]
    graphs, outs = [], []
    for i in range(2):
        out = torch.zeros_like(qd)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, out=out)
            if i:  # and once more in one graph, the stream named
                mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, out=out, stream=side)
        graphs.append(graph)
        outs.append(out)
    kept.fill_(255)  # counters that no call has left, partial results that are NaN
    for i in (0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        clean()
        compare_attend(c, outs[i], None, q, 0.1)
    assert (kept == 255).all()
    kept[:16384].zero_()
    with torch.cuda.stream(side):
        out = mmq.mmq_kv_attend(cache, batch, qd, scale=0.1)
    clean()
    compare_attend(c, out, None, q, 0.1)


def test_a_capture_of_a_named_stream_has_its_own_workspace():
    """The same where the captured stream is not the current one but joined to its capture."""
    from block_quantized_int8_mmq_gb300 import kv
    c = Case(79, [900, 2100], [1, 2], 8, 2, 128, 64, "bf16")
    cache, batch = c.upload()
    q = c.rows(8)
    qd, side, out = q.cuda(), torch.cuda.Stream(), torch.zeros_like(q, device="cuda")
    torch.cuda.synchronize()
    mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, stream=side)
    side.synchronize()
    kept = kv._workspaces[(0, side.cuda_stream, 128)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, out=out, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    kept.fill_(255)
    graph.replay()
    clean()
    compare_attend(c, out, None, q, 0.1)
    assert (kept == 255).all()
    kept[:16384].zero_()


@pytest.mark.parametrize("call", ["attend", "append", "read"])
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_made_for_another_stream_have_memory_of_their_own(call, raw):
    """A call on a stream that waits for nothing: what it returns must not lie where the current stream's
    pending work still reads (memory that was given back there), nor may its memory go to the current stream's
    next tensor while the call has not run."""
    c = Case(83, [40, 70], [20, 30], 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    q, k, v = (c.rows(h).cuda() for h in (4, 2, 2))
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    run = {"attend": lambda: mmq.mmq_kv_attend(cache, batch, q, scale=0.1, stream=stream),
           "append": lambda: mmq.mmq_kv_append(cache, batch, k, v, q=q, stream=stream),
           "read": lambda: mmq.mmq_kv_read(cache, batch, stream=stream)[0]}[call]
    first = run()  # (workspaces and modules are there)
    clean()
    first = first.clone()
    shape = first.shape
    held = torch.full(shape, 3.0, device="cuda")
    copy = torch.empty_like(held)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # 0.1 s
    copy.copy_(held)
    del held
    run()
    side.synchronize()
    torch.cuda.synchronize()
    assert (copy == 3.0).all()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    out = run()
    del out  # the call has not run yet
    mine = torch.full(shape, 5.0, device="cuda")
    clean()
    assert (mine == 5.0).all()
    out = run()
    side.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("dtype,rotary", [("f32", 64), ("bf16", 64), ("f16", 40)])
@pytest.mark.parametrize("news,lens,rows", [([30, 40, 5], [90, 40, 70], 65), ([1, 1, 1], [90, 89, 12], 89),
                                            ([90, 33, 8], [90, 33, 40], 1), ([3, 2, 2], [90, 64, 33], 32)])
def test_rows_past_the_rotation_tables_are_skipped(dtype, rotary, news, lens, rows):
    """The tables end inside a block, at its beginning, before a sequence's new tokens: the rows up to there
    are appended and turned, the others leave the cache and their row of q_out as they were."""
    c = Case(89 + rows, lens, news, 12, 2, 64, 32, dtype)
    q, k, v = (c.rows(h) for h in (12, 2, 2))
    cos, sin = tables(rows, rotary)
    cache, batch = c.upload()
    out = torch.full((c.T, 12, 64), 7.0, dtype=DT[dtype], device="cuda")
    mmq.mmq_kv_append(cache, batch, k.cuda(), v.cuda(), q=q.cuda(), rope=mmq.Rope(dev(cos), dev(sin)), q_out=out)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE
    ref, want = c.data.copy(), np.full(out.shape, 7.0, np.float32)
    for b, (n, m) in enumerate(zip(lens, news)):
        first, end = n - m, min(n, rows)
        for t in range(first, end):
            r = c.starts[b] + t - first
            for h in range(12):
                want[r, h] = kv_ref.rotate(q.float().numpy()[r, h], t, cos, sin, False)
        if end > first:
            kv_ref.append(ref, [c.starts[b], c.starts[b] + end - first], [end], c.table[b:b + 1], k.float().numpy(),
                          v.float().numpy(), 64, (cos, sin, False))
    assert np.array_equal(cache.data.cpu().numpy(), ref)
    assert torch.equal(out.cpu(), torch.from_numpy(want).to(DT[dtype]))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what,appended", [("page", (0, 1, 2)), ("length", (0, 2)), ("negative", (0, 2)), ("starts", (2,)),
                                           ("past tokens", (0, 1)), ("max_new", (2,))])
def test_what_is_out_of_range_is_all_that_is_skipped(what, new, appended):
    """Values out of range in device memory, one kind at a time: the sequences that are in order are appended and
    attended to, rows and records of the others keep what they held; of a wrong page, its own records alone."""
    c = Case(97, [90, 80, 70], [new] * 3, 4, 2, 64, 32, "f32")
    cache, batch = c.upload()
    q, k, v = (c.rows(h) for h in (4, 2, 2))
    starts, lens, table = c.starts.copy(), list(c.lens), c.table.copy()
    if what == "page":
        table[1, 2] = c.pages
    elif what == "length":
        lens[1] = table.shape[1] * 32 + 1
    elif what == "negative":
        lens[1] = -1
    elif what == "starts":
        starts[1] = 3 * new + 5
    elif what == "past tokens":
        starts[3] = 3 * new + 1
    else:
        starts[1] = 0  # sequence 1 has twice as many
    batch.starts.copy_(torch.from_numpy(starts))
    batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    batch.table.copy_(torch.from_numpy(table))
    turned, out, lse = (torch.full(s, 9.0, device="cuda") for s in (q.shape, q.shape, q.shape[:2]))
    mmq.mmq_kv_append(cache, batch, k.cuda(), v.cuda(), q=q.cuda(), q_out=turned)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE
    mmq.mmq_kv_attend(cache, batch, q.cuda(), scale=0.1, out=out, lse=lse)
    torch.cuda.synchronize()
    assert mmq.mmq_get_device_error() == MMQ_ERR_RANGE
    ref = np.concatenate([c.data, c.data[:1]])  # one more page takes what the wrong one would
    at = np.zeros(c.T, bool)
    for b in appended:
        kv_ref.append(ref, [starts[b], starts[b + 1]], [lens[b]], table[b:b + 1], k.numpy(), v.numpy(), 64)
        at[starts[b]:starts[b + 1]] = True
    ref = ref[:c.pages]
    assert np.array_equal(cache.data.cpu().numpy(), ref)
    assert torch.equal(turned[at].cpu(), q[at]) and (turned[~at] == 9.0).all()
    assert (out[~at] == 9.0).all() and (lse[~at] == 9.0).all()
    for b in appended:
        if what == "page" and b == 1:
            continue
        one = Case.__new__(Case)
        one.data, one.starts, one.lens, one.table, one.D, one.dt = ref, [0, new], [lens[b]], table[b:b + 1], 64, "f32"
        rows = slice(starts[b], starts[b + 1])
        compare_attend(one, out[rows], lse[rows], q[rows], 0.1)


def test_outputs_made_in_a_capture_of_a_named_stream():
    """A call on a stream that is joined to the current one's capture, its output made by the call."""
    c = Case(101, [900, 70], [1, 2], 8, 2, 128, 64, "f16")
    cache, batch = c.upload()
    q = c.rows(8)
    qd, side = q.cuda(), torch.cuda.Stream()
    mmq.mmq_kv_attend(cache, batch, qd, scale=0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        first = mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        del first
        out = mmq.mmq_kv_attend(cache, batch, qd, scale=0.1, stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        kept = out + 0
    for _ in range(2):
        kept.zero_()
        graph.replay()
        clean()
        compare_attend(c, kept, None, q, 0.1)
