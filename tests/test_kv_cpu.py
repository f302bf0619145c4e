"""The key/value cache without a GPU: record sizes, the refusals of its C entry points (nothing is
launched, so any aligned address stands for device memory), and the reference the GPU tests compare
with, pinned by values worked by hand."""
import ctypes

import numpy as np
import pytest

import kv_ref

mmq = pytest.importorskip("block_quantized_int8_mmq_gb300")
torch = pytest.importorskip("torch")
from block_quantized_int8_mmq_gb300 import kv  # noqa: E402

SHAPE, NULL, ALIGN, ARG = -1, -3, -4, -9
A = 1 << 20  # a 16-byte aligned address


def call(fn, **change):
    """One of the entries on well-formed arguments but for `change`."""
    f = dict(data=A, pages=4, page=64, heads=2, dim=128, starts=A, lens=A, table=A, table_stride=8, seqs=1, tokens=0,
             max_new=1, table_pages=8, dtype=0, k=A, v=A, q=A, ts=512, hs=128, q_heads=4, cos=A, sin=A, rows=64,
             rotary=128, q_out=A, out=A, lse=A, ws=A, ws_bytes=1 << 40, scale=0.1, window=0, cache=True, batch=True)
    f.update(change)
    L = mmq.lib()
    c = kv._Cache(f["data"], f["pages"], f["page"], f["heads"], f["dim"])
    b = kv._Batch(f["starts"], f["lens"], f["table"], f["table_stride"], f["seqs"], f["tokens"], f["max_new"],
                  f["table_pages"])
    rows = [kv._Rows(f[n], f["ts"], f["hs"]) for n in "kvq"]
    rope = kv._Rope(f["cos"], f["sin"], f["rows"], f["rotary"], 0)
    p = ctypes.addressof
    head = (p(c) if f["cache"] else None, p(b) if f["batch"] else None, f["dtype"])
    if fn == "append":
        return L.mmq_kv_append(*head, p(rows[0]), p(rows[1]), p(rows[2]), f["q_heads"], p(rope), f["q_out"], None)
    if fn == "read":
        return L.mmq_kv_read(*head, f["k"], f["v"], None)
    return L.mmq_kv_attend(*head, p(rows[2]), f["q_heads"], f["scale"], f["window"], f["out"], f["lse"], f["ws"],
                           f["ws_bytes"], None)


def test_sizes():
    assert [mmq.mmq_kv_block_bytes(d) for d in (64, 128, 256)] == [4112, 8208, 16400]
    assert mmq.mmq_kv_block_bytes(96) == mmq.mmq_kv_block_bytes(0) == mmq.mmq_kv_block_bytes(-64) == 0
    assert mmq.mmq_kv_workspace_bytes(128) > 4096 and mmq.mmq_kv_workspace_bytes(100) == 0
    assert mmq.mmq_status_string(-11) == "MMQ_ERR_RANGE"


@pytest.mark.parametrize("fn", ["append", "read", "attend"])
def test_no_tokens_is_no_work(fn):
    assert call(fn) == 0
    assert call(fn, k=None, v=None, q=None, out=None, q_out=None) == 0
    assert call(fn, tokens=5, seqs=0, starts=None, lens=None, table=None) == 0


@pytest.mark.parametrize("fn", ["append", "read", "attend"])
@pytest.mark.parametrize("change,status", [
    (dict(cache=False), NULL), (dict(batch=False), NULL), (dict(data=None), NULL), (dict(data=A + 8), ALIGN),
    (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(page=48), SHAPE), (dict(page=0), SHAPE), (dict(heads=0), SHAPE),
    (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(seqs=-1), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(max_new=-1), SHAPE), (dict(table_pages=-1), SHAPE), (dict(table_stride=7), SHAPE),
    (dict(table_pages=1 << 25, table_stride=1 << 25), SHAPE), (dict(starts=None), NULL), (dict(lens=None), NULL),
    (dict(table=None), NULL), (dict(lens=A + 2), ALIGN), (dict(dtype=3), ARG), (dict(dtype=-1), ARG)])
def test_refusals_of_the_cache_and_the_batch(fn, change, status, capfd):
    assert call(fn, **change) == status
    assert "mmq_kv_" + fn in capfd.readouterr().err


@pytest.mark.parametrize("fn,change,status", [
    ("append", dict(k=None, tokens=1), NULL), ("append", dict(v=None, tokens=1), NULL),
    ("append", dict(k=A + 8), ALIGN), ("append", dict(ts=514), ALIGN), ("append", dict(hs=130), ALIGN),
    ("append", dict(dtype=1, hs=132), ALIGN), ("append", dict(q_heads=3), SHAPE), ("append", dict(q_heads=0), SHAPE),
    ("append", dict(q_out=None, tokens=1), NULL), ("append", dict(q_out=A + 4), ALIGN),
    ("append", dict(rotary=132), SHAPE), ("append", dict(rotary=12), SHAPE), ("append", dict(cos=None), NULL),
    ("append", dict(sin=A + 4), ALIGN), ("read", dict(k=None, tokens=1), NULL), ("read", dict(v=A + 8), ALIGN),
    ("attend", dict(q=None, tokens=1), NULL), ("attend", dict(out=None, tokens=1), NULL), ("attend", dict(out=A + 8), ALIGN),
    ("attend", dict(lse=A + 2), ALIGN), ("attend", dict(ws=None), NULL), ("attend", dict(ws=A + 16), ALIGN),
    ("attend", dict(ws_bytes=4096), SHAPE), ("attend", dict(scale=0.0), ARG), ("attend", dict(scale=-1.0), ARG),
    ("attend", dict(scale=float("nan")), ARG), ("attend", dict(scale=float("inf")), ARG), ("attend", dict(window=-1), ARG),
    ("attend", dict(q_heads=3), SHAPE)])
def test_refusals_of_each_call(fn, change, status, capfd):
    assert call(fn, **change) == status
    assert "mmq_kv_" + fn in capfd.readouterr().err


def test_handles_refuse_host_tensors():
    with pytest.raises(ValueError):
        mmq.KVCache(torch.zeros((1, 1, 1, 8208), dtype=torch.uint8))
    with pytest.raises(ValueError):
        mmq.KVBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                    torch.zeros((1, 1), dtype=torch.int32), 0, 0)
    with pytest.raises(ValueError):
        mmq.Rope(torch.zeros(4, 4), torch.zeros(4, 4))
    with pytest.raises(ValueError):
        mmq.KVCache.empty(1, 1, 96)


def test_reference_append_by_hand():
    """Two tokens into a block that keeps one: 127 * 2 and -254 against an older code 100 at scale 1."""
    dim = 64
    data = np.zeros((1, 1, 1, kv_ref.rec_bytes(dim)), np.uint8)
    kc, vc, d = kv_ref.split(data[0, 0, 0], dim)
    kc[0, :3] = (100, -127, 1)
    d[:] = (1.0, 4.0)
    vc[0, 0] = 5
    vc[1:] = 77  # rows that are not the sequence's
    k, v = np.zeros((2, 1, dim), np.float32), np.zeros((2, 1, dim), np.float32)
    k[0, 0, 0], k[1, 0, 1] = 254.0, -3.0
    v[1, 0, 2] = 508.0
    kv_ref.append(data, [0, 2], [3], np.array([[0]]), k, v, dim)
    assert d.tolist() == [2.0, 4.0]
    assert kc[0, :3].tolist() == [50, -64, 0]  # 100 / 2, rint(-63.5) to even, rint(0.5) to even
    assert kc[1, 0] == 127 and kc[2, 1] == -2  # rint(-1.5) to even
    assert vc[0, 0] == 5 and vc[2, 2] == 127 and (vc[3:] == 77).all()


def test_reference_attention_by_hand():
    """One key twice as likely as the other: out = (2 v0 + v1) / 3, lse = ln 3 with s = (ln 2, 0)."""
    dim = 64
    data = np.zeros((1, 1, 1, kv_ref.rec_bytes(dim)), np.uint8)
    kc, vc, d = kv_ref.split(data[0, 0, 0], dim)
    kc[0, 0] = 100
    vc[0, 0], vc[1, 1] = 3, 6
    d[:] = (0.01, 1.0)
    q = np.zeros((2, 1, dim))
    q[:, 0, 0] = np.log(2.0) / (100 * float(np.float32(0.01)))
    out, lse, _, _ = kv_ref.attend(data, [0, 2], [2], np.array([[0]]), q, dim, 1.0)
    assert np.allclose(out[1, 0, :2], [2.0, 2.0], atol=1e-12) and np.isclose(lse[1, 0], np.log(3.0))
    assert np.allclose(out[0, 0, :2], [3.0, 0.0])
    out, _, _, _ = kv_ref.attend(data, [0, 2], [2], np.array([[0]]), q, dim, 1.0, window=1)
    assert np.allclose(out[1, 0, :2], [0.0, 6.0])


def test_reference_rotation_is_a_rotation():
    cos, sin = np.float32([[1, 1], [0, 0.6]]), np.float32([[0, 0], [1, 0.8]])
    x = np.float32([1, 2, 3, 4, 5])
    assert np.allclose(kv_ref.rotate(x, 1, cos, sin, False), [-3, 2 * 0.6 - 4 * 0.8, 1, 4 * 0.6 + 2 * 0.8, 5])
    assert np.allclose(kv_ref.rotate(x, 1, cos, sin, True), [-2, 1, 3 * 0.6 - 4 * 0.8, 4 * 0.6 + 3 * 0.8, 5])
    assert kv_ref.rotate(x, 0, cos, sin, True).tolist() == x.tolist()


class OnDevice:
    """A tensor's outside on GPU 1: what a call looks at before it launches."""
    device, is_cuda = torch.device("cuda", 1), True

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A

    def numel(self):
        return 1 << 40


class Launches:
    """The library with its launching entries replaced by a note of the call."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(mmq.lib(), name)
        return lambda *a: self.calls.append(name) or 0


@pytest.mark.parametrize("current", [0, 1])
def test_a_cache_of_another_device_is_refused(current, monkeypatch):
    """The library launches on the current device, whatever stream and addresses it gets."""
    from types import SimpleNamespace as S
    cache, batch = S(device=OnDevice.device, heads=2, dim=64, _p=0), S(device=OnDevice.device, tokens=3, _p=0)
    k, q, ws = OnDevice(3, 2, 64), OnDevice(3, 4, 64), OnDevice(1 << 20, dtype=torch.uint8)
    fake = Launches()
    monkeypatch.setattr(kv, "_lib", fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    calls = [lambda: kv.mmq_kv_append(cache, batch, k, k, q=q, q_out=q, stream=0),
             lambda: kv.mmq_kv_append(cache, batch, k, k, stream=0),
             lambda: kv.mmq_kv_read(cache, batch, k_out=k, v_out=k, stream=0),
             lambda: kv.mmq_kv_attend(cache, batch, q, out=q, workspace=ws, stream=0)]
    for call in calls:
        if current == 1:
            call()
        else:
            with pytest.raises(ValueError, match="current device"):
                call()
    assert len(fake.calls) == (4 if current == 1 else 0)


def test_workspaces_are_zeroed_behind_their_own_device(monkeypatch):
    """After a call that gave up, every device that has a workspace is waited for, not the current one alone."""
    log = []

    class Space:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

        def __getitem__(self, part):
            return self

        def zero_(self):
            log.append(("zero", self.device.index))

    def synchronize(device=None):
        log.append(("wait", 0 if device is None else torch.device(device).index))

    monkeypatch.setattr(torch.cuda, "synchronize", synchronize)
    monkeypatch.setattr(kv, "_workspaces", {(i, 0, 64): Space(i) for i in (1, 0)})
    kv._clean_workspaces()
    for i in (0, 1):
        at = log.index(("zero", i))
        assert ("wait", i) in log[:at] and ("wait", i) in log[at:]


@pytest.mark.parametrize("change", [dict(seqs=1 << 24, heads=1 << 14, q_heads=1 << 14, page=32, table_pages=1 << 25),
                                    dict(seqs=1 << 24, heads=32766, q_heads=32766, page=1 << 20, table_pages=1 << 10),
                                    dict(seqs=1 << 23, heads=4, page=64, table_pages=4)])
def test_more_records_than_can_be_numbered_are_refused(change, capfd):
    """2^63 of them, close to 2^64, 2^28: past and within 64 bits, the last one is taken."""
    big = change["seqs"] > 1 << 23
    assert call("attend", table_stride=change["table_pages"], **change) == (SHAPE if big else 0)
    assert ("2^31" in capfd.readouterr().err) == big


def grown(steps, dim=128, seed=3):
    """One block of 32 normal tokens, appended steps[i] at a time, token t times size(t): what was put in, what the
    cache holds after each step, and the key scales that the block has had."""
    rng = np.random.default_rng(seed)

    def fill(size):
        x = (rng.normal(0, 1, (32, 1, dim)) * np.array([size(t) for t in range(32)])[:, None, None]).astype(np.float32)
        data, table, n, scales = np.zeros((1, 1, 1, kv_ref.rec_bytes(dim)), np.uint8), np.array([[0]]), 0, []
        for m in steps:
            kv_ref.append(data, [0, m], [n + m], table, x[n:n + m], x[n:n + m], dim)
            n += m
            scales.append(float(kv_ref.split(data[0, 0, 0], dim)[2][0]))
        return x, kv_ref.values(data, table, 0, n, dim, 0), scales

    return fill


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


@pytest.mark.parametrize("size", [lambda t: 1.0, lambda t: 1.0 + 7.0 * t / 31])
def test_what_a_block_rounds_away(size):
    """A token is rounded under its block's scale, by half a step at most, and once more by half of the new step
    whenever the scale grows; a rounding's deviation is step / sqrt(12)."""
    x, got, scales = grown([32])(size)
    assert np.abs(got - x).max() <= scales[0] / 2 * (1 + 1e-5)
    assert rms(got - x) <= 1.1 * scales[0] / np.sqrt(12)
    x, got, scales = grown([1] * 32)(size)
    for t in range(32):
        seen = sorted(set(scales[t:]))
        assert np.abs(got[t] - x[t]).max() <= sum(seen) / 2 * (1 + 1e-5)
        assert rms(got[t] - x[t]) <= 1.5 * np.sqrt(sum(d * d for d in seen) / 12)


def test_rejected_drafts_leave_their_scale_and_a_new_append_of_the_block_takes_it_back():
    """Four drafts of eight times the size behind 20 tokens, then the sequence goes on from token 20: the block keeps
    the drafts' scale, and its older tokens are rounded under it.  Appended once more from the block's beginning,
    with what the cache held before the drafts, they are what they were."""
    dim, table = 128, np.array([[0]])
    rng = np.random.default_rng(7)
    x, drafts, more = (rng.normal(0, s, (n, 1, dim)).astype(np.float32) for n, s in ((20, 1.0), (4, 8.0), (12, 1.0)))
    data = np.zeros((1, 1, 1, kv_ref.rec_bytes(dim)), np.uint8)
    kv_ref.append(data, [0, 20], [20], table, x, x, dim)
    before = [kv_ref.values(data, table, 0, 20, dim, w, np.float32) for w in (0, 1)]
    small = float(kv_ref.split(data[0, 0, 0], dim)[2][0])
    kv_ref.append(data, [0, 4], [24], table, drafts, drafts, dim)
    large = float(kv_ref.split(data[0, 0, 0], dim)[2][0])
    assert large > 6 * small
    left = data.copy()
    kv_ref.append(left, [0, 12], [32], table, more, more, dim)
    assert float(kv_ref.split(left[0, 0, 0], dim)[2][0]) == np.float32(large)
    off = kv_ref.values(left, table, 0, 20, dim, 0) - x
    assert np.abs(off).max() <= (small + large) / 2 * (1 + 1e-5)
    assert 0.8 * large / np.sqrt(12) <= rms(off) <= 1.2 * large / np.sqrt(12)
    kv_ref.append(data, [0, 32], [32], table, np.concatenate([before[0], more]), np.concatenate([before[1], more]), dim)
    scale = float(kv_ref.split(data[0, 0, 0], dim)[2][0])
    assert scale <= 1.3 * small
    assert rms(kv_ref.values(data, table, 0, 20, dim, 0) - x) <= 1.5 * np.sqrt((small ** 2 + scale ** 2) / 12)
