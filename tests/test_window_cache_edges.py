"""Calls at the edges of the windowed attention and the 4-bit cache: tokens that were never written, row counts
past the grid's 32 bits, extreme numbers, the shared list of units, other devices."""
import ctypes

import numpy as np
import pytest
import torch

from recurrent_memory_transformer_anti_b200 import rmt
from test_window_cache import TORCH, Setup, attend_ref, check_attention, decode_ref, encode_ref, f64, normal, visible

gpu = pytest.mark.gpu


# ------------------------------------------------------------ tokens that nobody sees, never written

HALF = [  # dh, H, Hkv, lens, n_q, window, sinks; at most 32 units an item, and more
    (64, 8, 2, [300, 0, 70], 1, 100, 0), (64, 8, 2, [300, 40], 1, 100, 5), (32, 4, 2, [333], 3, 90, 70),
    (128, 4, 2, [300, 129], 2, 77, 1), (128, 16, 1, [500], 1, 33, 33), (64, 12, 1, [1000, 200], 5, 1, 3),
    (64, 8, 2, [5000, 300, 0], 1, 3001, 0), (64, 8, 1, [5000, 5], 3, 2900, 70), (32, 4, 2, [5100], 2, 2999, 3),
    (128, 4, 2, [2500, 1700], 2, 1300, 37), (128, 24, 2, [2600], 3, 1500, 1)]


@gpu
@pytest.mark.parametrize("fill", [0xFF, 0xF8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,H,Hkv,lens,n_q,window,sinks", HALF)
def test_cache_attention_needs_no_tokens_that_no_row_sees(cuda_ok, dtype, dh, H, Hkv, lens, n_q, window, sinks, fill):
    """Only the sinks and what the rows' windows reach are ever written; every other byte of the pages stands for
    NaN (0xFF) or infinity (0xF8) where it is a scale."""
    n, M = len(lens), max(lens)
    s = Setup(lens, Hkv, dh, seed=n, fill=fill)
    k, v = (normal(70 + i, (n, M, Hkv * dh), dtype) for i in (0, 1))  # row t: token t
    first = [max(0, t - n_q - window + 1) for t in lens]
    rows = max(t - f for t, f in zip(lens, first))
    newest = [torch.zeros(n, max(rows, 1), Hkv * dh, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    for b in range(n):
        for x, src in zip(newest, (k, v)):
            x[b, :lens[b] - first[b]] = src[b, first[b]:lens[b]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rmt.rmt_cache_write(s.cache, *newest, max(rows, 1), n_new=i32([t - f for t, f in zip(lens, first)]), dtype=dtype)
    if sinks:
        head = i32([min(sinks, t) for t in lens])
        c = rmt.rmt_cache(s.pages, s.table, head, Hkv, dh)
        rmt.rmt_cache_write(c, k[:, :sinks].contiguous(), v[:, :sinks].contiguous(), min(sinks, M), n_new=head, dtype=dtype)
    q = normal(72, (n, n_q, H * dh), dtype)
    got = f64(s.attend(q, n_q, H, window, sinks, dtype))
    rmt.rmt_sync(None)
    held = [decode_ref(*encode_ref(f64(x).reshape(n, M, Hkv, dh))) for x in (k, v)]
    for b in range(n):
        kk, vv = (x[b, :lens[b]] for x in held)
        ref = attend_ref(f64(q)[b].reshape(n_q, H, dh), kk, vv, np.arange(lens[b] - n_q, lens[b]), window, sinks)
        check_attention(got[b].reshape(n_q, H, dh), ref, np.abs(vv).max() if vv.size else 0.0, dtype)


# ------------------------------------------------------------------------- many rows in one call

@gpu
def test_cache_rows_whose_threads_pass_32_bits(cuda_ok):
    """A padded batch of 34 (written) and 17 (read) sequences of 2^23 rows, of which each has three: 16 and 8 rows a
    CTA, 256 threads a CTA, so that sequences from 32 and 16 on begin behind thread 2^32."""
    dh, M, n, new = 128, 2 ** 23, 34, 3
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * n * M * dh + 2 ** 32:
        pytest.skip("needs 77 GB")
    x = torch.empty(n, M, dh, dtype=torch.bfloat16, device="cuda")
    x[:, :new] = normal(1, (n, new, dh), "bf16")
    codes, byte = encode_ref(f64(x[:, :new]))
    s = Setup([5] * n, 1, dh, fill=0xA5)
    n_new = torch.full((n,), new, dtype=torch.int32, device="cuda")
    rmt.rmt_cache_write(s.cache, x, x, M, n_new=n_new)
    rmt.rmt_sync(None)
    parts, page = s.halves(), s.table.cpu().numpy()[:, 0]
    for i in (0, 2):
        np.testing.assert_array_equal(parts[i][page, 0, 2:5], codes[..., 0::2] | (codes[..., 1::2] << 4))
        np.testing.assert_array_equal(parts[i + 1][page, 0, 2:5], byte)
    x[:, :new + 1] = -77.0
    half = n // 2
    first = rmt.rmt_cache(s.pages, s.table[:half].contiguous(), s.lens[:half].contiguous(), 1, dh)
    rmt.rmt_cache_read(first, x[:half], x[half:], M, n_new=n_new)
    rmt.rmt_sync(None)
    for got in (x[:half], x[half:]):
        np.testing.assert_array_equal(f64(got[:, :new]), decode_ref(codes, byte)[:half])
        assert (got[:, new] == -77.0).all()
    del x, got
    torch.cuda.empty_cache()


def test_more_rows_than_any_device_holds_are_refused():
    c = rmt.rmt_cache_struct(256, 256, 256, 4, 2 ** 10, 2, 4096, 128)
    lib = rmt.lib()
    for fn in (lib.rmt_cache_write, lib.rmt_cache_read):
        for M in (2 ** 8 + 1, 2 ** 20):
            assert fn(ctypes.byref(c), 256, 256, 4096 * 128, M, None, 1, None) == rmt.RMT_EINVAL
            assert "2^37" in rmt.rmt_last_error()


# ------------------------------------------------------------------------------ what rmt_sync reports

def met_bad_page(device="cuda", stream=None):
    """Reads a row through a table entry that is no page."""
    table, lens = (torch.full(sh, val, dtype=torch.int32, device=device) for sh, val in (((1, 1), 9), ((1,), 1)))
    c = rmt.rmt_cache(torch.zeros(4608, dtype=torch.uint8, device=device), table, lens, 1, 64)
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=device)
    torch.cuda.synchronize(device)
    rmt.rmt_cache_read(c, k, k.clone(), 1, stream=stream)


def sync_error(stream=None):
    with pytest.raises(rmt.RmtError) as e:
        rmt.rmt_sync(None, stream=stream)
    rmt.rmt_sync(None, stream=stream)  # the word was cleared
    return e.value


@gpu
def test_sync_reports_on_the_stream_it_is_given(cuda_ok):
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream()):
        met_bad_page(stream=stream)
        assert sync_error(stream).status == rmt.RMT_EINVAL
    for handle in (0, 1, 2):  # NULL, cudaStreamLegacy, cudaStreamPerThread
        met_bad_page(stream=handle)
        assert sync_error(handle).status == rmt.RMT_EINVAL


@gpu
def test_sync_reports_what_a_device_met_that_is_not_the_current_one(cuda_ok):
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    with torch.cuda.device(0):
        stream = torch.cuda.Stream(1)
        met_bad_page("cuda:1", stream)
        rmt.rmt_sync(None)  # device 0 met nothing
        assert sync_error(stream).status == rmt.RMT_EINVAL
        met_bad_page("cuda:1", torch.cuda.default_stream(1))
        assert sync_error(torch.cuda.default_stream(1)).status == rmt.RMT_EINVAL


@gpu
def test_sync_names_every_fault_of_the_word(cuda_ok):
    met_bad_page()
    rmt.rmt_wait_selftest(100)
    e = sync_error()
    assert e.status == rmt.RMT_ETIMEOUT
    assert "wait gave up" in str(e) and "page table entry" in str(e)


# ------------------------------------------------------------------------------------ devices

class On:
    """A host tensor that says it is on another device (the calls are refused, or reach a fake library)."""

    def __init__(self, t, device):
        self.t, self.device = t, device

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.t, name)


class FakeLibrary:
    """Notes the calls that reach the library."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


def streaming_calls(at):
    """name -> (call, names of its tensors); at(name, tensor) gives the tensor as a call sees it."""
    i32, bf = torch.int32, torch.bfloat16
    pages, table, lens = at("pages", torch.zeros(2 * 4608, dtype=torch.uint8)), at("page_table", torch.zeros(2, 1, dtype=i32)), \
        at("lens", torch.zeros(2, dtype=i32))
    rows = {n: at(n, torch.zeros(2, 3, 64, dtype=bf)) for n in ("k", "v", "q", "out")}
    n_new, ws = at("n_new", torch.zeros(2, dtype=i32)), at("workspace", torch.zeros(1 << 16, dtype=torch.uint8))
    qkv = at("qkv", torch.zeros(2, 3, 192, dtype=bf))
    cache = lambda: rmt.rmt_cache(pages, table, lens, 1, 64)
    held = ("pages", "page_table", "lens")
    return {
        "write": (lambda: rmt.rmt_cache_write(cache(), rows["k"], rows["v"], 3, n_new=n_new), held + ("k", "v", "n_new")),
        "read": (lambda: rmt.rmt_cache_read(cache(), rows["k"], rows["v"], 3, n_new=n_new), held + ("k", "v", "n_new")),
        "attention": (lambda: rmt.rmt_attention_cache(cache(), rows["q"], rows["out"], 3, 1, 0, 0, ws),
                      held + ("q", "out", "workspace")),
        "window": (lambda: rmt.rmt_attention_window(qkv, rows["out"], 2, 3, 1, 1, 64, 0, lens=lens), ("qkv", "out", "lens"))}


@pytest.mark.parametrize("call", ["write", "read", "attention", "window"])
def test_tensors_on_another_device_or_the_host_are_refused(monkeypatch, call):
    fake = FakeLibrary()
    fake.rmt_cache_page_bytes = rmt.lib().rmt_cache_page_bytes
    monkeypatch.setattr(rmt, "_lib", fake)
    run, names = streaming_calls(lambda name, t: On(t, 0))[call]
    run()
    assert len(fake.calls) == 1
    for other in (-1, 1):
        for bad in names:
            run, _ = streaming_calls(lambda name, t: On(t, other if name == bad else 0))[call]
            with pytest.raises(ValueError):
                run()
    assert len(fake.calls) == 1


@pytest.mark.parametrize("call", ["write", "read", "attention", "window"])
@pytest.mark.parametrize("device", [0, 3])
def test_calls_go_to_the_current_stream_of_their_tensors_device(monkeypatch, call, device):
    fake = FakeLibrary()
    fake.rmt_cache_page_bytes = rmt.lib().rmt_cache_page_bytes
    monkeypatch.setattr(rmt, "_lib", fake)
    monkeypatch.setattr(rmt, "_current_stream", lambda d: 7000 + d)
    streaming_calls(lambda name, t: On(t, device))[call][0]()
    (name, args), = fake.calls
    assert args[-1] == 7000 + device


def test_sync_on_another_devices_default_stream_makes_that_device_current(monkeypatch):
    seen = []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("enter", self.device))

        def __exit__(self, *a):
            seen.append(("exit", self.device))

    class Library:
        def rmt_sync(self, h, stream):
            seen.append((h, stream))
            return 0

    monkeypatch.setattr(torch.cuda, "device", Current)
    monkeypatch.setattr(rmt, "_lib", Library())
    stream = type("Stream", (), dict(device=torch.device("cuda", 3), cuda_stream=0))()
    rmt.rmt_sync(None, stream=stream)
    assert seen == [("enter", stream.device), (None, 0), ("exit", stream.device)]


# ------------------------------------------------------------------------------- extreme queries

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,T,n_q", [(64, 300, 1), (64, 5000, 1), (64, 5000, 5), (128, 300, 3), (128, 4000, 1), (32, 5000, 2)])
def test_cache_attention_of_queries_whose_scores_pass_fp32(cuda_ok, dtype, dh, T, n_q):
    """Queries near the type's end: scores up to 10^41, of either sign. All the weight is one key's, or equal keys'."""
    H, Hkv = 6, 2
    s = Setup([T], Hkv, dh)
    k = torch.full((1, T, Hkv, dh), 4.0, device="cuda")
    k[:, T // 3] = 7.0  # the largest score of positive queries
    k[:, T // 2] = 0.25  # the least negative of negative ones
    k[:, :, 1] *= torch.linspace(0.5, 2.0, T, device="cuda")[None, :, None]
    v = normal(5, (1, T, Hkv * dh), "f32")
    rmt.rmt_cache_write(s.cache, k.reshape(1, T, -1), v, T, dtype="f32")
    gain = torch.tensor([3e38, -3e38, 2e36, -3e38, 3e38, -1e37], device="cuda")
    q = gain[None, None, :, None].expand(1, n_q, H, dh).to(TORCH[dtype]).reshape(1, n_q, -1).contiguous()
    got = f64(s.attend(q, n_q, H, 0, 0, dtype))
    rmt.rmt_sync(None)
    (kk, vv), = s.values()
    ref = attend_ref(f64(q)[0].reshape(n_q, H, dh), kk, vv, np.arange(T - n_q, T), 0, 0)
    check_attention(got[0].reshape(n_q, H, dh), ref, np.abs(vv).max(), dtype)


# --------------------------------------------------- bounds that one term of 16 bits does not meet

def attend_and_bound(q, k, v, i, window, sinks, score, key, total, floor=0.0):
    """The formula in 64 bits and how far a result may be off it, for rows of every head of one sequence.

    A score s_j = sum_c q_c k_jc / sqrt(dh) that is off by `score` of a_j = sum_c |q_c k_jc| / sqrt(dh), and a weight that
    is off by `key` of itself, move the result by at most sum_j p_j |v_j - out| (score a_j + key) to first order (1%
    on top for the rest). Sums of weights and of weighted values, each off by `total` of the sum of its terms'
    magnitudes, add 2 total sum_j p_j |v_j|. Weights that are also off by `floor` of the largest one, however small they
    are themselves, add floor sum_j |v_j - out|: the largest is at most 1 of their sum."""
    rows, H, dh = q.shape
    Hkv = k.shape[1]
    seen = visible(i, np.arange(k.shape[0]), window, sinks)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(H):
        kh, vh = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
        for r in range(rows):
            at = np.nonzero(seen[r])[0]
            if at.size == 0:
                continue
            s, a = kh[at] @ q[r, h] / np.sqrt(dh), np.abs(kh[at]) @ np.abs(q[r, h]) / np.sqrt(dh)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[r, h] = o = p @ vh[at]
            tol[r, h] = 1.01 * ((p * (score * a + key)) @ np.abs(vh[at] - o)) + 2 * total * (p @ np.abs(vh[at])) + \
                floor * np.abs(vh[at] - o).sum(0)
    return out, tol


def cache_bounds(dh, dtype, units, items):
    """score, key and total above for the cache kernel, and the result's own rounding.

    Operands: fp32 queries and weights as two f16 terms (2^-22 of a value). f16's smallest step is 2^-24: a weight's last term
    rounds by up to 2^-25 while the largest is held at 2^7 or more, so every weight, down to those that become 0, is off by
    up to 2^-32 of the largest (`floor`); a query's by 2^-35 of the row's largest, in the 4 of `score`. A tensor
    core's step sums 16 products; a step is taken to lose 2^-22 of its terms' magnitudes. dh / 16 steps a
    score (twice with two terms), 4 a unit of 64 keys, the units of a warp after one another, the parts of an item after those.
    The exponential is off by 2^-22, its argument's two roundings by 2^-23 of the scores' size, in `score`
    since a_j >= |s_j|, twice for a reference that was raised. bf16: weights are f16 (2^-11 of a value), and their sum
    takes them as rounded; the result is bf16 (2^-8)."""
    f32 = dtype == "f32"
    terms = 2 if f32 else 1
    steps = terms * 4 * -(-units * items // (8 * 148)) + units
    return dict(score=(terms * dh / 16 + f32 + 4) * 2.0 ** -22, key=2.0 ** -22 + (2.0 ** -22 if f32 else 2.0 ** -11),
                total=steps * 2.0 ** -22, floor=2.0 ** -32), 2.0 ** -24 if f32 else 2.0 ** -8


def window_bounds(dh, n):
    """The same for the fp32 window kernel, n the most keys a row sees: dh FMA a score, the query's scale two roundings,
    the difference from the maximum one of at most twice a_j; exp2 two units of its last place; n terms a sum, in tiles
    whose maxima change the earlier ones by another such weight and product (one tile in 64 keys, and one for the sinks)."""
    u = 2.0 ** -24
    return dict(score=(dh + 2 + 2 + 1) * u, key=4 * u, total=(n + 6 * (n // 64 + 2)) * u), u


def check_bounds(got, ref, tol, rounding):
    err = np.abs(got - ref)
    ok = err <= tol + rounding * np.abs(ref)
    assert np.isfinite(got).all() and ok.all(), (float(err.max()), float((err / np.maximum(tol, 1e-300)).max()))


@gpu
@pytest.mark.parametrize("dh,T", [(64, 40), (64, 9), (128, 40), (32, 50), (64, 130)])
def test_fp32_cache_attention_carries_more_than_one_f16_term(cuda_ok, dh, T):
    H, Hkv, n_q = 16, 4, 4
    s = Setup([T], Hkv, dh)
    s.fill(81)
    q = normal(82, (1, n_q, H * dh), "f32") * 2
    got = f64(s.attend(q, n_q, H, 0, 0, "f32"))
    rmt.rmt_sync(None)
    (k, v), = s.values()
    units = -(-T // (32 if dh == 128 else 64))
    bounds, rounding = cache_bounds(dh, "f32", units, 8)
    ref, tol = attend_and_bound(f64(q)[0].reshape(n_q, H, dh), k, v, np.arange(T - n_q, T), 0, 0, **bounds)
    check_bounds(got[0].reshape(n_q, H, dh), ref, tol, rounding)


@gpu
@pytest.mark.parametrize("dh,M,window,sinks", [(64, 200, 60, 3), (128, 150, 0, 0), (32, 300, 64, 64), (64, 130, 1, 2)])
def test_fp32_window_attention_carries_fp32(cuda_ok, dh, M, window, sinks):
    H, Hkv = 6, 2
    qkv = normal(83, (2, M, (H + 2 * Hkv) * dh), "f32")
    out = torch.zeros(2, M, H * dh, device="cuda")
    rmt.rmt_attention_window(qkv, out, 2, M, H, Hkv, dh, window, sinks, dtype="f32")
    rmt.rmt_sync(None)
    bounds, rounding = window_bounds(dh, min(M, window + sinks) if window else M)
    for g in range(2):
        q, k, v = (t.reshape(M, -1, dh) for t in np.split(f64(qkv)[g], [H * dh, (H + Hkv) * dh], axis=1))
        ref, tol = attend_and_bound(q, k, v, np.arange(M), window, sinks, **bounds)
        check_bounds(f64(out)[g].reshape(M, H, dh), ref, tol, 3 * rounding)


# --------------------------------------------------------------- the list of units that all share

SHARED = [  # dh, H, Hkv, lens, n_q, window, sinks, max_pages: more than 32 units an item can have
    (64, 8, 2, [5000, 300, 0, 2100], 1, 0, 0, None), (64, 32, 8, [5000, 4097, 64], 1, 3001, 70, None),
    (64, 12, 2, [5000, 0, 33], 2, 2999, 70, None), (64, 8, 2, [4200, 5000], 3, 0, 0, None),
    (64, 16, 2, [4800], 5, 3000, 1, None), (64, 6, 1, [2500, 1, 3000], 64, 2100, 130, None),
    (32, 8, 2, [5000, 70], 1, 3001, 70, None), (32, 8, 2, [5000], 4, 0, 0, None), (32, 8, 1, [0, 4000, 3], 5, 2200, 64, None),
    (128, 8, 2, [3000, 129, 0], 1, 1500, 70, None), (128, 4, 1, [2500, 1400], 3, 1301, 33, None),
    (128, 16, 2, [2200], 5, 0, 0, None), (64, 8, 8, [100, 0, 1, 64, 65], 1, 0, 0, 400), (128, 8, 2, [40, 257], 2, 0, 0, 300),
    (64, 8, 2, [5000, 5000, 5000, 5000, 5000] * 8, 1, 4000, 4, None)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,H,Hkv,lens,n_q,window,sinks,max_pages", SHARED)
def test_cache_attention_of_long_items_equals_the_formula(cuda_ok, dtype, dh, H, Hkv, lens, n_q, window, sinks, max_pages):
    s = Setup(lens, Hkv, dh, seed=len(lens), max_pages=max_pages)
    s.fill(91)
    n, rows = len(lens), n_q * (H // Hkv)
    q = normal(92, (n, n_q, H * dh), dtype) * 2
    got = f64(s.attend(q, n_q, H, window, sinks, dtype))
    rmt.rmt_sync(None)
    tok = 32 if dh == 128 else 64
    units = max(lens) // tok + 1
    tiles = -(-rows // (16 if dtype == "bf16" and rows > 8 else 8))
    held = s.values()
    for b in range(0, n, max(1, n // 5)):
        k, v = held[b]
        pos = np.arange(lens[b] - n_q, lens[b])
        bounds, rounding = cache_bounds(dh, dtype, units, n * Hkv * tiles)
        ref, tol = attend_and_bound(f64(q)[b].reshape(n_q, H, dh), k, v, pos, window, sinks, **bounds)
        check_bounds(got[b].reshape(n_q, H, dh), ref, tol, rounding)
        assert not got[b].reshape(n_q, -1)[pos < 0].any()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,group,T,n_q,window,sinks", [
    (64, 1, 900, 2, 300, 70), (64, 4, 5000, 2, 3001, 70), (64, 4, 5000, 3, 2900, 64), (128, 2, 700, 1, 301, 33),
    (128, 4, 3000, 3, 1700, 31), (32, 4, 5000, 5, 2950, 129), (32, 1, 600, 1, 70, 1)])
def test_each_visible_token_and_no_other_decides(cuda_ok, dtype, dh, group, T, n_q, window, sinks):
    """A key/value head for each token at a border, whose key outweighs all others where it is visible."""
    lo = T - n_q - window + 1  # the first row's oldest key
    at = [0, sinks - 1, sinks, lo - 1, lo, lo + n_q - 1, lo + 64 - lo % 64, T - n_q, T - 1, T - 2]
    Hkv = len(at)
    H = group * Hkv
    s = Setup([T], Hkv, dh)
    sign = torch.sign(normal(93, (Hkv, dh), "f32"))
    k = normal(94, (1, T, Hkv, dh), "f32") * 0.3
    for h, t in enumerate(at):
        k[0, t, h] = 4 * sign[h]
    v = normal(95, (1, T, Hkv * dh), "f32")
    rmt.rmt_cache_write(s.cache, k.reshape(1, T, -1), v, T, dtype="f32")
    q = (12.0 / dh ** 0.5 * sign).repeat_interleave(group, 0)[None, None].expand(1, n_q, H, dh)
    q = q.to(TORCH[dtype]).reshape(1, n_q, -1).contiguous()
    got = f64(s.attend(q, n_q, H, window, sinks, dtype))[0].reshape(n_q, H, dh)
    rmt.rmt_sync(None)
    (kk, vv), = s.values()
    pos = np.arange(T - n_q, T)
    tiles = -(-n_q * group // (16 if dtype == "bf16" and n_q * group > 8 else 8))
    bounds, rounding = cache_bounds(dh, dtype, T // (32 if dh == 128 else 64) + 1, Hkv * tiles)
    ref, tol = attend_and_bound(f64(q)[0].reshape(n_q, H, dh), kk, vv, pos, window, sinks, **bounds)
    check_bounds(got, ref, tol, rounding)
    seen = visible(pos, np.array(at), window, sinks)
    for h in range(H):
        near = np.abs(got[:, h] - vv[at[h // group], h // group]).max(-1) < 0.05
        np.testing.assert_array_equal(near, seen[:, h // group])


# ------------------------------------------------------------------------ graphs and the debug build

@gpu
def test_two_captured_graphs_that_share_a_workspace(cuda_ok):
    """Long items (two kernels and the workspace) captured twice with other queries; replayed in turn after the lengths
    grow, each gives what an eager call gives."""
    dh, H, Hkv, lens = 64, 8, 2, [4500, 0, 700]
    s = Setup([t + 8 for t in lens], Hkv, dh, max_pages=80)
    s.fill(3, "bf16")
    s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    qs = [normal(i, (3, 2, H * dh), "bf16") for i in (1, 2)]
    outs = [torch.zeros_like(q) for q in qs]
    ws = torch.empty(rmt.rmt_attention_cache_workspace(s.cache, 2, H, 0, 0), dtype=torch.uint8, device="cuda")
    run = lambda q, o: rmt.rmt_attention_cache(s.cache, q, o, 2, H, 0, 0, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(qs[0], outs[0])
    torch.cuda.synchronize()
    graphs = []
    for q, o in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(q, o)
    for step in range(3):
        s.lens.add_(torch.tensor([1, step, 2], dtype=torch.int32, device="cuda"))
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        got = [o.clone() for o in outs]
        for q, o, x in zip(qs, outs, got):
            run(q, o)
            rmt.rmt_sync(None)
            assert torch.equal(o, x) and torch.isfinite(x).all() and x[0].any()


@gpu
def test_streaming_operators_of_the_debug_build(cuda_ok):
    """The library compiled with -DRMT_DEBUG, in a child process, over cases of every kernel."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    assert os.path.exists(rmt.DEBUG_LIB_PATH)
    cases = ["test_write_and_read_equal_the_formula", "test_cache_attention_equals_the_formula",
             "test_window_attention_equals_the_formula", "test_many_sequences"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        *[f"tests/test_window_cache.py::{c}" for c in cases]], cwd=root, capture_output=True, text=True,
                       timeout=600, env=dict(os.environ, RMT_LIBRARY=rmt.DEBUG_LIB_PATH))
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]


@gpu
@pytest.mark.parametrize("dh,group,n,longest", [(64, 2, 1200, 2048), (64, 5, 2500, 2047), (128, 4, 1300, 1024), (32, 1, 3000, 1000)])
def test_more_short_items_than_warps_can_share(cuda_ok, dh, group, n, longest):
    """Whole items that one or two warps of a CTA take alone, of up to 32 units, several after one another."""
    lens = [(i * 37) % 90 if i % 40 else longest - i // 40 for i in range(n)]
    s = Setup(lens, 1, dh)
    s.fill(3, "bf16")
    q = normal(4, (n, 1, group * dh), "bf16")
    got = f64(s.attend(q, 1, group, 0, 0, "bf16"))
    rmt.rmt_sync(None)
    held = s.values()
    bounds, rounding = cache_bounds(dh, "bf16", 32, 8 * 148)  # a warp may have all 32 units of an item
    for b in list(range(0, n, 200)) + list(range(7, n, 97)) + [n - 1]:
        k, v = held[b]
        ref, tol = attend_and_bound(f64(q[b]).reshape(1, group, dh), k, v, np.array([lens[b] - 1]), 0, 0, **bounds)
        check_bounds(got[b].reshape(1, group, dh), ref, tol, rounding)
