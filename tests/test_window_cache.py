"""Windowed attention with sinks and the 4-bit key/value cache: against plain numpy in 64 bits, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

from recurrent_memory_transformer_anti_b200 import rmt

PAGE = rmt.RMT_CACHE_PAGE
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
gpu = pytest.mark.gpu


# ------------------------------------------------------------------- the formulas, in numpy

# the numbers a scale byte stands for: 5 exponent bits, 3 mantissa bits, steps of 2^-17 below 2^-14
SCALES = np.array([(b % 8) * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(226)])


def encode_ref(x):
    """[..., dh] -> (codes q + 8, scale bytes), in 64 bits."""
    x = np.where(np.isnan(x), 0.0, x).astype(np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    want = np.minimum(np.abs(blocks).max(-1), 64512.0) / 7
    dist = np.abs(want[..., None] - SCALES)
    near = dist == dist.min(-1, keepdims=True)
    first = near.argmax(-1)
    last = near.shape[-1] - 1 - near[..., ::-1].argmax(-1)
    byte = np.where(first % 2 == 0, first, last)  # one candidate, or two neighbours: the even one
    s = SCALES[byte][..., None]
    q = np.where(s > 0, np.rint(blocks / np.where(s > 0, s, 1.0)), 0.0)
    return (np.clip(q, -7, 7) + 8).astype(np.uint8).reshape(x.shape), byte.astype(np.uint8)


def decode_ref(codes, byte):
    q = codes.astype(np.float64) - 8
    return (q.reshape(*q.shape[:-1], q.shape[-1] // 16, 16) * SCALES[byte][..., None]).reshape(q.shape)


def visible(i, j, window, sinks):
    ok = j[None] <= i[:, None]
    return ok & ((i[:, None] - j[None] < window) | (j[None] < sinks)) if window else ok


def attend_ref(q, k, v, i, window, sinks):
    """q [rows, H, dh], k and v [keys, Hkv, dh] at positions 0.., rows at positions i -> [rows, H, dh]."""
    rows, H, dh = q.shape
    Hkv = k.shape[1]
    seen = visible(i, np.arange(k.shape[0]), window, sinks)
    out = np.zeros(q.shape)
    for h in range(H):
        kh, vh = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
        for r in range(rows):
            at = np.nonzero(seen[r])[0]
            if at.size == 0:
                continue
            s = kh[at] @ q[r, h] / np.sqrt(dh)
            p = np.exp(s - s.max())
            out[r, h] = p @ vh[at] / p.sum()
    return out


def f64(t):
    return t.detach().double().cpu().numpy()


# Largest error of an attention output against the formula. bf16: the result's own rounding (2^-8 of
# it) and the rounding of every softmax weight to 16 bits (at most 2^-8 of it for bf16 weights; the
# weights of a row sum to 1, so at most 2^-8 max|v|). fp32: weights and queries carry 22 bits or
# more, and a sum of up to 2^12 terms in fp32 loses at most 2^-24 * 2^9 per 2^3 terms taken at once.
def check_attention(got, ref, vmax, dtype):
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * vmax if dtype == "bf16" else 2.0 ** -14 * vmax
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and (err <= tol).all(), float((err - tol).max())


def normal(seed, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(TORCH[dtype])


class Setup:
    """A cache whose pages are handed out in random order and filled with `fill` bytes."""

    def __init__(self, lens, Hkv, dh, seed=0, fill=0xFF, spare=2, max_pages=None):
        self.lengths, self.Hkv, self.dh = list(lens), Hkv, dh
        n = len(self.lengths)
        per = max_pages or max(1, (max(self.lengths) + PAGE - 1) // PAGE)
        used = n * per + spare
        order = np.random.default_rng(seed).permutation(used)[:n * per].reshape(n, per)
        self.table = torch.tensor(order.astype(np.int32), device="cuda")
        self.pages = torch.full((used, Hkv, 72 * dh), fill, dtype=torch.uint8, device="cuda")
        self.lens = torch.tensor(np.array(self.lengths, np.int32), device="cuda")
        self.cache = rmt.rmt_cache(self.pages, self.table, self.lens, Hkv, dh)

    def halves(self):
        """Numpy views of the pages: codes and scale bytes of keys, then of values."""
        p = self.pages.cpu().numpy()
        c, s = 32 * self.dh, 4 * self.dh
        cut = np.split(p, [c, c + s, 2 * c + s], axis=-1)
        shape = p.shape[:2]
        return [x.reshape(*shape, PAGE, -1) for x in cut]

    def values(self):
        """What the cache holds for each sequence: lists of (keys, values) [len, Hkv, dh] in 64 bits."""
        parts = self.halves()
        out = []
        table = self.table.cpu().numpy()
        for b, T in enumerate(self.lengths):
            t = np.arange(T)
            page, row = table[b, t // PAGE], t % PAGE
            kv = []
            for i in (0, 2):
                packed = parts[i][page, :, row]
                codes = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], self.dh)
                kv.append(decode_ref(codes, parts[i + 1][page, :, row]))
            out.append(kv)
        return out

    def fill(self, seed, dtype="f32"):
        """Write every token of every sequence (in one call), return what was written."""
        M = max(self.lengths)
        k, v = (normal(seed + s, (len(self.lengths), M, self.Hkv * self.dh), dtype) for s in (0, 1))
        rmt.rmt_cache_write(self.cache, k, v, M, n_new=self.lens, dtype=dtype)
        rmt.rmt_sync(None)
        return k, v

    def attend(self, q, n_q, H, window, sinks, dtype, stream=None, workspace=None):
        out = torch.full((len(self.lengths), n_q, H * self.dh), float("nan"), dtype=TORCH[dtype], device="cuda")
        if workspace is None:
            size = rmt.rmt_attention_cache_workspace(self.cache, n_q, H, window, sinks)
            workspace = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
        rmt.rmt_attention_cache(self.cache, q, out, n_q, H, window, sinks, workspace, dtype=dtype, stream=stream)
        return out


# --------------------------------------------------------------------- write and read back

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,Hkv,lens,new", [
    (64, 8, [1], [1]), (64, 8, [130, 64, 1, 0, 65], [1, 1, 1, 1, 1]), (64, 2, [200, 77, 63], [200, 13, 63]),
    (128, 3, [129, 5, 640], [129, 0, 131]), (32, 1, [64, 3], [64, 3]), (128, 1, [1, 2, 3], [1, 1, 1]),
    (64, 5, [0, 0], [0, 0])])
def test_write_and_read_equal_the_formula(cuda_ok, dtype, dh, Hkv, lens, new):
    s = Setup(lens, Hkv, dh, fill=0xA5)
    M, n = max(max(new), 1), len(lens)
    ld = (3 + 2 * Hkv) * dh  # rows inside packed q, k, v rows
    qkv = normal(7, (n, M, ld), dtype) * torch.exp(normal(8, (n, M, 1), "f32") * 3).to(TORCH[dtype])
    k, v = qkv[..., 3 * dh:(3 + Hkv) * dh], qkv[..., (3 + Hkv) * dh:]
    n_new = torch.tensor(new, dtype=torch.int32, device="cuda")
    before = [x.copy() for x in s.halves()]
    rmt.rmt_cache_write(s.cache, k, v, M, n_new=n_new, dtype=dtype)
    ko, vo = (torch.full((n, M, Hkv * dh), -77.0, dtype=TORCH[dtype], device="cuda") for _ in range(2))
    rmt.rmt_cache_read(s.cache, ko, vo, M, n_new=n_new, dtype=dtype)
    rmt.rmt_sync(None)
    after, want = s.halves(), before
    table = s.table.cpu().numpy()
    refs = [np.full((n, M, Hkv * dh), -77.0) for _ in range(2)]
    for half, x in ((0, f64(k)), (2, f64(v))):
        x = x.reshape(n, M, Hkv, dh)
        for b in range(n):
            for i in range(min(new[b], lens[b])):
                i0 = i + max(0, new[b] - lens[b])
                pos = lens[b] - new[b] + i0
                codes, byte = encode_ref(x[b, i0])
                want[half][table[b, pos // PAGE], :, pos % PAGE] = codes[..., 0::2] | (codes[..., 1::2] << 4)
                want[half + 1][table[b, pos // PAGE], :, pos % PAGE] = byte
                refs[half // 2][b, i0] = decode_ref(codes, byte).reshape(-1)
    for got, ref in zip(after, want):  # the written rows, and every other byte as it was
        np.testing.assert_array_equal(got, ref)
    np.testing.assert_array_equal(f64(ko), refs[0])
    np.testing.assert_array_equal(f64(vo), refs[1])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_of_special_values_and_ties(cuda_ok, dtype):
    dh, rows = 64, []
    inf, nan = float("inf"), float("nan")
    base = np.linspace(-1.0, 1.0, dh)
    for f in (0.0, 1.0, 7 * 2.0 ** -18, 7 * 2.0 ** -17, 3e-5, 4e-4, 64512.0, 7e4, 3e38, 1e-30):
        rows.append(base * f)
    for x in (inf, -inf, nan):
        r = base * 3
        r[5], r[40] = x, x
        rows.append(r)
    rows.append(np.full(dh, nan))
    # every multiple of half a step: ties to even, and the scales' own ties (amax / 7 between two bytes)
    for amax in (7.0, 7 * 1.0625, 7 * 1.1875, 7 * 0.53125, 7 * 9216.0, 7 * 2.0 ** -15 * 1.0625):
        rows.append(np.resize(np.concatenate(([amax], np.arange(-7.5, 7.75, 0.5) * amax / 7)), dh))
    r = np.random.default_rng(3)
    rows += list(r.standard_normal((64, dh)) * np.exp2(r.integers(-20, 14, (64, 1))))
    x = torch.tensor(np.array(rows), dtype=torch.float32).to(TORCH[dtype]).cuda()[None]
    if dtype == "f32":  # neighbours of ties, one step of fp32 away
        y = x.clone()
        y.view(torch.int32)[...] += torch.randint(-1, 2, y.shape, device="cuda", dtype=torch.int32)
        x = torch.cat((x, torch.where(torch.isfinite(x), y, x)), 1)
    M = x.shape[1]
    s = Setup([M], 1, dh)
    rmt.rmt_cache_write(s.cache, x, x, M, dtype=dtype)
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    rmt.rmt_cache_read(s.cache, ko, vo, M, dtype=dtype)
    rmt.rmt_sync(None)
    want = decode_ref(*encode_ref(f64(x)))
    np.testing.assert_array_equal(f64(ko), want)
    np.testing.assert_array_equal(f64(vo), want)


@gpu
@pytest.mark.parametrize("Hkv", [4, 2])
def test_write_and_read_of_every_bf16_as_a_blocks_largest(cuda_ok, Hkv):
    """Each non-negative bf16 but NaN as the largest of 16 channels, the others at halves of its steps and between;
    the same rows again and again until a launch takes several heads a warp."""
    dh, per = 128, Hkv * 8
    r = np.random.default_rng(5)
    top = torch.arange(0x7F81, dtype=torch.int16).view(torch.bfloat16).double().numpy()
    top = np.concatenate((top, np.full(-len(top) % per, 1.0)))
    scale = SCALES[encode_ref(np.repeat(top, 16)[None])[1][0]]
    q = np.concatenate((np.arange(-7, 8) + 0.5 * r.choice([-1, 1], 15), [0.0]))[:15]
    x = np.concatenate((top[:, None], scale[:, None] * (q + r.choice([0.0, 0.25], (len(top), 15)))), 1)
    x[:, 1:] = np.clip(x[:, 1:], -top[:, None], top[:, None])
    x = torch.tensor(x.reshape(1, -1, Hkv * dh)).bfloat16()
    want = decode_ref(*encode_ref(x.double().numpy()))[0]
    rows = x.shape[1]
    times = -(-20000 // rows)
    k = x.cuda().repeat(1, times, 1)
    v = k.flip(1)
    M = k.shape[1]
    s = Setup([M], Hkv, dh)
    rmt.rmt_cache_write(s.cache, k, v, M)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    rmt.rmt_cache_read(s.cache, ko, vo, M)
    rmt.rmt_sync(None)
    for got in (ko[0], vo[0].flip(0)):
        np.testing.assert_array_equal(f64(got[:rows]), want)
        assert torch.equal(got.view(times, rows, -1), got[:rows].expand(times, -1, -1))


@gpu
def test_lengths_and_pages_that_do_not_fit_are_reported_and_skipped(cuda_ok):
    dh, Hkv, H = 64, 2, 4
    s = Setup([130, 64, 100], Hkv, dh, fill=0)
    s.fill(1)
    good = s.attend(normal(5, (3, 1, H * dh), "bf16"), 1, H, 0, 0, "bf16")
    rmt.rmt_sync(None)
    q = normal(5, (3, 1, H * dh), "bf16")
    keep = s.table.clone(), s.lens.clone()
    pages = s.pages.clone()
    k = normal(9, (3, 1, Hkv * dh), "bf16")
    for bad in (lambda: s.table[1].fill_(10 ** 6), lambda: s.table[1].fill_(-1), lambda: s.lens[1:2].fill_(10 ** 6),
                lambda: s.lens[1:2].fill_(2 ** 31 - 1)):
        bad()
        for call in (lambda: rmt.rmt_cache_write(s.cache, k, k, 1), lambda: rmt.rmt_cache_read(s.cache, k, k, 1)):
            call()
            with pytest.raises(rmt.RmtError) as e:
                rmt.rmt_sync(None)
            assert e.value.status == rmt.RMT_EINVAL
        s.pages.copy_(pages)
        out = s.attend(q, 1, H, 0, 0, "bf16")
        with pytest.raises(rmt.RmtError) as e:
            rmt.rmt_sync(None)
        assert e.value.status == rmt.RMT_EINVAL
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])  # the other sequences
        assert torch.isfinite(out).all()
        s.table.copy_(keep[0])
        s.lens.copy_(keep[1])
    rmt.rmt_sync(None)
    s.lens[1:2].fill_(-5)  # as an empty slot
    out = s.attend(q, 1, H, 0, 0, "bf16")
    rmt.rmt_sync(None)
    assert (out[1] == 0).all() and torch.equal(out[0], good[0])


# --------------------------------------------------------------- attention over the cache

DECODE = [  # dh, H, Hkv, lens, n_q, window, sinks
    (64, 8, 2, [1], 1, 0, 0), (64, 32, 8, [64, 65, 63, 0, 200], 1, 0, 0), (64, 4, 4, [700], 1, 0, 0),
    (128, 16, 4, [1500, 3, 128], 1, 0, 0), (128, 6, 2, [257, 90], 3, 0, 0), (32, 4, 1, [70, 129], 2, 0, 0),
    (32, 3, 1, [500], 1, 40, 3), (64, 16, 1, [333, 40], 1, 0, 0), (64, 24, 1, [333, 40], 5, 0, 0),
    (128, 40, 2, [200, 1], 2, 0, 0), (64, 8, 1, [4000], 1, 1, 0), (64, 8, 1, [4000, 30], 1, 100, 4),
    (64, 8, 2, [2000, 64, 128, 1], 4, 64, 64), (128, 8, 2, [1000, 500], 3, 65, 130), (64, 2, 1, [3, 2, 1], 5, 0, 0),
    (64, 2, 1, [3, 900], 5, 2, 1), (128, 64, 1, [300], 1, 0, 0), (64, 7, 7, [150] * 9, 1, 0, 0)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,H,Hkv,lens,n_q,window,sinks", DECODE)
def test_cache_attention_equals_the_formula(cuda_ok, dtype, dh, H, Hkv, lens, n_q, window, sinks):
    s = Setup(lens, Hkv, dh, seed=len(lens))  # rows behind a sequence's end: bytes that stand for NaN
    s.fill(11)
    wide = normal(12, (len(lens), n_q, H * dh + 64), dtype)  # strided rows
    q = wide[..., :H * dh]
    out = s.attend(q, n_q, H, window, sinks, dtype)
    rmt.rmt_sync(None)
    got = f64(out)
    for b, (k, v) in enumerate(s.values()):
        ref = attend_ref(f64(q)[b].reshape(n_q, H, dh), k, v, np.arange(lens[b] - n_q, lens[b]), window, sinks)
        vmax = np.abs(v).max() if v.size else 0.0
        check_attention(got[b].reshape(n_q, H, dh), ref, vmax, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_attention_of_large_and_small_numbers(cuda_ok, dtype):
    """Scores far apart, rows of queries from 1e-30 to 1e30, values from 1e-3 to 6e4."""
    dh, H, Hkv, T = 64, 8, 2, 300
    s = Setup([T], Hkv, dh)
    k = normal(1, (1, T, Hkv * dh), "f32") * 4
    v = normal(2, (1, T, Hkv * dh), "f32") * torch.exp(normal(3, (1, T, 1), "f32") * 3)
    v[0, 100, 3] = 6e4
    rmt.rmt_cache_write(s.cache, k, v, T, dtype="f32")
    q = normal(4, (1, 1, H * dh), dtype)
    gain = torch.tensor([1.0, 5.0, 1e-30, 1e-3, 20.0, 1e30, 0.0, 0.3], device="cuda").repeat_interleave(dh)
    q = (q.float() * gain).to(TORCH[dtype])
    out = f64(s.attend(q, 1, H, 0, 0, dtype))
    rmt.rmt_sync(None)
    (kk, vv), = s.values()
    ref = attend_ref(f64(q)[0].reshape(1, H, dh), kk, vv, np.array([T - 1]), 0, 0)
    check_attention(out[0].reshape(1, H, dh)[:, [0, 1, 2, 3, 4, 6, 7]], ref[:, [0, 1, 2, 3, 4, 6, 7]],
                    np.abs(vv).max(), dtype)
    # at 1e30 a score's rounding decides between keys only if two are that close: one key has all the weight
    check_attention(out[0].reshape(1, H, dh)[:, [5]], ref[:, [5]], np.abs(vv).max(), dtype)


@gpu
@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("f32", 64), ("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("which", ["keys", "values"])
def test_cache_attention_of_the_largest_and_smallest_scales(cuda_ok, dtype, dh, which):
    """Blocks up to the format's ends (scales 8192 and 9216, 2^-17), of both signs, in one of 2000 tokens."""
    H, Hkv, T = 4, 1, 2000
    for size in (6.4e4, 3e4, 1e-4, 6e-5):
        s = Setup([T], Hkv, dh)
        kv = [normal(i, (1, T, dh), "f32") for i in (1, 2)]
        x = kv[which == "values"]
        if size > 1:
            x[0, 1234] *= size / x[0, 1234].abs().max()
        else:
            x *= size / 3
        rmt.rmt_cache_write(s.cache, *kv, T, dtype="f32")
        q = normal(4, (1, 1, H * dh), dtype)
        if which == "keys":
            q = (q.float() * (3.0 / size)).to(TORCH[dtype])
        out = f64(s.attend(q, 1, H, 0, 0, dtype))
        rmt.rmt_sync(None)
        (k, v), = s.values()
        if size > 1 and which == "values":
            assert s.halves()[3].max() == 0xFF and np.abs(v).max() >= 0.9 * size
        ref = attend_ref(f64(q)[0].reshape(1, H, dh), k, v, np.array([T - 1]), 0, 0)
        check_attention(out[0].reshape(1, H, dh), ref, np.abs(v).max(), dtype)


@gpu
def test_cache_attention_of_queries_that_are_not_finite(cuda_ok):
    s = Setup([100], 1, 64)
    s.fill(1)
    q = normal(2, (1, 2, 4 * 64), "bf16")
    want = s.attend(q, 2, 4, 0, 0, "bf16").reshape(2, 4, 64)
    q[0, 1, 70] = float("nan")
    q[0, 0, 200] = float("inf")
    got = s.attend(q, 2, 4, 0, 0, "bf16").reshape(2, 4, 64)
    rmt.rmt_sync(None)
    for i, h in ((1, 1), (0, 3)):
        assert torch.isnan(got[i, h]).all()
        got[i, h] = want[i, h]
    assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("lens", [[700], [5000]])
def test_cache_attention_of_a_row_does_not_depend_on_the_other_rows(cuda_ok, lens):
    """Other heads' queries, and another token's, change: the row's bits do not."""
    dh, H, Hkv = 64, 8, 2
    s = Setup(lens, Hkv, dh)
    s.fill(61, "bf16")
    q = normal(62, (1, 2, H, dh), "bf16")
    want = s.attend(q.reshape(1, 2, -1), 2, H, 0, 0, "bf16").reshape(2, H, dh)
    for t, h in ((0, 0), (1, 5), (1, 7)):
        x = q * 40
        x[0, t, h] = q[0, t, h]
        got = s.attend(x.reshape(1, 2, -1), 2, H, 0, 0, "bf16").reshape(2, H, dh)
        rmt.rmt_sync(None)
        assert torch.equal(got[t, h], want[t, h])
        assert not torch.equal(got, want)


@gpu
@pytest.mark.parametrize("n_q,window", [(1, 0), (2, 100)])
def test_rows_of_unused_slots_give_zeros_whatever_they_hold(cuda_ok, n_q, window):
    s = Setup([0, 3000, 1], 1, 64)
    s.fill(1)
    q = normal(2, (3, n_q, 4 * 64), "bf16")
    want = s.attend(q, n_q, 4, window, 0, "bf16")
    q[0] = float("nan")
    q[2, :n_q - 1] = float("inf")
    got = s.attend(q, n_q, 4, window, 0, "bf16")
    rmt.rmt_sync(None)
    assert torch.equal(got, want) and not got[0].any() and not got[2, :n_q - 1].any()


@gpu
@pytest.mark.parametrize("n", [255, 256, 257, 700])
def test_many_sequences(cuda_ok, n):
    """More sequences than a CTA has threads, lengths from 0 to 2500: each result is the one-sequence call's."""
    lens = [(i * 37) % 90 if i % 50 else 2500 - i for i in range(n)]
    s = Setup(lens, 1, 64)
    s.fill(3, "bf16")
    q = normal(4, (n, 1, 2 * 64), "bf16")
    got = f64(s.attend(q, 1, 2, 0, 0, "bf16"))
    rmt.rmt_sync(None)
    vals = s.values()
    for b in list(range(0, n, 7)) + list(range(0, n, 50)) + [n - 1]:
        k, v = vals[b]
        ref = attend_ref(f64(q)[b].reshape(1, 2, 64), k, v, np.array([lens[b] - 1]), 0, 0)
        check_attention(got[b].reshape(1, 2, 64), ref, np.abs(v).max() if v.size else 0.0, "bf16")


@gpu
def test_cache_offsets_past_32_bits(cuda_ok):
    dh, Hkv, H = 128, 8, 16
    page = rmt.rmt_cache_page_bytes(Hkv, dh)
    n = 2 ** 32 // page + 40
    pages = torch.empty(n * page, dtype=torch.uint8, device="cuda")
    outs = []
    for first in (0, n - 3):
        table = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None].contiguous()
        lens = torch.tensor([150], dtype=torch.int32, device="cuda")
        c = rmt.rmt_cache(pages, table, lens, Hkv, dh)
        k, v = normal(1, (1, 150, Hkv * dh), "bf16"), normal(2, (1, 150, Hkv * dh), "bf16")
        rmt.rmt_cache_write(c, k, v, 150)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        rmt.rmt_cache_read(c, ko, vo, 150)
        ws = torch.empty(rmt.rmt_attention_cache_workspace(c, 1, H), dtype=torch.uint8, device="cuda")
        out = torch.zeros(1, 1, H * dh, dtype=torch.bfloat16, device="cuda")
        rmt.rmt_attention_cache(c, normal(3, (1, 1, H * dh), "bf16"), out, 1, H, 0, 0, ws)
        rmt.rmt_sync(None)
        outs.append((ko, vo, out))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and a.abs().max() > 0


# ---------------------------------------------------------------------- windowed attention

WINDOW = [  # dh, H, Hkv, G, M, lens, window, sinks
    (64, 4, 1, 2, 1, None, 5, 2), (64, 8, 2, 2, 130, None, 0, 0), (64, 4, 2, 1, 300, None, 64, 4),
    (64, 4, 4, 1, 129, None, 1, 0), (64, 4, 4, 1, 140, None, 1, 1), (64, 6, 2, 3, 261, [261, 0, 130], 100, 7),
    (64, 8, 1, 2, 700, [700, 33], 33, 300), (128, 4, 1, 1, 333, None, 200, 16), (128, 3, 1, 2, 257, [200, 257], 0, 0),
    (128, 2, 2, 1, 513, None, 128, 128), (32, 4, 2, 2, 150, [1, 150], 40, 3), (64, 20, 1, 1, 100, None, 30, 9),
    (64, 40, 2, 1, 65, None, 0, 5), (64, 16, 1, 1, 400, None, 256, 0), (128, 8, 1, 1, 384, [383], 383, 1),
    (64, 5, 1, 2, 290, None, 131, 8), (64, 2, 1, 1, 1100, None, 1040, 3), (128, 12, 4, 1, 200, None, 1000, 1000),
    (64, 32, 8, 3, 333, [333, 0, 67], 90, 70), (128, 16, 2, 2, 300, [300, 17], 129, 5), (32, 24, 6, 3, 333, None, 77, 33)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,H,Hkv,G,M,lens,window,sinks", WINDOW)
def test_window_attention_equals_the_formula(cuda_ok, dtype, dh, H, Hkv, G, M, lens, window, sinks):
    qkv = normal(21, (G, M, (H + 2 * Hkv) * dh), dtype)
    dev = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    lens = lens or [M] * G
    clean = qkv.clone()
    for g in range(G):  # rows behind the end hold what no row may see
        qkv[g, lens[g]:] = float("nan")
    out = torch.full((G, M, H * dh), -77.0, dtype=TORCH[dtype], device="cuda")
    rmt.rmt_attention_window(qkv, out, G, M, H, Hkv, dh, window, sinks, lens=dev, dtype=dtype)
    rmt.rmt_sync(None)
    got, x = f64(out), f64(clean)
    for g in range(G):
        T = lens[g]
        assert (got[g, T:] == -77.0).all()
        k = x[g, :T, H * dh:(H + Hkv) * dh].reshape(T, Hkv, dh)
        v = x[g, :T, (H + Hkv) * dh:].reshape(T, Hkv, dh)
        ref = attend_ref(x[g, :T, :H * dh].reshape(T, H, dh), k, v, np.arange(T), window, sinks)
        check_attention(got[g, :T].reshape(T, H, dh), ref, np.abs(v).max() if T else 0.0, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dh", [64, 128])
def test_window_attention_keeps_masked_values_out(cuda_ok, dtype, bad, dh):
    """A key or value that is not finite reaches the rows that see it, and no others."""
    H, Hkv, M, window, sinks = 4, 2, 400, 90, 4
    qkv = normal(31, (1, M, (H + 2 * Hkv) * dh), dtype)
    run = lambda x: (rmt.rmt_attention_window(x, o := torch.zeros(1, M, H * dh, dtype=x.dtype, device="cuda"), 1, M, H,
                                              Hkv, dh, window, sinks, dtype=dtype), rmt.rmt_sync(None), o)[2]
    want = run(qkv).reshape(M, H, dh)
    for at in (0, 3, 4, 127, 128, 200, 399):
        for head in range(Hkv):
            for part in (H, H + Hkv):  # a key, a value
                x = qkv.clone()
                x[0, at, (part + head) * dh + 5] = bad
                got = run(x).reshape(M, H, dh)
                sees = visible(np.arange(M), np.array([at]), window, sinks)[:, 0]
                for h in range(H):
                    mine = torch.tensor(sees & (h // (H // Hkv) == head), device="cuda")
                    assert torch.equal(got[~mine, h], want[~mine, h]), (at, head, part, h)
                    if part > H or np.isnan(bad):
                        assert (~torch.isfinite(got[mine, h])).any(-1).all(), (at, head, part, h)


@gpu
@pytest.mark.parametrize("dtype,dh,sinks", [("bf16", 64, 0), ("bf16", 64, 4), ("bf16", 128, 0), ("bf16", 128, 4),
                                            ("f32", 64, 4)])
def test_window_attention_of_scores_that_rise_far_above_the_first(cuda_ok, dtype, dh, sinks):
    """Scores far above those of the first keys a row sees: by 2^184 in one head, by 2^20 with values near the
    type's end in another, by a little again and again in a third; the fourth has none of that."""
    H, Hkv, G, M, window = 8, 4, 2, 900, 300
    qkv = normal(51, (G, M, (H + 2 * Hkv) * dh), dtype).reshape(G, M, H + 2 * Hkv, dh)
    a = dh ** -0.5
    qkv[:, :, :6] = 8.0  # heads of the first three key heads: score 8 sqrt(dh) times a key's common value
    tok = torch.arange(M, device="cuda")
    up = lambda lo, hi: torch.where(tok < 420, lo, hi).to(qkv.dtype)[:, None]
    qkv[:, :, H] = up(-8 * a, 8 * a)  # -64 and 64
    qkv[:, :, H + 1] = up(0.0, 1.75 * a)  # 0 and 14
    qkv[:, :, H + Hkv + 1] *= 1e36
    qkv[:, :, H + 2] = (tok.to(qkv.dtype) / 32 * a)[:, None]  # a quarter of a unit per token
    qkv = qkv.reshape(G, M, -1)
    out = torch.zeros(G, M, H * dh, dtype=TORCH[dtype], device="cuda")
    rmt.rmt_attention_window(qkv, out, G, M, H, Hkv, dh, window, sinks, dtype=dtype)
    rmt.rmt_sync(None)
    got, x = f64(out).reshape(G, M, H, dh), f64(qkv).reshape(G, M, H + 2 * Hkv, dh)
    for g in range(G):
        ref = attend_ref(x[g, :, :H], x[g, :, H:H + Hkv], x[g, :, H + Hkv:], np.arange(M), window, sinks)
        for h in range(H):
            check_attention(got[g, :, h], ref[:, h], np.abs(x[g, :, H + Hkv + h // 2]).max(), dtype)


@gpu
@pytest.mark.parametrize("dh,M,G", [(64, 900, 8), (64, 6000, 8), (64, 700, 33), (128, 900, 8)])
def test_window_attention_of_many_sequences_whose_scores_rise(cuda_ok, dh, M, G):
    """The same sequence G times, every other one without its jump by 2^184, gives what it gives alone, to the bit;
    and again."""
    H, Hkv, window, sinks = 16, 8, 300, 2
    qkv = normal(53, (1, M, H + 2 * Hkv, dh), "bf16").repeat(2, 1, 1, 1)
    qkv[:, :, :H] = 8.0
    a = dh ** -0.5
    qkv[:, :, H:H + Hkv] = -8 * a
    qkv[0, M // 2:, H:H + Hkv:3] = 8 * a
    alone = []
    for x in qkv:
        out = torch.zeros(1, M, H * dh, dtype=torch.bfloat16, device="cuda")
        rmt.rmt_attention_window(x.reshape(1, M, -1), out, 1, M, H, Hkv, dh, window, sinks)
        alone.append(out)
    batch = qkv.reshape(2, M, -1)[torch.arange(G, device="cuda") % 2].contiguous()
    for _ in range(2):
        out = torch.zeros(G, M, H * dh, dtype=torch.bfloat16, device="cuda")
        rmt.rmt_attention_window(batch, out, G, M, H, Hkv, dh, window, sinks)
        rmt.rmt_sync(None)
        assert torch.isfinite(out).all()
        for g in range(G):
            assert torch.equal(out[g], alone[g % 2][0]), g


@gpu
@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("sinks", [0, 4])
def test_window_attention_keeps_a_rows_bits_whatever_later_scores_are(cuda_ok, dtype, dh, sinks):
    """Scores that rise by a quarter per token, and the same with a jump by 2^184 from token 420 on: the rows
    before it, in the same query tiles as rows that see it, come out alike to the bit."""
    H, Hkv, M, window = 4, 2, 700, 300
    qkv = normal(52, (1, M, H + 2 * Hkv, dh), dtype)
    a = dh ** -0.5
    tok = torch.arange(M, device="cuda")
    qkv[:, :, :H] = 8.0
    qkv[:, :, H:H + Hkv] = ((tok % 256).to(qkv.dtype) / 32 * a)[:, None, None]
    outs = []
    for jump in (0.0, 16.0):
        x = qkv.clone()
        x[:, 420:, H] += jump * a
        out = torch.zeros(1, M, H * dh, dtype=TORCH[dtype], device="cuda")
        rmt.rmt_attention_window(x.reshape(1, M, -1), out, 1, M, H, Hkv, dh, window, sinks, dtype=dtype)
        rmt.rmt_sync(None)
        assert torch.isfinite(out).all()
        outs.append(out.reshape(M, H, dh))
    assert torch.equal(outs[0][:420], outs[1][:420]) and torch.equal(outs[0][:, 2:], outs[1][:, 2:])


@gpu
@pytest.mark.parametrize("dtype,dh", [("bf16", 32), ("f32", 64), ("bf16", 64), ("bf16", 128), ("f32", 128)])
def test_window_attention_shows_a_value_that_is_not_finite_whatever_its_weight(cuda_ok, dtype, dh):
    """Token 7's weight is below 2^-1000 in every row but its own; its value is infinite."""
    H, M, window, sinks = 2, 150, 60, 2
    qkv = torch.zeros(1, M, 3 * H * dh, dtype=TORCH[dtype], device="cuda")
    qkv[..., :2 * H * dh] = 16.0
    qkv[0, 7, H * dh:2 * H * dh] = -16.0  # scores 256 sqrt(dh) and its negative, powers of e
    qkv[..., 2 * H * dh:] = normal(3, (1, M, H * dh), dtype)
    qkv[0, 7, 2 * H * dh + 3] = float("inf")  # head 0
    out = torch.zeros(1, M, H * dh, dtype=TORCH[dtype], device="cuda")
    rmt.rmt_attention_window(qkv, out, 1, M, H, H, dh, window, sinks, dtype=dtype)
    rmt.rmt_sync(None)
    fin = torch.isfinite(out.reshape(M, H, dh)).all(-1).cpu().numpy()
    sees = visible(np.arange(M), np.array([7]), window, sinks)[:, 0]
    np.testing.assert_array_equal(fin[:, 0], ~sees)
    assert fin[:, 1].all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_attention_of_large_and_small_queries(cuda_ok, dtype):
    H, Hkv, dh, M = 7, 1, 64, 300
    gain = torch.tensor([1.0, 1e-30, 20.0, 1e4, 1e8, 1e30, 0.0], device="cuda").repeat_interleave(dh)
    qkv = normal(61, (1, M, (H + 2 * Hkv) * dh), dtype).float()
    qkv[..., :H * dh] *= gain
    qkv = qkv.to(TORCH[dtype])
    out = torch.zeros(1, M, H * dh, dtype=TORCH[dtype], device="cuda")
    rmt.rmt_attention_window(qkv, out, 1, M, H, Hkv, dh, 100, 3, dtype=dtype)
    rmt.rmt_sync(None)
    x = f64(qkv)[0]
    q, k, v = (t.reshape(M, -1, dh) for t in np.split(x, [H * dh, (H + Hkv) * dh], axis=1))
    got, ref = f64(out).reshape(M, H, dh), attend_ref(q, k, v, np.arange(M), 100, 3)
    small, large = [0, 1, 2, 6], [3, 4, 5]
    check_attention(got[:, small], ref[:, small], np.abs(v).max(), dtype)
    # a score s in fp32 is off by at most 64 * 2^-24 of sum |q k|, so weights may differ where two scores
    # are that close: there the result lies between the values, elsewhere it is the formula's
    assert np.isfinite(got).all() and (np.abs(got) <= np.abs(v).max() * (1 + 2.0 ** -7)).all()
    for h in large:
        s = q[:, h] @ k[:, 0].T / 8
        s = np.where(visible(np.arange(M), np.arange(M), 100, 3), s, -np.inf)
        noise = (np.abs(q[:, h]) @ np.abs(k[:, 0]).T).max(1) / 8 * 64 * 2.0 ** -24
        top = np.sort(s, 1)
        clear = (noise < 2.0 ** -10) | (np.where(M > 1, top[:, -1] - top[:, -2], np.inf) > 2 * noise + 40)
        check_attention(got[clear, h], ref[clear, h], np.abs(v).max(), dtype)


@gpu
def test_window_attention_past_32_bits(cuda_ok):
    H, Hkv, dh, M = 64, 16, 128, 360000
    qkv = torch.zeros(2, M, (H + 2 * Hkv) * dh, dtype=torch.bfloat16, device="cuda")
    x = normal(5, (150, (H + 2 * Hkv) * dh), "bf16")
    qkv[:, :150] = x
    qkv[1, -1] = x[0]
    out = torch.zeros(2, M, H * dh, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([150, 150], dtype=torch.int32, device="cuda")
    rmt.rmt_attention_window(qkv, out, 2, M, H, Hkv, dh, 50, 3, lens=lens)
    rmt.rmt_sync(None)
    assert torch.equal(out[0, :150], out[1, :150]) and out[1, :150].abs().max() > 0
    assert not out[:, 150:].any()


# ------------------------------------------------------------------- together, and as used

@gpu
@pytest.mark.parametrize("dtype,dh,H,Hkv,window,sinks", [("bf16", 64, 8, 2, 70, 4), ("f32", 128, 4, 1, 100, 1),
                                                         ("bf16", 128, 8, 2, 0, 0)])
def test_prompt_then_tokens(cuda_ok, dtype, dh, H, Hkv, window, sinks):
    """Prompts of different lengths through the window and into the cache, then tokens one by one: each
    token's result is the windowed attention of its row over the keys and values the cache holds."""
    lens = [130, 64, 1]
    n, steps = len(lens), 6
    s = Setup(lens, Hkv, dh, max_pages=4)
    M, width = max(lens) + steps, (H + 2 * Hkv) * dh
    qkv = normal(41, (n, M, width), dtype)
    k0 = H * dh
    keys, values = qkv[..., k0:k0 + Hkv * dh], qkv[..., k0 + Hkv * dh:]
    out = torch.zeros(n, M, H * dh, dtype=TORCH[dtype], device="cuda")
    rmt.rmt_attention_window(qkv, out, n, M, H, Hkv, dh, window, sinks, lens=s.lens, dtype=dtype)
    rmt.rmt_cache_write(s.cache, keys, values, M, n_new=s.lens, dtype=dtype)
    ws = torch.empty(rmt.rmt_attention_cache_workspace(s.cache, 1, H, window, sinks), dtype=torch.uint8, device="cuda")
    rows = []
    for _ in range(steps):
        row = torch.stack([qkv[b, s.lengths[b]] for b in range(n)])[:, None]
        s.lens += 1
        s.lengths = [t + 1 for t in s.lengths]
        rmt.rmt_cache_write(s.cache, row[..., k0:k0 + Hkv * dh], row[..., k0 + Hkv * dh:], 1, dtype=dtype)
        rows.append(s.attend(row[..., :k0], 1, H, window, sinks, dtype, workspace=ws))
    # what the cache holds, laid out as rows again, through the windowed attention
    held = qkv.clone()
    kv = [torch.zeros(n, M, Hkv * dh, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    rmt.rmt_cache_read(s.cache, *kv, M, n_new=s.lens, dtype=dtype)
    for b in range(n):
        held[b, :s.lengths[b], k0:] = torch.cat([x[b, :s.lengths[b]] for x in kv], -1)
    again = torch.zeros_like(out)
    rmt.rmt_attention_window(held, again, n, M, H, Hkv, dh, window, sinks, lens=s.lens, dtype=dtype)
    rmt.rmt_sync(None)
    vals = s.values()
    for b in range(n):
        T = s.lengths[b]
        k, v = vals[b]
        pos = np.arange(T - steps, T)
        ref = attend_ref(f64(qkv)[b, T - steps:T, :k0].reshape(steps, H, dh), k, v, pos, window, sinks)
        for i in range(steps):
            check_attention(f64(rows[i])[b].reshape(H, dh), ref[i], np.abs(v).max(), dtype)
        check_attention(f64(again)[b, T - steps:T].reshape(steps, H, dh), ref, np.abs(v).max(), dtype)


@gpu
def test_captured_calls_replay_with_new_lengths_and_inputs(cuda_ok):
    """One token's step captured once: later replays read the lengths, tables and rows of their time."""
    dh, H, Hkv, lens = 64, 8, 2, [100, 700, 3]
    s = Setup(lens, Hkv, dh, max_pages=16)
    s.fill(1, "bf16")
    row = normal(2, (3, 1, (H + 2 * Hkv) * dh), "bf16")
    qkv = normal(3, (1, 200, (H + 2 * Hkv) * dh), "bf16")
    k0 = H * dh
    out = torch.zeros(3, 1, k0, dtype=torch.bfloat16, device="cuda")
    wout = torch.zeros(1, 200, k0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(rmt.rmt_attention_cache_workspace(s.cache, 1, H, 90, 4), dtype=torch.uint8, device="cuda")

    def step():
        rmt.rmt_cache_write(s.cache, row[..., k0:k0 + Hkv * dh], row[..., k0 + Hkv * dh:], 1)
        rmt.rmt_attention_cache(s.cache, row[..., :k0], out, 1, H, 90, 4, ws)
        rmt.rmt_attention_window(qkv, wout, 1, 200, H, Hkv, dh, 50, 4)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for it in range(3):
        s.lens += 1 + it
        row.copy_(normal(10 + it, tuple(row.shape), "bf16"))
        qkv.copy_(normal(20 + it, tuple(qkv.shape), "bf16"))
        before = s.pages.clone()
        graph.replay()
        torch.cuda.synchronize()
        got, wgot, pages = out.clone(), wout.clone(), s.pages.clone()
        s.pages.copy_(before)
        step()
        rmt.rmt_sync(None)
        # as bits: from the second replay on the lengths take in tokens that no call has written, whose
        # bytes may stand for NaN
        bits = [x.view(torch.int16) for x in (got, out, wgot, wout)]
        assert torch.equal(*bits[:2]) and torch.equal(*bits[2:]) and torch.equal(pages, s.pages)
        assert it > 0 or torch.isfinite(out).all()


@gpu
def test_calls_on_two_streams_at_once_and_again_give_the_same_bits(cuda_ok):
    dh, H, Hkv = 64, 16, 2
    s = Setup([3000, 10, 900], Hkv, dh)
    s.fill(1, "bf16")
    qs = [normal(i, (3, 2, H * dh), "bf16") for i in range(2)]
    want = [s.attend(q, 2, H, 0, 0, "bf16") for q in qs]
    rmt.rmt_sync(None)
    for _ in range(5):
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for st, q in zip(streams, qs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(s.attend(q, 2, H, 0, 0, "bf16"))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# -------------------------------------------------------------------------------- refusals

def _cache(**kw):
    f = dict(pages=256, page_table=256, lens=256, n_pages=4, n_seqs=2, max_pages=2, n_kv_heads=2, head_dim=64)
    f.update(kw)
    return rmt.rmt_cache_struct(*[f[n] for n, _ in rmt.rmt_cache_struct._fields_])


BAD_CACHES = [dict(pages=None), dict(page_table=None), dict(lens=None), dict(n_pages=0), dict(n_seqs=0),
              dict(max_pages=0), dict(max_pages=2 ** 25), dict(n_kv_heads=0), dict(n_kv_heads=5000), dict(head_dim=48),
              dict(pages=264), dict(lens=257), dict(page_table=258)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_refusals(bad):
    lib, c = rmt.lib(), _cache(**bad)
    ref = ctypes.byref(c)
    assert lib.rmt_cache_write(ref, 256, 256, 1024, 1, None, 1, None) == rmt.RMT_EINVAL
    assert lib.rmt_cache_read(ref, 256, 256, 1024, 1, None, 1, None) == rmt.RMT_EINVAL
    assert lib.rmt_attention_cache(ref, 256, 1024, 256, 1, c.n_kv_heads or 1, 0, 0, 256, 1 << 40, 1, None) == rmt.RMT_EINVAL
    assert lib.rmt_attention_cache_workspace(ref, 1, c.n_kv_heads or 1, 0, 0) == 0
    assert rmt.rmt_last_error()


def test_row_refusals():
    lib, c = rmt.lib(), _cache()
    ref = ctypes.byref(c)
    for fn in (lib.rmt_cache_write, lib.rmt_cache_read):
        ok = [ref, 256, 256, 128, 1, None, 1, None]
        for i, v in ((0, None), (1, None), (2, None), (1, 264), (2, 250), (3, 127), (3, 132), (4, 0), (4, -1), (5, 3),
                     (6, 2), (6, 9)):
            a = list(ok)
            a[i] = v
            assert fn(*a) == rmt.RMT_EINVAL, (i, v)


def test_attention_refusals():
    lib, c = rmt.lib(), _cache()
    ref = ctypes.byref(c)
    need = lib.rmt_attention_cache_workspace(ref, 1, 4, 0, 0)
    assert need > 0
    ok = [ref, 256, 256, 256, 1, 4, 0, 0, 256, need, 1, None]
    for i, v in ((0, None), (1, None), (1, 258), (2, 255), (2, 260), (3, None), (3, 264), (4, 0), (4, 65), (5, 0), (5, 3),
                 (6, -1), (7, -1), (8, None), (8, 260), (9, need - 1), (10, 2)):
        a = list(ok)
        a[i] = v
        assert lib.rmt_attention_cache(*a) == rmt.RMT_EINVAL, (i, v)
    ok = [256, 256, 1, 8, 4, 2, 64, 5, 1, None, 1, None]
    for i, v in ((0, None), (1, None), (0, 258), (1, 264), (2, 0), (2, 70000), (3, 0), (3, 2 ** 30 + 1), (4, 3), (4, 0),
                 (5, 0), (6, 48), (7, -1), (8, -2), (9, 3), (10, 2)):
        a = list(ok)
        a[i] = v
        assert lib.rmt_attention_window(*a) == rmt.RMT_EINVAL, (i, v)


def test_page_bytes_and_binding_checks():
    assert rmt.rmt_cache_page_bytes(8, 64) == 8 * 2 * 64 * (32 + 4)
    assert rmt.rmt_cache_page_bytes(1, 128) == 9216
    with pytest.raises(ValueError):
        rmt.rmt_cache_page_bytes(1, 48)
    t, z = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(4 * 4608, dtype=torch.uint8)
    c = rmt.rmt_cache(pages, t, z, 1, 64)
    assert (c.struct.n_pages, c.struct.n_seqs, c.struct.max_pages) == (4, 2, 3)
    with pytest.raises(ValueError):
        rmt.rmt_cache(pages[:-1], t, z, 1, 64)
    with pytest.raises(TypeError):
        rmt.rmt_cache(pages, t.long(), z, 1, 64)
    with pytest.raises(ValueError):
        rmt.rmt_cache(pages, t, z[:1], 1, 64)
    x = torch.zeros(2, 5, 100, dtype=torch.bfloat16)
    assert rmt._rows(x[..., 8:72], 2, 5, 64, "bf16") == (x.data_ptr() + 16, 100)
    assert rmt._rows(x[:, :1, :64], 2, 1, 64, "bf16")[1] == 500
    assert rmt._rows(torch.zeros(1, 1, 2, 32), 1, 1, 64, "f32")[1] == 64
    for bad, width, dtype in ((x[:, ::2, :64], 64, "bf16"), (x[..., :128:2], 50, "bf16"), (x[..., :64], 64, "f32"),
                              (x[:, :4, :64], 64, "bf16"), (x[..., :64].transpose(0, 1), 64, "bf16"),
                              (x[..., 0], 1, "bf16"), (x[0, 0], 100, "bf16"), (x, 64, "bf16")):
        with pytest.raises((ValueError, TypeError)):
            rmt._rows(bad, 2, 5, width, dtype)
    w, o = torch.zeros(2, 5, 96, dtype=torch.bfloat16), torch.zeros(2, 5, 32, dtype=torch.bfloat16)
    for args, kw in (((w, o[:, :4].clone()), {}), ((w.float(), o), {}), ((w, o.float()), {}), ((w, w[..., :32]), {}),
                     ((w[..., :64].clone(), o), {}), ((w, o), dict(lens=z[:1])), ((w, o), dict(lens=z.long()))):
        with pytest.raises((ValueError, TypeError)):  # out or qkv too short, of the wrong type or not contiguous; lens
            rmt.rmt_attention_window(*args, 2, 5, 1, 1, 32, 0, **kw)
    k = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rmt.rmt_cache_write(c, k, k, 5, n_new=z[:1])
    for out in (k[:, :4].clone(), k.float(), k[..., :32]):
        with pytest.raises((ValueError, TypeError)):
            rmt.rmt_attention_cache(c, k, out, 5, 1, 0, 0, torch.zeros(1 << 20, dtype=torch.uint8))
