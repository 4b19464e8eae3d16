"""The paged K/V cache on the GPU against plain float64 forms: quantised writes, reads back,
attention of the newest tokens, and the calls together as a serving loop makes them.

Codes, scales and values read back must be exact. The attention's tolerance is derived: a
logit is an f32 sum of D exact products, off by at most D f32 units (2^-23, a truncating
sum) of sum|q k|, and its exponential by two units more; that error e enters numerator
and denominator; the sums over n cells add at most n units, the rest of the chain (scale,
split f16 weights, merge) a few tens of units. A weight is held as two f16 terms of
2^7 p, where the running maximum that p is relative to lags the largest logit by up to 2^8:
what is below half an f16 subnormal step of them, 2^-25 2^-7, is lost, so each of the n
weights is off by 2^-32 of the largest at most (this term counts where an output's own
weights are all tiny).
"""
import numpy as np
import pytest
import torch

import sparse_attention_decode_02_b200 as Q
from oracle import paged_oracle as P
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

FORMATS = {"f16": Q.QSA_PAGE_F16, "fp8": Q.QSA_PAGE_FP8, "int4": Q.QSA_PAGE_INT4}
BAD_INDEX, CAPACITY = 6, 2
UNIT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_library()


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


class Pool:
    """A paged cache of sequences with the given capacities, its pages in random order, and
    the f16 rows written to it (one array a sequence)."""

    def __init__(self, caps, fmt, heads, dim, page, seed=0, spare=3, gap=0, poison=True):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.heads, self.dim, self.page = fmt, heads, dim, page
        need = [-(-c // page) for c in caps]
        self.width, n = max(max(need), 1), sum(need) + spare
        row, kind = {"f16": (dim, torch.float16), "fp8": (dim, torch.uint8), "int4": (dim // 2, torch.uint8)}[fmt]
        mk = lambda *s, dtype: torch.zeros(n, 1 + gap, *s, dtype=dtype, device="cuda")  # noqa: E731
        self.big = [mk(heads, page, row, dtype=kind) for _ in range(2)]
        if fmt != "f16":
            s = (heads, page) if fmt == "fp8" else (heads, page, dim // 32)
            self.big += [mk(*s, dtype=torch.float32 if fmt == "fp8" else torch.float16) for _ in range(2)]
        if poison:     # what no sequence holds is NaN
            for t in self.big:
                t.fill_(float("nan") if t.dtype != torch.uint8 else 0x7F)
        parts = [t[:, gap] for t in self.big]     # with a gap: one layer of a pool of several
        self.cache = Q.PagedKV(parts[0], parts[1], FORMATS[fmt], *parts[2:])
        self.parts = parts + [None] * (4 - len(parts))
        ids = self.rng.permutation(n)
        self.table = np.full((len(caps), self.width), -1, np.int64)   # unused entries are no page
        at = 0
        for i, k in enumerate(need):
            self.table[i, :k] = ids[at:at + k]
            at += k
        self.table_dev = _i32(self.table)
        self.lens = [0] * len(caps)
        self.rows = [[np.zeros((0, heads, dim), np.float16) for _ in caps] for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def random_rows(self, counts, scale=1.0):
        n = sum(counts)
        return [(self.rng.standard_normal((n, self.heads, self.dim)) * scale).astype(np.float16) for _ in range(2)]

    def append(self, counts, kv=None, stream=None):
        k, v = kv if kv is not None else self.random_rows(counts)
        start = np.concatenate([[0], np.cumsum(counts)])
        self.cache.write(H.to_dev(k), H.to_dev(v), self.table_dev, _i32(self.lens), _i32(start), status=self.status,
                         stream=stream)
        for i, c in enumerate(counts):
            for x, rows in ((k, self.rows[0]), (v, self.rows[1])):
                rows[i] = np.concatenate([rows[i][:self.lens[i]], x[start[i]:start[i + 1]]])
            self.lens[i] += c
        return k, v

    def values(self, i):
        """The float64 K and V of sequence i that its stored rows stand for."""
        return [P.values(*P.quantise(rows[i], self.fmt), self.fmt) for rows in self.rows]

    def attend(self, q, lse=True, sm_scale=0.0, lens=None, **kw):
        S, T, Hq, D = q.shape
        out = torch.full((S, T, Hq, D), float("nan"), device="cuda")
        l = torch.full((S, T, Hq), float("nan"), device="cuda") if lse else None
        ws = torch.full((self.cache.workspace_bytes(Hq, T),), 0xFF, dtype=torch.uint8, device="cuda")
        self.cache.attend(q if torch.is_tensor(q) else H.to_dev(q), self.table_dev,
                          _i32(self.lens if lens is None else lens), out, ws, lse=l, sm_scale=sm_scale,
                          status=self.status, **kw)
        return out, l

    def check(self, q, out, lse, sm_scale=None, code=0):
        out = out.cpu().numpy().astype(np.float64)
        lse = lse.cpu().numpy().astype(np.float64)
        for i, n in enumerate(self.lens):
            k, v = self.values(i)
            assert_attention(out[i], lse[i], q[i], k, v, sm_scale, f"sequence {i} of {n} tokens")
        assert int(self.status) == code


def assert_attention(out, lse, q, k, v, sm_scale=None, what=""):
    want, want_lse, bound, depth = P.attention(q, k, v, sm_scale)
    n, D = len(k), q.shape[-1]
    e = (D * depth + 8 * (np.abs(np.where(np.isfinite(want_lse), want_lse, 0)) + depth + 1)) * UNIT
    tol = (2 * e[..., None] + (n + 64) * UNIT) * bound + n * 2.0 ** -32 * np.abs(v).max(initial=0.0)
    assert np.isfinite(out).all(), f"{what}: out is not finite"
    assert (np.abs(out - want) <= tol).all(), f"{what}: {np.max(np.abs(out - want) / np.maximum(tol, 1e-30)):.3g} of tolerance"
    empty = np.isinf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty), what
    tol = e + (n + 64) * UNIT
    assert (np.abs(lse - np.where(empty, 0, want_lse))[~empty] <= tol[~empty]).all(), f"{what}: lse"


def _query(rng, S, T, Hq, D, scale=1.0):
    return (rng.standard_normal((S, T, Hq, D)) * scale).astype(np.float16)


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,dim,page,gap", [(1, 64, 16, 0), (4, 128, 32, 0), (3, 64, 128, 2), (8, 128, 256, 1)])
def test_written_rows_are_exact_and_nothing_else_changes(fmt, heads, dim, page, gap):
    counts = [5, 0, 1, 40, 0, 300, 17]
    p = Pool([60, 4, 30, 100, 0, 310, 40], fmt, heads, dim, page, seed=dim + page, gap=gap)
    p.lens = [11, 0, 29, 3, 0, 10, 16]     # what they hold already is not looked at here
    for i, n in enumerate(p.lens):
        for rows in p.rows:
            rows[i] = np.zeros((n, heads, dim), np.float16)
    old, before = [t.clone() for t in p.big], list(p.lens)
    k, v = p.append(counts)
    torch.cuda.synchronize()
    assert int(p.status) == 0
    want = [t.cpu().numpy().copy() for t in old]
    at = 0
    for i, c in enumerate(counts):
        for j in range(c):
            pos = before[i] + j
            for t, x in ((0, k), (1, v)):
                codes, scales = P.quantise(x[at], fmt)
                want[t][p.table[i, pos // page], gap, :, pos % page] = codes
                if scales is not None:
                    want[t + 2][p.table[i, pos // page], gap, :, pos % page] = scales
            at += 1
    for t, w in zip(p.big, want):
        got = t.cpu().numpy()
        assert np.array_equal(got.view(np.uint8), w.view(np.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (4, 128, 64), (5, 128, 16)])
def test_rows_read_back_are_the_stored_values(fmt, heads, dim, page):
    p = Pool([200, 3, 0, 77], fmt, heads, dim, page, seed=1)
    p.append([190, 1, 0, 77])
    first, counts = [13, 0, 0, 70], [150, 1, 0, 7]
    start = np.concatenate([[0], np.cumsum(counts)])
    n = start[-1]
    full = lambda: torch.full((n + 5, heads, dim), 9.0, dtype=torch.float16, device="cuda")  # noqa: E731
    k, v, only = full(), full(), full()
    p.cache.read(k, v, p.table_dev, _i32(first), _i32(start), status=p.status)
    p.cache.read(None, only, p.table_dev, _i32(first), _i32(start), status=p.status)
    assert int(p.status) == 0
    for t, got in ((0, k), (1, v), (1, only)):
        want = np.full((n + 5, heads, dim), 9.0, np.float16)    # rows behind the last sequence stay
        for i, c in enumerate(counts):
            codes, scales = P.quantise(p.rows[t][i][first[i]:first[i] + c], fmt)
            if fmt == "fp8":    # the f32 product, rounded to f16
                x = P.values(codes, np.ones_like(scales), fmt).astype(np.float32) * scales[..., None]
            else:
                x = P.values(codes, scales, fmt)
            want[start[i]:start[i + 1]] = x.astype(np.float16)
        assert np.array_equal(got.cpu().numpy(), want)


def test_rows_of_a_fused_projection_and_special_values():
    """Rows that lie apart, and zeros, tiny, huge, infinite and NaN values."""
    for fmt in FORMATS:
        p = Pool([64], fmt, 2, 128, 16)
        fused = torch.randn(40, 1024, device="cuda").half()
        k, v = fused[:, 512:768].unflatten(1, (2, 128)), fused[:, 768:].unflatten(1, (2, 128))
        fused[3, 512:640] = 0
        fused[4, 512:520] = 6e-8
        fused[5, 512:640] = (fused[5, 512:640].float() * 2e4).clamp(-65504, 65504).half()     # huge, not infinite
        fused[6, 520] = float("inf")
        fused[7, 600] = float("nan")
        fused[8, 512:640] = 6e-8
        rows = fused.cpu().numpy()
        start, first = _i32([0, 40]), _i32([0])
        p.cache.write(k, v, p.table_dev, first, start, status=p.status)
        back = torch.empty(40, 1024, dtype=torch.float16, device="cuda")
        p.cache.read(back[:, :256].unflatten(1, (2, 128)), back[:, 256:512].unflatten(1, (2, 128)), p.table_dev, first,
                     start, status=p.status)
        got = back[:, :512].reshape(40, 4, 128).cpu().numpy()
        src = rows[:, 512:].reshape(40, 4, 128)
        fine = [r for r in range(40) if r not in (6, 7)]
        codes, scales = P.quantise(src[fine], fmt)
        want = P.values(codes, np.ones_like(scales), fmt).astype(np.float32) * scales[..., None] if fmt == "fp8" \
            else P.values(codes, scales, fmt)
        assert np.array_equal(got[fine], want.astype(np.float16)), fmt
        if fmt == "f16":
            assert np.array_equal(got.view(np.uint16), src.view(np.uint16))
        else:       # not finite where the input is not, the other heads' rows untouched by it
            assert not np.isfinite(got[6, 0, 8]) and np.isnan(got[7, 0, 88])
            assert np.isfinite(got[6:8, 1:]).all()
            if fmt == "int4":
                assert np.isnan(got[6, 0, :32]).all() and np.isfinite(got[6, 0, 32:]).all()
                assert np.isnan(got[7, 0, 64:96]).all() and np.isfinite(got[7, 0, :64]).all()
        assert int(p.status) == 0


def test_4bit_rows_of_the_largest_values_are_finite():
    """Groups whose largest value is each of f16's, 65504 among them, and attention over those."""
    n = 0x7c00
    p = Pool([n], "int4", 1, 64, 256)
    k, v = np.zeros((n, 1, 64), np.float16), np.zeros((n, 1, 64), np.float16)
    k[:, 0, 40] = v[:, 0, 3] = np.arange(n, dtype=np.uint16).view(np.float16)
    v[:, 0, 4] = -v[:, 0, 3]
    p.append([n], (k, v))
    back = [torch.empty(n, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    p.cache.read(*back, p.table_dev, _i32([0]), _i32([0, n]), status=p.status)
    for x, want in zip(back, p.values(0)):
        assert torch.isfinite(x).all() and np.array_equal(x.cpu().numpy().astype(np.float64), want)
    # every weight is 1 / n
    q = np.zeros((1, 1, 4, 64), np.float16)
    out, lse = p.attend(q)
    p.check(q, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_without_a_place_are_skipped_and_reported(fmt):
    p = Pool([32, 32, 32], fmt, 2, 64, 16)
    p.append([32, 32, 32])
    old = [t.clone() for t in p.big]
    k = torch.randn(4, 2, 64, device="cuda").half()
    cases = [([33, 0, 0], [0, 4, 4, 4], None, CAPACITY), ([-4, 0, 0], [0, 4, 4, 4], None, BAD_INDEX),
             ([0, 0, 0], [0, 4, 4, 4], 7, BAD_INDEX), ([0, 0, 0], [0, 4, 4, 4], -1, BAD_INDEX),
             ([0, 2 ** 31 - 2, 0], [0, 0, 4, 4], None, CAPACITY)]
    for first, start, page, code in cases:
        table = p.table_dev.clone()
        if page is not None:
            table[0, 0] = 10 ** 6 if page > 0 else page
        p.status.zero_()
        p.cache.write(k, k, table, _i32(first), _i32(start), status=p.status)
        assert int(p.status) == code, (first, page)
        p.cache.write(k, k, table, _i32(first), _i32(start))           # without a status word
        for a, b in zip(p.big, old):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        p.status.zero_()
        x, y = torch.ones_like(k), torch.ones_like(k)
        p.cache.read(x, y, table, _i32(first), _i32(start), status=p.status)
        assert int(p.status) == code and not x.any() and not y.any()


# ------------------------------------------------------------------ attention

LENS = [0, 1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300]
SHAPES = [(1, 1, 64, 16), (8, 1, 64, 32), (2, 2, 128, 16), (32, 4, 128, 64), (4, 4, 128, 128), (6, 2, 64, 256),
          (15, 3, 128, 32), (7, 1, 128, 16)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("hq,hkv,dim,page", SHAPES)
def test_attention_of_many_lengths(fmt, T, hq, hkv, dim, page):
    p = Pool(LENS, fmt, hkv, dim, page, seed=T)
    p.append(LENS)
    q = _query(p.rng, len(LENS), T, hq, dim)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,hq,hkv,dim,n", [(1, 32, 4, 128, 5003), (4, 8, 1, 64, 4097), (3, 16, 2, 128, 9001), (1, 1, 1, 64, 20000)])
def test_attention_of_one_long_sequence(fmt, T, hq, hkv, dim, n):
    p = Pool([n], fmt, hkv, dim, 64, seed=n)
    p.append([n])
    q = _query(p.rng, 1, T, hq, dim)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_with_large_logits_and_small_or_large_values(fmt):
    """Weights from 1 down past f32's range; rows whose sizes differ by orders of magnitude."""
    counts = [70, 200]
    p = Pool(counts, fmt, 2, 128, 16, seed=5)
    k, v = p.random_rows(counts)
    v = (v * np.exp2(p.rng.integers(-12, 12, (270, 2, 1)))).astype(np.float16)
    k[10:14] *= 20
    p.append(counts, (k, v))
    q = _query(p.rng, 2, 2, 16, 128, scale=8.0)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("size", [1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("other", ["zero", "large", "both", "ladder"])
@pytest.mark.parametrize("fmt,T,hq,dim", [("fp8", 1, 8, 128), ("fp8", 4, 8, 128), ("fp8", 3, 4, 64), ("int4", 1, 8, 128)])
def test_small_values_beside_rows_of_other_sizes(size, other, fmt, T, hq, dim):
    """V rows of zeros (whose e4m3 scale is 1), large ones whose keys give them next to no
    weight, and sizes that fall from row to row do not cost the other rows their precision.

    The logits z are exact (one non-zero dim), so the exponent (z - reference) log2(e) has four
    roundings and the exponential two units, with a reference within 8 ln(2) of the largest.
    Two f16 terms of 2^7 p leave 2^-25 of p behind at most, or p itself; for e4m3 relative to a
    power of two at most 2^8 above the row's scale: 2^-24 of the largest weight."""
    lens = [120, 9, 40, 2500]
    p = Pool(lens, fmt, 1, dim, 16, seed=3)
    n = sum(lens)
    k, v = np.zeros((n, 1, dim), np.float16), p.rng.standard_normal((n, 1, dim)) * size
    k[..., 0] = p.rng.integers(-2, 3, (n, 1)) / 4
    if other == "ladder":
        v *= np.exp2(-0.75 * (np.arange(n) % 16))[:, None, None]
    if other in ("zero", "both"):
        v[p.rng.random(n) < 0.1] = 0
        v[[3, 123, 132]] = 0
    if other in ("large", "both"):
        far = p.rng.random(n) < 0.1
        far[[5, 125, 135]], far[[0, 120, 129, 169]] = True, False
        v[far] *= 3000
        k[far, :, 0] = -60
    p.append(lens, (k, v.astype(np.float16)))
    q = np.zeros((len(lens), T, hq, dim), np.float16)
    q[..., 0] = 8.0
    out, lse = (x.cpu().numpy().astype(np.float64) for x in p.attend(q, sm_scale=0.25))
    for i, m in enumerate(lens):
        kk, vv = p.values(i)
        want, want_lse, bound, _ = P.attention(q[i], kk, vv, 0.25)
        for u in range(T):
            seen = m - T + u + 1
            z, size_of = kk[:seen, 0, 0] * 8.0 * 0.25, np.abs(vv[:seen, 0])
            w = np.exp(z - want_lse[u, 0])
            e = (np.abs(z - z.max()) + 8 * np.log(2) + 1) * 2 * UNIT
            left = np.minimum(w, w.max() * (2.0 ** -24 if fmt == "fp8" else 2.0 ** -32))
            tol = (w * e) @ size_of + (w @ e + (seen + 64) * UNIT) * bound[u] + left @ size_of
            assert (np.abs(out[i, u] - want[u]) <= tol).all(), f"{i} {u}: {np.max(np.abs(out[i, u] - want[u]) / tol):.3g}"
            assert (np.abs(lse[i, u] - want_lse[u]) <= w @ e + (seen + 64) * UNIT + UNIT * np.abs(want_lse[u])).all()


def test_attention_of_constant_rows():
    """Equal keys: every cell has the same weight; equal values come back as they are."""
    p = Pool([1000], "f16", 1, 64, 16)
    k, v = np.ones((1000, 1, 64), np.float16), np.full((1000, 1, 64), 3.0, np.float16)
    p.append([1000], (k, v))
    q = np.full((1, 1, 8, 64), -30000.0, np.float16)    # every logit is the same huge negative number
    out, lse = p.attend(q)
    assert torch.allclose(out, torch.full_like(out, 3.0), rtol=1e-6)
    z = -30000.0 * 64 / 8
    assert abs(float(lse[0, 0, 0]) - (z + np.log(1000))) <= 2 * abs(z) * UNIT


def assert_exact_logits(out, lse, q, k, v, sm_scale=None, what=""):
    """For queries and keys whose products and sums are exact in f32, whatever their size. The
    exponent (s - max) sm_scale log2(e) is then off by four roundings of half a unit, and what
    has an exponent below -150 has no weight in f32: 150 ln(2) 4 2^-24 and two units of the
    exponential make the error of a weight."""
    want, want_lse, bound, _ = P.attention(q, k, v, sm_scale)
    n = len(k)
    e = 150 * np.log(2) * 2 * UNIT + 2 * UNIT
    tol = (2 * e + (n + 64) * UNIT) * bound + n * 2.0 ** -32 * np.abs(v).max()
    assert np.isfinite(out).all() and np.isfinite(lse).all(), f"{what}: not finite"
    assert (np.abs(out - want) <= tol).all(), f"{what}: {np.max(np.abs(out - want) / tol):.3g} of tolerance"
    assert (np.abs(lse - want_lse) <= 2 * UNIT * np.abs(want_lse) + e + (n + 64) * UNIT).all(), f"{what}: lse"


HUGE = [([5000], 1), ([37, 700, 1], 1), ([20, 5], 4), ([900], 3), ([33] * 460, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,T", HUGE)
@pytest.mark.parametrize("sm_scale", [0.0, 1.0, 1e4, 1e20])
def test_logits_of_any_size(fmt, lens, T, sm_scale):
    """Logits as large as f16 rows and an accepted scale make them, equal and not, in whole
    segments and in segments cut into parts: the largest ones share the weight."""
    p = Pool(lens, fmt, 1, 128, 16, seed=len(lens))
    n = sum(lens)
    k, v = np.zeros((n, 1, 128), np.float16), p.random_rows(lens)[1]
    k[..., 1] = 57344                           # makes every scale a power of two: stored exactly
    k[..., 0] = p.rng.choice([57344, 49152], (n, 1))
    p.append(lens, (k, v))
    assert all((p.values(i)[0] == p.rows[0][i]).all() for i in range(len(lens)))
    q = np.zeros((len(lens), T, 4, 128), np.float16)
    q[..., 0] = p.rng.choice([60000, -60000, 30000, 2.0 ** -14], (len(lens), T, 4))
    out, lse = (x.cpu().numpy().astype(np.float64) for x in p.attend(q, sm_scale=sm_scale))
    assert int(p.status) == 0
    for i in range(len(lens)):
        kk, vv = p.values(i)
        assert_exact_logits(out[i], lse[i], q[i], kk, vv, sm_scale, f"sequence {i}")


@pytest.mark.parametrize("value", [100, 2000, 8000, 30000, 65504])
@pytest.mark.parametrize("n,T", [(10, 1), (5000, 1), (700, 4)])
def test_equal_logits_of_any_size(value, n, T):
    """Rows and queries of one value: every cell has the same weight, however large the logit."""
    p = Pool([n], "f16", 1, 128, 64, seed=n)
    k, v = np.full((n, 1, 128), value, np.float16), p.random_rows([n])[1]
    p.append([n], (k, v))
    q = np.full((1, T, 8, 128), value, np.float16)
    out, lse = (x.cpu().numpy().astype(np.float64)[0] for x in p.attend(q))
    for u in range(T):
        seen = n - T + u + 1
        want, bound = v[:seen, 0].astype(np.float64).mean(0), np.abs(v[:seen, 0].astype(np.float64)).mean(0)
        assert (np.abs(out[u] - want) <= (seen + 64) * UNIT * bound + 2.0 ** -32 * np.abs(v).max()).all()
        # (the sum of 128 products is off by up to 128 units)
        z = float(np.float16(value)) ** 2 * 128 / np.sqrt(128)
        assert (np.abs(lse[u] - (z + np.log(seen))) <= 130 * UNIT * z + (seen + 64) * UNIT).all()


@pytest.mark.parametrize("step", [2.0 ** 25, 2.0 ** 27, 2.0 ** 29])
def test_large_logits_that_differ_by_their_last_bits(step):
    """q.K = step + the smallest f32 differences from it: the weights are those of the differences."""
    n = 300
    p = Pool([n], "f16", 1, 128, 16, seed=7)
    k, v = np.zeros((n, 1, 128), np.float16), p.random_rows([n])[1]
    k[..., 0], k[..., 1] = 2.0 ** 14, p.rng.integers(0, 6, (n, 1)) * step * 2.0 ** -23
    p.append([n], (k, v))
    q = np.zeros((1, 1, 8, 128), np.float16)
    q[..., 0], q[..., 1] = step / 2.0 ** 14, 1.0
    for sm_scale in (1.0, 0.125, 0.01):
        out, lse = (x.cpu().numpy().astype(np.float64) for x in p.attend(q, sm_scale=sm_scale))
        assert_exact_logits(out[0], lse[0], q[0], *p.values(0), sm_scale, f"scale {sm_scale}")


def test_a_logit_that_overflows_to_minus_infinity_has_no_weight():
    """q k beyond f32 is not reachable from f16 rows, but infinite keys are: -inf logits drop
    out, and a sequence with nothing else is empty."""
    p = Pool([20, 20], "f16", 1, 64, 16)
    k, v = p.random_rows([20, 20])
    k[5:9] = 0
    k[5:9, :, 0] = -np.inf
    k[20:] = 0
    k[20:, :, 0] = -np.inf
    p.append([20, 20], (k, v))
    q = np.abs(_query(p.rng, 2, 1, 4, 64)) + np.float16(0.1)
    out, lse = p.attend(q)
    keep = [c for c in range(20) if not 5 <= c < 9]
    kk, vv = p.values(0)
    assert_attention(out[0].cpu().numpy().astype(np.float64), lse[0].cpu().numpy().astype(np.float64), q[0], kk[keep], vv[keep])
    assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [2, 4])
def test_what_a_query_does_not_see_does_not_matter(fmt, T):
    """NaN and infinite rows among the newest tokens: queries before them are exact."""
    counts = [90, 16, 17, T, 33]
    for bad in range(1, T):         # the first of the newest T that holds no numbers
        p = Pool(counts, fmt, 2, 128, 16, seed=T)
        k, v = p.random_rows(counts)
        at = 0
        for c in counts:
            for x in (k, v):
                x[at + c - T + bad] = np.nan
                if bad + 1 < T:
                    x[at + c - T + bad + 1] = np.inf
            at += c
        p.append(counts, (k, v))
        q = _query(p.rng, len(counts), T, 8, 128)
        out, lse = p.attend(q)
        for i, c in enumerate(counts):
            kk, vv = p.values(i)
            n = c - T + bad
            if n == 0:
                continue
            assert_attention(out[i, :bad].cpu().numpy().astype(np.float64), lse[i, :bad].cpu().numpy().astype(np.float64),
                             q[i, :bad], kk[:n], vv[:n], what=f"bad {bad} of {c}")
            assert torch.isnan(out[i, bad:]).any(-1).all()      # those that see them say so


@pytest.mark.parametrize("T,n", [(1, 40), (1, 3000), (2, 77), (4, 16), (4, 900)])
@pytest.mark.parametrize("dim", [64, 128])
def test_infinite_values_that_a_query_sees(T, n, dim):
    """An infinite V value makes that dim of the output infinite, a NaN or two infinities that
    differ make it NaN, whether all of the newest queries see the cell or some; no other dim
    changes."""
    p = Pool([n], "f16", 2, dim, 16, seed=n)
    k, v = p.random_rows([n])
    v[3, 0, 5], v[n // 2, 0, 6], v[7, 0, 7] = np.inf, -np.inf, np.nan
    v[1, 0, 8], v[9, 0, 8] = np.inf, -np.inf
    v[2, 0, 9] = v[11, 0, 9] = np.inf
    v[n - 1, 0, 10], v[n - 1, 1, 11] = np.inf, -np.inf      # cells that only the last query sees
    v[n - T, 1, 12] = np.inf                                # and one that all do
    p.append([n], (k, v))
    q = _query(p.rng, 1, T, 8, dim)
    out, lse = (x.cpu().numpy().astype(np.float64)[0] for x in p.attend(q))
    with np.errstate(invalid="ignore"):
        for u in range(T):
            seen = n - T + u + 1
            kk, vv = p.values(0)
            for h in range(8):
                z = kk[:seen, h // 4] @ q[0, u, h].astype(np.float64) / np.sqrt(dim)
                w = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
                want = (w[:, None] * vv[:seen, h // 4]).sum(0)
                fine, got = np.isfinite(want), out[u, h]
                assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (u, h, got[~fine], want[~fine])
                depth = (np.abs(kk[:seen, h // 4]) @ np.abs(q[0, u, h].astype(np.float64))).max() / np.sqrt(dim)
                e = (dim * depth + 8 * (2 * depth + np.log(seen) + 1)) * UNIT
                bound = (w[:, None] * np.abs(vv[:seen, h // 4])).sum(0)
                size = np.abs(vv[np.isfinite(vv)]).max()
                tol = (2 * e + (seen + 64) * UNIT) * bound[fine] + seen * 2.0 ** -32 * size
                assert (np.abs(got[fine] - want[fine]) <= tol).all()


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
@pytest.mark.parametrize("T,n", [(1, 50), (3, 700), (4, 5000)])
def test_visible_values_that_are_no_numbers_in_8_and_4_bits(fmt, T, n):
    """What a stored row reads back as decides: a NaN stays in its dim (e4m3) or its group of 32 (4
    bits), an infinity takes the row or the group; a K row without numbers takes its head's
    results. Everything else is as if they were not there."""
    p = Pool([n, 40], fmt, 3, 64, 16, seed=n)
    k, v = p.random_rows([n, 40])
    v[3, 0, 5] = np.nan
    v[n // 2, 1, 40] = np.inf
    v[n // 2 + 1] *= 2.0 ** -12
    k[7, 2, 9] = np.nan
    p.append([n, 40], (k, v))
    q = _query(p.rng, 2, T, 6, 64)
    out, lse = (x.cpu().numpy().astype(np.float64) for x in p.attend(q))
    lost = [range(5, 6), range(64), range(64)] if fmt == "fp8" else [range(32), range(32, 64), range(64)]
    for x, (a, b) in ((k, (7, 2)), (v, (3, 0)), (v, (n // 2, 1))):      # the same rows without them
        x[a, b] = np.where(np.isfinite(x[a, b]), x[a, b], 0)
    clean = Pool([n, 40], fmt, 3, 64, 16, seed=n)
    clean.append([n, 40], (k, v))
    assert np.isnan(lse[0, :, 4:]).all()
    for i in range(2):
        kk, vv = p.values(i)
        for g in range(3):
            hs = slice(2 * g, 2 * g + 2)
            gone = list(lost[g]) if i == 0 else []
            keep = [d for d in range(64) if d not in gone]
            assert np.isnan(out[i, :, hs][..., gone]).all()
            if not keep:
                continue
            want, want_lse, bound, depth = P.attention(q[i], *clean.values(i))
            e = (64 * depth + 8 * (np.abs(want_lse) + depth + 1)) * UNIT
            tol = ((2 * e[..., None] + (n + 64) * UNIT) * bound + n * 2.0 ** -31 * np.abs(clean.values(i)[1]).max())[:, hs]
            assert (np.abs(out[i, :, hs] - want[:, hs]) <= tol)[..., keep].all(), (i, g)


@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("T,n", [(1, 50), (2, 40), (4, 900)])
def test_zero_codes_of_a_scale_that_is_no_number(scale, T, n):
    """e4m3 codes of zero stand for 0 times the row's scale, which is NaN for these scales, in
    attention as in what is read back, beside rows of any size."""
    p = Pool([n, n], "fp8", 2, 64, 16, seed=n)
    k, v = p.random_rows([n, n])
    v[5::7] *= 2.0 ** -12
    p.append([n, n], (k, v))
    page, place = int(p.table[0, 0]), 3
    p.parts[1][page, 1, place] = 0
    p.parts[3][page, 1, place] = float(scale)
    back = torch.empty(n, 2, 64, dtype=torch.float16, device="cuda")
    p.cache.read(None, back, p.table_dev, _i32([0, 0]), _i32([0, n, n]))
    assert torch.isnan(back[place, 1]).all() and int(torch.isnan(back).sum()) == 64
    q = _query(p.rng, 2, T, 4, 64)
    out, lse = (x.cpu().numpy().astype(np.float64) for x in p.attend(q))
    assert np.isnan(out[0, :, 2:]).all()
    for i, hs in ((0, slice(0, 2)), (1, slice(0, 4))):
        kk, vv = (x[:, : hs.stop // 2] for x in p.values(i))
        assert_attention(out[i, :, hs], lse[i, :, hs], q[i][:, hs], kk, vv)
    assert np.isfinite(lse).all()


def test_scale_strides_and_no_lse():
    p = Pool([100, 40, 7], "fp8", 2, 64, 32, gap=2)
    p.append([100, 40, 7])
    q = _query(p.rng, 3, 2, 8, 64)
    p.check(q, *p.attend(q, sm_scale=0.3), sm_scale=0.3)
    wide = torch.zeros(3, 2, 12, 64, dtype=torch.float16, device="cuda")     # q of a fused projection
    wide[:, :, :8] = H.to_dev(q)
    a, la = p.attend(wide[:, :, :8])
    b, lb = p.attend(q)
    c, _ = p.attend(q, lse=False)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(c, b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,gap", [(16, 0), (48, 16), (112, 80), (0, 16)])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (3, 128, 32)])
def test_pages_at_multiples_of_16_bytes(fmt, offset, gap, heads, dim, page):
    """Pages and scales that start at any multiple of 16 bytes, and lie such multiples apart: equal
    to the bit to the same pages one after another."""
    p = Pool([70, 33, 0, 260], fmt, heads, dim, page, seed=dim)
    lens = [70, 33, 0, 260]
    parts = []
    for t in p.parts:
        if t is None:
            parts.append(None)
            continue
        n, size, each = len(t), t[0].numel(), t.element_size()
        flat = torch.full((offset // each + n * (size + gap // each) + 64,), 77, dtype=t.dtype, device="cuda")
        at = flat[offset // each:]
        assert flat.data_ptr() % 256 == 0 and at.data_ptr() % 256 == offset
        strides = (size + gap // each,) + t[0].stride()
        parts.append(at.as_strided(t.shape, strides))
    other = Q.PagedKV(parts[0], parts[1], FORMATS[fmt], *parts[2:])
    k, v = p.append(lens)
    first, start = _i32([0] * 4), _i32(np.concatenate([[0], np.cumsum(lens)]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    other.write(H.to_dev(k), H.to_dev(v), p.table_dev, first, start, status=status)
    back = [torch.zeros(sum(lens), heads, dim, dtype=torch.float16, device="cuda") for _ in range(4)]
    p.cache.read(back[0], back[1], p.table_dev, first, start)
    other.read(back[2], back[3], p.table_dev, first, start, status=status)
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3])
    for T in (1, 3):
        q = H.to_dev(_query(p.rng, 4, T, 2 * heads, dim))
        out, lse = p.attend(q)
        got, got_lse = torch.empty_like(out), torch.empty_like(lse)
        ws = torch.empty(other.workspace_bytes(2 * heads, T), dtype=torch.uint8, device="cuda")
        other.attend(q, p.table_dev, _i32(lens), got, ws, lse=got_lse, status=status)
        assert torch.equal(out, got) and torch.equal(lse, got_lse)
    assert int(status) == 0 and int(p.status) == 0


def test_bad_lengths_and_pages_are_reported():
    p = Pool([64, 64, 64], "f16", 1, 64, 16)
    p.append([64, 64, 64])
    q = _query(p.rng, 3, 1, 4, 64)
    for lens, code in (([64, -5, 10], BAD_INDEX), ([64, 65, 10], CAPACITY), ([64, 2 ** 31 - 1, 10], CAPACITY)):
        p.status.zero_()
        out, lse = p.attend(q, lens=lens)
        assert int(p.status) == code
        for i in (0, 2):
            k, v = p.values(i)
            assert_attention(out[i].cpu().numpy().astype(np.float64), lse[i].cpu().numpy().astype(np.float64), q[i],
                             k[:lens[i]], v[:lens[i]])
        if lens[1] < 0:
            assert not out[1].any() and torch.isneginf(lse[1]).all()
    for bad in (-1, len(p.big[0]), 2 ** 31 - 1):
        p.status.zero_()
        table = p.table_dev.clone()
        table[0, 1] = bad       # cells 16..31 of sequence 0 are skipped
        out = torch.empty(3, 1, 4, 64, device="cuda")
        lse = torch.empty(3, 1, 4, device="cuda")
        ws = torch.empty(p.cache.workspace_bytes(4, 1), dtype=torch.uint8, device="cuda")
        p.cache.attend(H.to_dev(q), table, _i32(p.lens), out, ws, lse=lse, status=p.status)
        assert int(p.status) == BAD_INDEX
        for i in range(3):
            keep = [c for c in range(64) if i or not 16 <= c < 32]
            k, v = p.values(i)
            assert_attention(out[i].cpu().numpy().astype(np.float64), lse[i].cpu().numpy().astype(np.float64), q[i], k[keep], v[keep])
    p.status.zero_()


@pytest.mark.parametrize("S,top", [(200, 90), (1000, 40)])
def test_large_batches(S, top):
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.integers(0, top, S)]
    p = Pool(lens, "fp8", 2, 64, 16, seed=S)
    p.append(lens)
    q = _query(p.rng, S, 1, 4, 64)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("fmt", ["f16", "int4"])
@pytest.mark.parametrize("heads,T", [(1, 1), (3, 2)])
def test_batches_of_mostly_empty_slots(fmt, heads, T):
    """The few sequences of a large batch, thousands of empty slots before, between and behind them."""
    S = 20011
    held = {7: 900, 8: 3, 9: 64, 42: 65, 297: 1, 300: 17, 9000: 2500, 9255: 33, 9256: 200, 9513: 16, 19999: 130}
    lens = [0] * S
    for i, n in held.items():
        lens[i] = n
    p = Pool(lens, fmt, heads, 64, 16, seed=heads)
    p.append(lens)
    q = _query(p.rng, S, T, 2 * heads, 64)
    out, lse = p.attend(q)
    assert int(p.status) == 0
    for i in held:
        assert_attention(out[i].cpu().numpy().astype(np.float64), lse[i].cpu().numpy().astype(np.float64), q[i], *p.values(i),
                         what=f"slot {i}")
    empty = torch.ones(S, dtype=torch.bool, device="cuda")
    empty[list(held)] = False
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()


def test_runs_of_empty_slots_cost_little():
    """Two sequences whose border falls inside a team's share, with 8,190 empty slots between them or
    behind them: the same list of work, so the same bits, and about the same time (looking at
    the slots one by one took ten times as long)."""
    c = Q.alloc_paged_kv(64, 16, 4, 128, Q.QSA_PAGE_F16)
    for t in c.tensors[:2]:
        t.normal_()
    S, lens = 8192, (150000, 92000)
    table = torch.arange(9375, dtype=torch.int32, device="cuda")[None].expand(S, -1).remainder(64).contiguous()
    q = torch.randn(1, 1, 8, 128, device="cuda").half().expand(S, -1, -1, -1).contiguous()
    ws = torch.empty(c.workspace_bytes(8), dtype=torch.uint8, device="cuda")
    got, times = [], []
    for second in (1, S - 1):
        n = torch.zeros(S, dtype=torch.int32, device="cuda")
        n[0], n[second] = lens
        out, lse = torch.empty(S, 1, 8, 128, device="cuda"), torch.empty(S, 1, 8, device="cuda")
        best = float("inf")
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.attend(q, table, n, out, ws, lse=lse)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
        got.append((out[[0, second]], lse[[0, second]]))
        assert int((lse > float("-inf")).any(-1).sum()) == 2
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert times[1] < 3 * times[0], times


def test_one_very_long_among_short_sequences():
    lens = [1, 0, 30000, 5] + [64] * 30
    p = Pool(lens, "int4", 1, 128, 32, seed=9)
    p.append(lens)
    q = _query(p.rng, len(lens), 2, 8, 128)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_kv_heads(fmt):
    p = Pool([37, 5, 0, 200], fmt, 24, 64, 16, seed=6)
    p.append([37, 5, 0, 200])
    q = _query(p.rng, 4, 3, 24, 64)
    p.check(q, *p.attend(q))


@pytest.mark.parametrize("hq,hkv,dim,T", [(32, 4, 128, 1), (32, 4, 128, 4), (8, 1, 64, 2)])
def test_more_segments_than_teams_and_fewer(hq, hkv, dim, T):
    """Batches around the number of work shares of the GPU, whose borders then fall on segments'
    starts, ends and single tiles."""
    for S, top in ((1, 64 * 500), (3, 64 * 120), (74, 300), (111, 130), (148, 64), (300, 200)):
        lens = [top - i % min(top, 129) for i in range(S)]
        p = Pool(lens, "int4", hkv, dim, 128, seed=S)
        p.append(lens)
        q = _query(p.rng, S, T, hq, dim)
        out, lse = p.attend(q)
        keep = sorted({0, S // 3, S // 2, S - 1})
        for i in keep:
            k, v = p.values(i)
            assert_attention(out[i].cpu().numpy().astype(np.float64), lse[i].cpu().numpy().astype(np.float64), q[i], k, v,
                             what=f"{i} of {S}")
        # the others against the same cache one at a time
        ws = torch.empty(p.cache.workspace_bytes(hq, T), dtype=torch.uint8, device="cuda")
        one, one_lse = torch.empty(1, T, hq, dim, device="cuda"), torch.empty(1, T, hq, device="cuda")
        for i in range(0, S, 7):
            p.cache.attend(H.to_dev(q[i:i + 1]), p.table_dev[i:i + 1], _i32(lens[i:i + 1]), one, ws, lse=one_lse)
            assert torch.allclose(one[0], out[i], rtol=0, atol=2e-5) and torch.allclose(one_lse[0], lse[i], rtol=1e-5, atol=1e-5)


def test_sequences_that_share_pages():
    """Two sequences with a common prefix hold it once."""
    p = Pool([64, 40], "fp8", 2, 64, 16)
    p.append([64, 0])
    p.table[1, :2] = p.table[0, :2]
    p.table_dev = _i32(p.table)
    p.lens[1] = 32
    for rows in p.rows:
        rows[1] = rows[0][:32].copy()
    p.append([0, 5])        # goes on in a page of its own
    q = _query(p.rng, 2, 2, 8, 64)
    p.check(q, *p.attend(q))


def test_pages_past_32_bit_offsets():
    """The last pages of a pool of more than 2^32 bytes (and 2^31 elements)."""
    n, heads, page, dim = 17000, 4, 256, 128        # 262,144 bytes a page: 4.5 GB each for K and V
    pages = [torch.empty(n, heads, page, dim, dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = Q.PagedKV(*pages, Q.QSA_PAGE_F16)
    table = _i32([[n - 1, 5, n - 3]])
    k, v = (torch.randn(600, heads, dim, device="cuda").half() for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(k, v, table, _i32([0]), _i32([0, 600]), status=status)
    back = [torch.empty_like(k) for _ in range(2)]
    cache.read(*back, table, _i32([0]), _i32([0, 600]), status=status)
    assert torch.equal(back[0], k) and torch.equal(back[1], v)
    assert torch.equal(pages[0][n - 3, 1, 600 - 513], k[599, 1])
    q = torch.randn(1, 1, 8, dim, device="cuda").half()
    out, lse = torch.empty(1, 1, 8, dim, device="cuda"), torch.empty(1, 1, 8, device="cuda")
    ws = torch.empty(cache.workspace_bytes(8), dtype=torch.uint8, device="cuda")
    cache.attend(q, table, _i32([600]), out, ws, lse=lse, status=status)
    assert int(status) == 0
    assert_attention(out[0].cpu().numpy().astype(np.float64), lse[0].cpu().numpy().astype(np.float64), q[0].cpu().numpy(),
                     k.cpu().numpy().astype(np.float64), v.cpu().numpy().astype(np.float64))


# ------------------------------------------------------------------ together

def test_parts_of_a_sequence_on_several_devices_are_merged():
    """Two caches hold halves of a sequence; qsa_cp_merge joins their (out, lse)."""
    a, b = Pool([150], "f16", 2, 64, 16, seed=1), Pool([91], "f16", 2, 64, 16, seed=2)
    a.append([150])
    b.append([91])
    q = _query(a.rng, 1, 1, 8, 64)
    parts = [p.attend(q) for p in (a, b)]
    o = torch.stack([x[0][0, 0] for x in parts])
    l = torch.stack([x[1][0, 0] for x in parts])
    out = torch.empty(8, 64, device="cuda")
    Q.cp_merge(o, l, 2, 8, 64, out)
    k, v = (np.concatenate([x, y]) for x, y in zip(a.values(0), b.values(0)))
    want, want_lse, bound, depth = P.attention(q[0], k, v)
    assert (np.abs(out.cpu().numpy() - want[0]) <= 1e-4 * bound[0]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_serving_loop_with_drafts(fmt):
    """Write the newest token and its drafts, attend with all of them, verify, drop the
    rejected ones, go on: every step equals the plain forms on the accepted tokens."""
    T, hq, hkv, dim, vocab = 4, 8, 2, 64, 97
    p = Pool([200] * 5, fmt, hkv, dim, 16, seed=4)
    p.append([50, 1, 0, 100, 31])
    rng = p.rng
    for step in range(6):
        p.append([T] * 5)
        q = _query(rng, 5, T, hq, dim)
        p.check(q, *p.attend(q))
        target = rng.dirichlet(np.full(vocab, 0.3), (5, T)).astype(np.float32)
        draft = ((target[:, :-1] + rng.dirichlet(np.full(vocab, 0.3), (5, T - 1))) / 2).astype(np.float32)
        tokens = np.array([[rng.choice(vocab, p=d / d.sum()) for d in s.astype(np.float64)] for s in draft], np.int32)
        u = rng.random((5, T), np.float32)
        acc, nxt = (torch.empty(5, dtype=torch.int32, device="cuda") for _ in range(2))
        Q.verify_drafts(*(H.to_dev(x) for x in (target, draft, tokens, u)), acc, nxt, status=p.status)
        want = [P.verify(target[i], draft[i], tokens[i], u[i]) for i in range(5)]
        assert [tuple(x) for x in torch.stack([acc, nxt], 1).tolist()] == want
        p.lens = [n - (T - 1) + m for n, (m, _) in zip(p.lens, want)]
        for rows in p.rows:
            for i, n in enumerate(p.lens):
                rows[i] = rows[i][:n]


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_steps_replay_with_other_lengths(fmt):
    """One graph of write + attend + read, replayed as the sequences grow and change places."""
    S, hq, hkv, dim = 3, 8, 2, 128
    p = Pool([300] * S, fmt, hkv, dim, 32, seed=8)
    p.append([40, 1, 130])
    dev = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    k, v, q, back_k, back_v = dev(S, hkv, dim), dev(S, hkv, dim), dev(S, 1, hq, dim), dev(S, hkv, dim), dev(S, hkv, dim)
    first, lens, out, lse = dev(S, dtype=torch.int32), dev(S, dtype=torch.int32), torch.zeros(S, 1, hq, dim, device="cuda"), torch.zeros(S, 1, hq, device="cuda")
    table, start = p.table_dev.clone(), _i32(range(S + 1))
    ws = torch.empty(p.cache.workspace_bytes(hq, 1), dtype=torch.uint8, device="cuda")

    def step():
        p.cache.write(k, v, table, first, start, status=p.status)
        p.cache.attend(q, table, lens, out, ws, lse=lse, status=p.status)
        p.cache.read(back_k, back_v, table, first, start, status=p.status)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        first.copy_(_i32(p.lens))
        lens.copy_(first + 1)
        step()
    stream.synchronize()
    graphs = []
    for _ in range(2):          # two graphs that share the workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        graphs.append(g)
    for it in range(4):
        kn, vn = p.random_rows([1] * S)
        qn = _query(p.rng, S, 1, hq, dim)
        order = p.rng.permutation(S)
        table.copy_(_i32(p.table[order]))
        first.copy_(_i32([p.lens[i] for i in order]))
        lens.copy_(first + 1)
        for d, s in ((k, kn), (v, vn), (q, qn)):
            d.copy_(H.to_dev(s))
        graphs[it % 2].replay()
        torch.cuda.synchronize()
        for j, i in enumerate(order):
            for rows, x, got in ((p.rows[0], kn, back_k), (p.rows[1], vn, back_v)):
                rows[i] = np.concatenate([rows[i], x[j:j + 1]])
            p.lens[i] += 1
            kk, vv = p.values(i)
            assert_attention(out[j].cpu().numpy().astype(np.float64), lse[j].cpu().numpy().astype(np.float64), qn[j], kk, vv)
            assert np.allclose(back_k[j].cpu().numpy(), kk[-1], rtol=2.0 ** -10)
        assert int(p.status) == 0


_FIRST_CALLS = """
import sys
sys.path.insert(0, %r)
import torch
import sparse_attention_decode_02_b200 as Q
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
c = Q.alloc_paged_kv(8, 32, 2, 64, Q.QSA_PAGE_INT4)
k, v = (torch.randn(100, 2, 64, device="cuda").half() for _ in range(2))
x, y = torch.zeros_like(k), torch.zeros_like(v)
q, out = torch.randn(1, 3, 10, 64, device="cuda").half(), torch.zeros(1, 3, 10, 64, device="cuda")
table, first, start, lens, status = i32([[3, 1, 6, 2]]), i32([0]), i32([0, 100]), i32([100]), i32([0])
ws = torch.empty(c.workspace_bytes(10, 3), dtype=torch.uint8, device="cuda")
p, u = torch.full((1, 2, 50), 0.02, device="cuda"), torch.full((1, 2), 0.51, device="cuda")
m, t, d = i32([9]), i32([9]), i32([[0]])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.write(k, v, table, first, start, status=status)
    c.attend(q, table, lens, out, ws, status=status)
    c.read(x, y, table, first, start, status=status)
    Q.verify_drafts(p, None, d, u, m, t, status=status)
g.replay()
torch.cuda.synchronize()
z = torch.einsum("uhd,nhd->uhn", q[0].float(), x.float().repeat_interleave(5, 1)) / 8
z = z.masked_fill(torch.arange(100, device="cuda") > 97 + torch.arange(3, device="cuda")[:, None, None], float("-inf"))
want = torch.einsum("uhn,nhd->uhd", z.softmax(-1), y.float().repeat_interleave(5, 1))
assert torch.allclose(out[0], want, atol=1e-5), (out[0] - want).abs().max()
assert int(status) == 0 and int(m) == 0 and int(t) == 25, (int(status), int(m), int(t))
print("first calls captured")
"""


def test_first_calls_of_a_process_may_be_captured():
    """Nothing that a first call does (attributes, descriptors, loading the kernels) breaks a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS % root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stdout + r.stderr


def test_two_streams_with_a_workspace_each():
    pools = [Pool([6000, 5], "f16", 4, 128, 64, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    data = []
    for p in pools:
        p.append([6000, 5])
        q = _query(p.rng, 2, 1, 32, 128)
        data.append((q, H.to_dev(q), torch.empty(2, 1, 32, 128, device="cuda"), torch.empty(2, 1, 32, device="cuda"),
                     torch.empty(p.cache.workspace_bytes(32, 1), dtype=torch.uint8, device="cuda"), _i32(p.lens)))
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, (_, qd, out, lse, ws, lens) in zip(pools, streams, data):
            p.cache.attend(qd, p.table_dev, lens, out, ws, lse=lse, stream=s)
    torch.cuda.synchronize()
    for p, (q, _, out, lse, _, _) in zip(pools, data):
        p.check(q, out, lse)


def test_same_inputs_give_the_same_bits():
    p = Pool([5000, 1, 700], "fp8", 4, 128, 16, seed=3)
    p.append([5000, 1, 700])
    q = _query(p.rng, 3, 4, 32, 128)
    a, b = p.attend(q), p.attend(q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refuses_a_flat_table():
    p = Pool([64], "f16", 1, 64, 16)
    q, out = torch.zeros(1, 1, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(1, 1, 4, 64, device="cuda")
    ws, rows = torch.zeros(p.cache.workspace_bytes(4), dtype=torch.uint8, device="cuda"), torch.zeros(3, 1, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        p.cache.attend(q, p.table_dev[0], _i32([1]), out, ws)
    with pytest.raises(ValueError):
        p.cache.write(rows, rows, p.table_dev[0], _i32([0]), _i32([0, 3]))


def test_binding_refusals():
    p = Pool([64], "fp8", 2, 64, 16)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.float16, device="cuda")
    out, ws = torch.zeros(1, 1, 4, 64, device="cuda"), torch.zeros(p.cache.workspace_bytes(4), dtype=torch.uint8, device="cuda")
    lens = _i32([1])
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(out=out.half()), dict(out=out[:, :, :2]), dict(lens=lens.long()),
                dict(lens=_i32([1, 1])), dict(table=p.table_dev.long()), dict(q=q[..., ::2]),
                dict(q=q.expand(1, 1, 4, 64)[:, :, ::2]), dict(status=torch.zeros(1, device="cuda"))):
        a = {**dict(q=q, table=p.table_dev, lens=lens, out=out, status=p.status), **bad}
        with pytest.raises(ValueError):
            p.cache.attend(a["q"], a["table"], a["lens"], a["out"], ws, status=a["status"])
    with pytest.raises(Q.QsaError):
        p.cache.attend(q, p.table_dev, lens, out, ws[:256])
    with pytest.raises(Q.QsaError):
        p.cache.attend(torch.zeros(1, 1, 18, 64, dtype=torch.float16, device="cuda"), p.table_dev, lens,
                       torch.zeros(1, 1, 18, 64, device="cuda"), ws)
    rows = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    start = _i32([0, 3])
    for bad in (dict(k=rows.float()), dict(k=rows[:2]), dict(k=rows[:1].expand(3, 2, 64)), dict(k=None),
                dict(k=rows[:, :, ::2]), dict(start=start[:1]), dict(first=lens.float())):
        a = {**dict(k=rows, first=_i32([0]), start=start), **bad}
        with pytest.raises(ValueError):
            p.cache.write(a["k"], rows, p.table_dev, a["first"], a["start"])
    with pytest.raises(ValueError):
        Q.PagedKV(p.parts[0], p.parts[1], Q.QSA_PAGE_FP8)                      # no scales
    with pytest.raises(ValueError):
        Q.PagedKV(p.parts[0][:1].expand(4, 2, 16, 64), p.parts[1][:4], Q.QSA_PAGE_FP8, p.parts[2][:4], p.parts[3][:4])
    with pytest.raises(Q.QsaError):
        z = torch.zeros(2, 2, 24, 64, dtype=torch.float16, device="cuda")
        Q.PagedKV(z, z, Q.QSA_PAGE_F16)
    empty = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    p.cache.write(empty, empty, p.table_dev, _i32([0]), _i32([0, 0]), status=p.status)
    p.cache.attend(q[:0], p.table_dev[:0], lens[:0], out[:0], ws, status=p.status)
    assert int(p.status) == 0
