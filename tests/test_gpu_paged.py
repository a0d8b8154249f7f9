"""The paged-cache kernels against the fp64 oracle.

Tolerances, fixed before the first run:

* output, element by element: the weights p are rounded to bf16 for the product with V (half a
  step, 2^-8 of each) and the result is rounded to bf16 (2^-8 of it), everything else is held in
  fp32: |err| <= 2^-8 |o| + 1.25 * 2^-8 * sum_j p_j |v_j| (the quarter covers the fp32 parts: score
  products of 128 terms, exponentials, sums);
* lse: a score is a sum of 128 products of bf16 numbers in fp32, off by at most
  128 * 2^-24 * sum |q_d k_d| / sqrt(128) (bounded here by |q| |k| / sqrt(128), Cauchy-Schwarz), the
  exponentials by 1e-5: |err| <= ds + 1e-5 + 4 * 2^-24 |lse|;
* weight: every p is off by twice that, relative: |err| <= (2 ds + 3e-5) * got + 2^-22 * |old + got|
  (the sums of at most a few thousand terms of one sign: pairwise in the kernel's fixed order);
* eviction and the write: exact.
"""
import numpy as np
import pytest

from oracle import paged

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
rkv = pytest.importorskip("rolling_kv_chunked_b200")

NAN = float("nan")


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """Streams, their pages in no order and with NaN wherever no token lies, and a chunk."""

    def __init__(self, seed, kvs, qs, hq, hk, page, extra_pages=3, side_by_side=False, look=1.0, spare_rows=5,
                 max_q=None, max_kv=None, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.kvs, self.qs, self.hq, self.hk, self.page = g, list(kvs), list(qs), hq, hk, page
        n = len(kvs)
        self.max_kv = max(list(kvs) + [1]) if max_kv is None else max_kv
        self.max_q = max(qs) if max_q is None else max_q
        width = -(-self.max_kv // page) if width is None else width
        total = sum(-(-k // page) for k in kvs)
        pages = total + extra_pages
        if side_by_side:
            both = torch.full((pages, 2, hk, page, 128), NAN, dtype=torch.bfloat16, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k = torch.full((pages, hk, page, 128), NAN, dtype=torch.bfloat16, device="cuda")
            self.v = torch.full_like(self.k, NAN)
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
        self.table = torch.full((n, width), -7, dtype=torch.int32)  # never to be followed past a stream's pages
        at = 0
        for s, kv in enumerate(kvs):
            c = -(-kv // page)
            self.table[s, :c] = perm[at:at + c]
            at += c
        self.table = self.table.cuda()
        self.kv_len = torch.tensor(kvs, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.rows = sum(qs)
        self.spare = spare_rows
        self.dk = [self.normal(kv, hk, 128) for kv in kvs]
        self.dv = [self.normal(kv, hk, 128) for kv in kvs]
        for s in range(n):
            self.put(s, 0, self.dk[s], self.dv[s])
        self.q = self.normal(self.rows + spare_rows, hq, 128, scale=look)
        self.q[self.rows:] = NAN
        self.pool = rkv.PagePool(self.k, self.v)
        self.batch = rkv.PagedBatch(self.table, self.kv_len, self.q_start, self.max_q, self.max_kv, self.status)

    def normal(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(torch.bfloat16)

    def put(self, s, first, k, v):
        for pages, x in ((self.k, k), (self.v, v)):
            pos = torch.arange(first, first + x.shape[0], device="cuda")
            pages[self.table[s].long()[pos // self.page], :, pos % self.page] = x

    def tokens(self, pages, s, n):
        pos = torch.arange(n, device="cuda")
        return pages[self.table[s].long()[pos // self.page], :, pos % self.page]

    def rows_of(self, s):
        a = int(sum(self.qs[:s]))
        return a, a + self.qs[s]

    def attend(self, causal=True, lse=True, weight=None, out=None, q=None, workspace=None, stream=None):
        out = torch.full((self.rows + self.spare, self.hq, 128), 7.0, dtype=torch.bfloat16, device="cuda") \
            if out is None else out
        z = torch.full((self.rows + self.spare, self.hq), 7.0, device="cuda") if lse else None
        rkv.paged_attention(self.pool, self.batch, self.q if q is None else q, out, causal=causal, lse=z, weight=weight,
                            workspace=workspace, stream=stream)
        return out, z

    def check(self, out, z, causal, weight=None, old=None, look=1.0):
        assert self.batch.poll() == rkv.OK
        o64, z64, w64 = f64(out), None if z is None else f64(z), None if weight is None else f64(weight)
        for s, (n, m) in enumerate(zip(self.kvs, self.qs)):
            a, b = self.rows_of(s)
            q, k, v = f64(self.q[a:b]), f64(self.dk[s]), f64(self.dv[s])
            want, lse, got, reach = paged.attend(q, k, v, causal)
            err = np.abs(o64[a:b] - want)
            tol = 2.0 ** -8 * np.abs(want) + 1.25 * 2.0 ** -8 * reach
            assert (err <= tol).all(), (s, n, m, float(np.nanmax(err - tol)), np.isnan(err).sum())
            size = (np.linalg.norm(q, axis=-1).max(initial=0) * np.linalg.norm(k, axis=-1).max(initial=0)
                    / np.sqrt(128))
            ds = 128 * 2.0 ** -24 * size
            if z is not None:
                blind = np.isinf(lse)
                assert np.array_equal(np.isneginf(z64[a:b]), blind)
                err = np.abs(z64[a:b][~blind] - lse[~blind])
                assert (err <= ds + 1e-5 + 4 * 2.0 ** -24 * np.abs(lse[~blind])).all(), (s, err.max())
            if weight is not None:
                want_w = paged.accumulate(f64(old[s])[:, :n], got, m) if m else f64(old[s])[:, :n]
                err = np.abs(w64[s][:, :n] - want_w)
                assert (err <= (2 * ds + 3e-5) * got + 2.0 ** -22 * np.abs(want_w)).all(), (s, n, m, err.max())
                assert torch.equal(weight[s, :, n:], old[s, :, n:])
        assert (o64[self.rows:] == 7.0).all()
        if z is not None:
            assert (z64[self.rows:] == 7.0).all()


SHAPES = [
    # kvs, qs, q_heads, kv_heads, page
    ([1], [1], 1, 1, 16),
    ([1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300], [1] * 11, 8, 2, 16),
    ([200, 0, 33, 0, 128], [1, 0, 1, 0, 0], 8, 8, 32),              # streams without tokens, without rows
    ([5, 77, 250], [1, 1, 1], 16, 1, 64),
    ([700, 1200], [1, 1], 21, 3, 128),
    ([64, 130, 257], [5, 16, 3], 3, 3, 16),                          # a few rows
    ([90, 3, 17], [5, 3, 17], 14, 2, 32),                            # a chunk that is all there is
    ([300, 140, 9], [40, 129, 9], 8, 2, 16),
    ([513, 260], [257, 260], 5, 5, 128),
    ([400, 129], [33, 127], 10, 2, 64),                              # five heads to one
    ([300], [150], 7, 1, 16),                                        # seven heads to one: 126 of 128 rows
    ([200, 50], [3, 2], 128, 1, 32),                                 # 128 heads to one
    ([260, 31], [4, 9], 96, 2, 16),                                  # 48 heads to one: 96 of 128 rows
    ([1500, 40, 900], [1, 40, 300], 4, 4, 32),                       # tokens and chunks in one call
    ([3, 0, 130], [5, 4, 140], 4, 2, 16),                            # chunks longer than the cache: rows that see nothing
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[1])}-{s[2]}-{s[3]}-p{s[4]}-{max(s[0])}")
def test_attention(shape, causal):
    kvs, qs, hq, hk, page = shape
    c = Cache(11, kvs, qs, hq, hk, page)
    old = torch.rand((len(kvs), hk, c.max_kv + 3), device="cuda")
    weight = old.clone()
    out, z = c.attend(causal, weight=weight)
    c.check(out, z, causal, weight, old)
    again, z2 = c.attend(causal)  # without weights: the same output
    c.check(again, z2, causal)


def test_attention_with_peaked_scores_and_wide_bounds():
    """Scores up to +-40 (a running maximum that jumps), and host bounds far above the lengths."""
    c = Cache(12, [1, 700, 1400], [1, 1, 1], 8, 2, 16, look=8.0, max_q=1, max_kv=6000)
    weight = torch.zeros((3, 2, 6000), device="cuda")
    old = weight.clone()
    out, z = c.attend(weight=weight)
    c.check(out, z, True, weight, old)
    c = Cache(13, [1, 700, 1400], [1, 100, 200], 8, 2, 16, look=8.0, max_q=999, max_kv=6000)
    weight = torch.zeros((3, 2, 6000), device="cuda")
    out, z = c.attend(weight=weight)
    c.check(out, z, True, weight, old)


@pytest.mark.parametrize("qs", [[1, 1], [4, 3], [13, 9], [27, 32], [90, 130]])
def test_one_far_larger_score_at_each_place(qs):
    """The running maximum moves by a hundred at one key: at the start, inside and at the end of a
    tile, in the last tile; the others' weights vanish."""
    kvs = [420, 300]
    for at in (0, 5, 127, 128, 200, 255, 256):
        c = Cache(14, kvs, qs, 4, 2, 16)
        for s in range(2):
            c.dk[s][at] = 3.0
            c.put(s, at, c.dk[s][at:at + 1], c.dv[s][at:at + 1])
        c.q[:c.rows] = (c.q[:c.rows].float() * 0.2 + 2.0).to(torch.bfloat16)
        out, z = c.attend(False)
        c.check(out, z, False)


@pytest.mark.parametrize("qs", [[1, 1, 1], [3, 1, 2], [70, 140, 1]])
def test_strides_and_pages_side_by_side(qs):
    c = Cache(15, [130, 400, 77], qs, 6, 2, 16, side_by_side=True)
    # q, k, v and out as slices of wider rows
    wide = torch.zeros((c.rows + c.spare, 6 + 2 + 2, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :6] = c.q
    q = wide[:, :6]
    back = torch.full((c.rows + c.spare, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, z = c.attend(out=back[:, 1:7], q=q)
    c.check(out, z, True)
    assert (back[:, 0] == 7.0).all() and (back[:, 7] == 7.0).all()


def test_a_cache_with_offsets_past_32_bits():
    """Pages whose element offsets pass 2^32: a page stride of 2^27 elements, 40 pages (10 GB)."""
    stride, pages, hk, page = 1 << 27, 40, 2, 64
    flat = torch.zeros(stride * (pages - 1) + 2 * hk * page * 128, dtype=torch.bfloat16, device="cuda")
    c = Cache(16, [700, 300], [1, 1], 4, hk, page)
    far = [flat.as_strided((pages, hk, page, 128), (stride, page * 128, 128, 1), off) for off in (0, hk * page * 128)]
    n = c.k.shape[0]
    ids = torch.arange(pages - n, pages, device="cuda")
    far[0][ids], far[1][ids] = c.k, c.v
    c.table = torch.where(c.table >= 0, c.table + (pages - n), c.table)
    c.k, c.v = far
    c.pool = rkv.PagePool(*far)
    c.batch = rkv.PagedBatch(c.table, c.kv_len, c.q_start, c.max_q, c.max_kv, c.status)
    out, z = c.attend()
    c.check(out, z, True)
    c.qs, c.max_q = [90, 131], 131
    c.rows = 221
    c.q_start = torch.tensor([0, 90, 221], dtype=torch.int32, device="cuda")
    c.q = c.normal(c.rows + c.spare, 4, 128)
    c.batch = rkv.PagedBatch(c.table, c.kv_len, c.q_start, c.max_q, c.max_kv, c.status)
    weight = torch.zeros((2, hk, 700), device="cuda")
    old = weight.clone()
    out, z = c.attend(weight=weight)
    c.check(out, z, True, weight, old)
    k = c.normal(c.rows, hk, 128)
    rkv.paged_write(c.pool, c.batch, k, k)
    assert torch.equal(c.tokens(c.k, 1, 300)[-131:], k[90:]) and torch.equal(c.tokens(c.v, 0, 700)[-90:], k[:90])
    rkv.paged_evict(c.pool, c.batch, weight, 256, 4, 100, torch.empty((2, hk, 256), dtype=torch.int32, device="cuda"),
                    torch.empty(2, dtype=torch.int32, device="cuda"))
    assert c.batch.poll() == rkv.OK


def test_many_streams():
    """More streams than one warp probes at once, some without rows."""
    n = 1100
    kvs = [(i * 37) % 90 for i in range(n)]
    qs = [min(k, (i * 5) % 4) for i, k in enumerate(kvs)]
    c = Cache(17, kvs, qs, 2, 1, 16)
    old = torch.rand((n, 1, 90), device="cuda")
    weight = old.clone()
    out, z = c.attend(weight=weight)
    c.check(out, z, True, weight, old)
    k, v = c.normal(c.rows + c.spare, 1, 128), c.normal(c.rows + c.spare, 1, 128)
    rkv.paged_write(c.pool, c.batch, k, v)
    for s in range(n):
        a, b = c.rows_of(s)
        assert torch.equal(c.tokens(c.k, s, kvs[s])[kvs[s] - qs[s]:], k[a:b])
    assert c.batch.poll() == rkv.OK


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kvs,qs,hq,hk,page", [
    ([1400], [1100], 40, 40, 16),                # 200 equal units on 148 SMs: a whole wave, and 52 shared in step
    ([700, 690, 710], [260, 250, 256], 16, 16, 64),  # 96 units of nearly one size, none whole: all shared in step
    ([1500, 60, 900, 10, 333], [700, 60, 40, 10, 200], 24, 8, 32),  # shared in a row, cut anywhere
    ([5000], [130], 2, 2, 128),                  # two units, 40 tiles each, over 80 thread blocks
    ([300] * 20, [32] * 20, 20, 20, 16),         # 32 rows: the last of the single-token form
    ([300] * 20, [33] * 20, 20, 20, 16),         # 33: the first of the chunk form
    ([3000, 40], [64, 30], 4, 4, 32),            # half a row tile, alone and beside fewer
    ([260, 90, 33, 16, 400], [16, 1, 8, 2, 4], 8, 4, 16),  # 32 rows and fewer in one batch
    ([900, 64, 2000, 65, 128], [5, 3, 4, 5, 1], 60, 5, 64),  # 12 heads to one: 60 rows and fewer
    ([300] * 20, [65] * 20, 20, 20, 16),         # just above half a row tile
])
def test_shared_work(kvs, qs, hq, hk, page, causal):
    c = Cache(31, kvs, qs, hq, hk, page)
    old = torch.rand((len(kvs), hk, c.max_kv), device="cuda")
    weight = old.clone()
    out, z = c.attend(causal, weight=weight)
    c.check(out, z, causal, weight, old)


@pytest.mark.parametrize("kvs,qs,hq,hk", [
    ([20000], [1], 1, 1),                    # one row in 296 parts
    ([20000], [1], 16, 1),
    ([19000, 37], [5, 1], 6, 1),             # 30 rows, and 6 in one part
    ([9000, 9000, 300], [1, 2, 1], 14, 2),   # six units: 7 and 14 rows
    ([15000], [1], 128, 1),                  # 128 rows in 118 parts
    ([9001, 700], [50, 40], 10, 2),          # two tiles of rows, 125 of 128 used, and a part of them
    ([5000] * 9, [60] * 9, 4, 2),            # 18 units: the last that are gathered
    ([5000] * 19, [60] * 19, 2, 1),          # 19: the first the usual way
])
def test_few_units_in_many_parts(kvs, qs, hq, hk):
    c = Cache(39, kvs, qs, hq, hk, 32)
    out, z = c.attend()
    c.check(out, z, True)


def test_many_streams_with_chunks():
    """More streams, and more blocks of rows, than the plan holds in shared memory."""
    n = 1100
    kvs = [(i * 37) % 120 for i in range(n)]
    qs = [min(k, (i * 7) % 60) for i, k in enumerate(kvs)]
    c = Cache(32, kvs, qs, 2, 2, 16)
    old = torch.rand((n, 2, c.max_kv), device="cuda")
    weight = old.clone()
    out, z = c.attend(weight=weight)
    c.check(out, z, True, weight, old)


@pytest.mark.parametrize("kvs,qs,hk,page", [([1], [1], 1, 16), ([33, 0, 16, 500], [1, 0, 16, 200], 3, 16),
                                            ([129, 128], [129, 1], 8, 128), ([70, 200], [7, 130], 40, 64)])
def test_write(kvs, qs, hk, page):
    c = Cache(18, kvs, qs, hk, hk, page)
    want_k, want_v = c.k.clone(), c.v.clone()
    wide = c.normal(c.rows + c.spare, 2 * hk + 1, 128)
    k, v = wide[:, :hk], wide[:, hk:2 * hk]
    rkv.paged_write(c.pool, c.batch, k, v)
    for s, (n, m) in enumerate(zip(kvs, qs)):
        a, b = c.rows_of(s)
        for pages, x in ((want_k, k), (want_v, v)):
            for i in range(m):
                pos = n - m + i
                pages[c.table[s, pos // page].long(), :, pos % page] = x[a + i]
    assert torch.equal(c.k.view(torch.int16), want_k.view(torch.int16))  # NaN and all: nothing else was touched
    assert torch.equal(c.v.view(torch.int16), want_v.view(torch.int16))
    assert c.batch.poll() == rkv.OK


def _evict_and_check(c, weight, keep, sinks, recent):
    n = len(c.kvs)
    before_k, before_v, before_w = c.k.clone(), c.v.clone(), weight.clone()
    kept = torch.full((n, c.hk, keep), 99, dtype=torch.int32, device="cuda")
    new_len = torch.full((n,), 99, dtype=torch.int32, device="cuda")
    rkv.paged_evict(c.pool, c.batch, weight, keep, sinks, recent, kept, new_len)
    assert c.batch.poll() == rkv.OK
    want_k, want_v, want_w = before_k.clone(), before_v.clone(), before_w.clone()
    host = before_w.cpu().numpy()
    lists = []
    for s, kv in enumerate(c.kvs):
        assert int(new_len[s]) == min(kv, keep)
        for h in range(c.hk):
            places = paged.kept(host[s, h, :kv], keep, sinks, recent)
            assert kept[s, h].tolist() == places + [-1] * (keep - len(places)), (s, h)
            lists.append(places)
            src = torch.tensor(places, dtype=torch.long, device="cuda")
            dst = torch.arange(len(places), device="cuda")
            row = c.table[s].long()
            for want, had in ((want_k, before_k), (want_v, before_v)):
                want[row[dst // c.page], h, dst % c.page] = had[row[src // c.page], h, src % c.page]
            want_w[s, h, :len(places)] = before_w[s, h, src]
    assert torch.equal(c.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), want_v.view(torch.int16))
    assert torch.equal(weight.view(torch.int32), want_w.view(torch.int32))
    return lists


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 16), (100, 0, 100), (100, 100, 0),
                                               (257, 5, 250), (300, 0, 0), (2000, 4, 64), (6000, 1, 1)])
def test_evict(keep, sinks, recent):
    c = Cache(19, [0, 1, 64, 65, 300, 301, 1025, 5000], [0] * 8, 3, 3, 16)
    weight = torch.rand((8, 3, 5003), generator=c.g, device="cuda") ** 4
    _evict_and_check(c, weight, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "zeros", "odd", "few"])
def test_evict_among_equals_and_odd_weights(kind):
    c = Cache(20, [2500, 700], [0, 0], 2, 2, 64)
    weight = torch.rand((2, 2, 2500), generator=c.g, device="cuda")
    if kind == "equal":
        weight[:] = 0.25
    elif kind == "zeros":
        weight[weight < 0.9] = 0.0
        weight[:, :, ::3] *= -1.0  # -0 and 0 are equal
    elif kind == "odd":
        weight[:, :, 5::7] = NAN
        weight[:, :, 3::11] = float("inf")
        weight[:, :, 4::13] = -float("inf")
        weight[:, :, 6::17] = 1e-42  # subnormal
        weight[:, :, 8::19] = -1e-42
    else:
        weight = (weight * 3).round()
    _evict_and_check(c, weight, 600, 7, 33)


@pytest.mark.parametrize("page,n,keep", [(16, 70001, 20011), (128, 70001, 20011), (128, 140001, 70000)])
def test_evict_a_long_stream(page, n, keep):
    c = Cache(21, [n], [0], 2, 2, page)
    weight = torch.rand((1, 2, n), generator=c.g, device="cuda") ** 8
    _evict_and_check(c, weight, keep, 64, 1000)


@pytest.mark.parametrize("max_kv", [700, 4097])
def test_evict_many_heads(max_kv):
    """More heads than SMs, short streams and streams that may be longer."""
    n = 40
    c = Cache(30, [(i * 97) % 700 + 1 for i in range(n)], [0] * n, 4, 4, 16, max_kv=max_kv)
    weight = torch.rand((n, 4, max_kv), generator=c.g, device="cuda") ** 3
    weight[:, 1] = (weight[:, 1] * 2).round()
    _evict_and_check(c, weight, 150, 3, 40)


@pytest.mark.parametrize("qs", [1, 6, 150])
def test_steps_of_a_cache_that_evicts(qs):
    """Write, attend with weights, evict, and again: three streams over many steps, against the
    oracle on plain lists of tokens, which evicts what the device's own weights say."""
    hq, hk, page, keep, sinks, recent = 4, 2, 16, 96, 4, 24
    steps = 7 if qs < 100 else 4
    g = torch.Generator(device="cuda").manual_seed(22)
    width = -(-(keep + qs) // page)
    pool_k = torch.full((3 * width, hk, page, 128), NAN, dtype=torch.bfloat16, device="cuda")
    pool_v = torch.full_like(pool_k, NAN)
    table = torch.randperm(3 * width, generator=g, device="cuda").to(torch.int32).view(3, width)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    weight = torch.full((3, hk, width * page), NAN, device="cuda")  # a slot's first value comes with its token
    pool = rkv.PagePool(pool_k, pool_v)
    length = torch.tensor([70, 20, 0], dtype=torch.int32, device="cuda")
    hist = []
    for s in range(3):
        n = int(length[s])
        k, v = (torch.randn((n, hk, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
        pos = torch.arange(n, device="cuda")
        pool_k[table[s].long()[pos // page], :, pos % page] = k
        pool_v[table[s].long()[pos // page], :, pos % page] = v
        weight[s, :, :n] = 0.5
        hist.append([[f64(k)[:, h] for h in range(hk)], [f64(v)[:, h] for h in range(hk)]])
    q_start = torch.tensor([0, qs, 2 * qs, 3 * qs], dtype=torch.int32, device="cuda")
    for step in range(steps):
        length += qs
        batch = rkv.PagedBatch(table, length, q_start, qs, width * page, status)
        q, k, v = (torch.randn((3 * qs, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hk, hk))
        out = torch.empty_like(q)
        old = weight.clone()
        rkv.paged_write(pool, batch, k, v)
        rkv.paged_attention(pool, batch, q, out, weight=weight)
        assert batch.poll() == rkv.OK
        for s in range(3):
            a, n = s * qs, int(length[s])
            for h in range(hk):
                for i, x in ((0, k), (1, v)):
                    hist[s][i][h] = np.concatenate([hist[s][i][h], f64(x[a:a + qs])[:, h]])
            ks, vs = (np.stack(hist[s][i], 1) for i in (0, 1))
            want, _, got, reach = paged.attend(f64(q[a:a + qs]), ks, vs, True)
            err = np.abs(f64(out[a:a + qs]) - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 1.25 * 2.0 ** -8 * reach).all(), (step, s)
            want_w = got + np.concatenate([f64(old[s])[:, :n - qs], np.zeros((hk, qs))], 1)
            ds = 128 * 2.0 ** -24 * np.linalg.norm(f64(q), axis=-1).max() * np.linalg.norm(ks, axis=-1).max() / 128 ** 0.5
            assert (np.abs(f64(weight[s])[:, :n] - want_w) <= (2 * ds + 3e-5) * got + 2.0 ** -22 * want_w).all(), (step, s)
        kept = torch.empty((3, hk, keep), dtype=torch.int32, device="cuda")
        host = weight.cpu().numpy()
        before = [int(x) for x in length]
        rkv.paged_evict(pool, batch, weight, keep, sinks, recent, kept, length)  # the lengths in place
        assert batch.poll() == rkv.OK
        for s in range(3):
            assert int(length[s]) == min(before[s], keep)
            for h in range(hk):
                places = paged.kept(host[s, h, :before[s]], keep, sinks, recent)
                assert kept[s, h, :len(places)].tolist() == places
                for i in (0, 1):
                    hist[s][i][h] = hist[s][i][h][places]


def test_same_call_same_bits():
    for qs in ([1, 1, 1], [60, 200, 9]):
        c = Cache(23, [900, 3000, 41], qs, 8, 2, 16)
        first = None
        for _ in range(3):
            weight = torch.ones((3, 2, 3000), device="cuda")
            got = [t.clone() for t in (*c.attend(weight=weight), weight)]
            first = first or got
            for x, y in zip(got, first):
                assert torch.equal(x[:c.rows] if x.dim() != 3 or x.dtype != torch.float32 else x,
                                   y[:c.rows] if y.dim() != 3 or y.dtype != torch.float32 else y)


@pytest.mark.parametrize("qs,later", [([1, 1, 1], [1, 0, 1]), ([30, 7, 90], [1, 100, 20])])
def test_captured_and_replayed_with_other_lengths(qs, later):
    """A graph reads the lengths, pages and rows of the moment: replayed after they changed."""
    c = Cache(24, [500, 130, 260], qs, 4, 2, 16, max_q=max(qs + later), spare_rows=8)
    weight = torch.zeros((3, 2, c.max_kv), device="cuda")
    out = torch.full((c.rows + c.spare, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((c.rows + c.spare, 4), 7.0, device="cuda")
    kx = c.normal(c.rows + c.spare, 2, 128)
    ws = torch.empty(rkv.paged_workspace_bytes(c.pool, c.batch, c.rows + c.spare, 4, True), dtype=torch.uint8, device="cuda")
    kept = torch.empty((3, 2, 200), dtype=torch.int32, device="cuda")
    new_len = torch.empty(3, dtype=torch.int32, device="cuda")

    def call():
        rkv.paged_write(c.pool, c.batch, kx, kx)
        rkv.paged_attention(c.pool, c.batch, c.q, out, lse=z, weight=weight, workspace=ws)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        trim = torch.cuda.CUDAGraph()
        with torch.cuda.graph(trim, stream=side):
            rkv.paged_evict(c.pool, c.batch, weight, 200, 2, 20, kept, new_len)

    def step():
        old = weight.clone()
        out.fill_(7.0)
        z.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for s, (n, m) in enumerate(zip(c.kvs, c.qs)):
            a, b = c.rows_of(s)
            for d in (c.dk, c.dv):
                d[s] = torch.cat([d[s][:n - m], kx[a:b]])
        c.check(out, z, True, weight, old)

    step()
    c.kvs, c.qs = [400, 130, 255], list(later)
    for s, n in enumerate(c.kvs):
        c.dk[s], c.dv[s] = c.dk[s][:n], c.dv[s][:n]
    c.kv_len.copy_(torch.tensor(c.kvs, dtype=torch.int32))
    c.q_start.copy_(torch.tensor(np.concatenate([[0], np.cumsum(c.qs)]), dtype=torch.int32))
    c.rows, total = sum(c.qs), c.rows + c.spare
    c.q[:] = c.normal(total, 4, 128)
    kx.copy_(c.normal(total, 2, 128))
    step()
    host = weight.cpu().numpy()
    trim.replay()
    torch.cuda.synchronize()
    assert new_len.tolist() == [200, 130, 200]
    for s, n in enumerate(c.kvs):
        for h in range(2):
            places = paged.kept(host[s, h, :n], 200, 2, 20)
            assert kept[s, h, :len(places)].tolist() == places


def test_two_streams_with_workspaces_of_their_own():
    cs = [Cache(25 + i, [900, 2000], [1, 1] if i else [100, 30], 8, 2, 16) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                got.append((c, *c.attend()))
    torch.cuda.synchronize()
    for c, out, z in got:
        c.check(out, z, True)
    c = cs[0]  # a stream given by argument, and as a number
    for st in (streams[0], streams[0].cuda_stream):
        torch.cuda.synchronize()
        out, z = c.attend(stream=st)
        torch.cuda.synchronize()
        c.check(out, z, True)


def test_bad_lengths_and_pages_are_reported_and_not_followed():
    for qs in ([1, 1, 1], [20, 130, 3]):
        c = Cache(26, [200, 300, 100], qs, 4, 2, 16, max_q=max(qs))
        weight = torch.ones((3, 2, c.max_kv), device="cuda")
        old = weight.clone()
        c.kv_len[1] = 301  # above max_kv
        out, z = c.attend(weight=weight)
        assert c.batch.poll() == rkv.ERR_PAGE and c.batch.poll() == rkv.OK
        a, b = c.rows_of(1)
        assert (out[a:b] == 7.0).all() and torch.equal(weight[1], old[1])
        assert torch.isfinite(out[:a].float()).all() and torch.isfinite(out[b:c.rows].float()).all()
        c.kv_len[1] = -1
        c.attend()
        assert c.batch.poll() == rkv.ERR_PAGE
        k = c.normal(c.rows, 2, 128)
        before = c.k.clone()
        rkv.paged_write(c.pool, c.batch, k, k)
        assert c.batch.poll() == rkv.ERR_PAGE
        assert torch.equal(c.tokens(c.k, 0, 200)[-qs[0]:], k[:qs[0]])
        kept = torch.zeros((3, 2, 50), dtype=torch.int32, device="cuda")
        new_len = torch.zeros(3, dtype=torch.int32, device="cuda")
        rkv.paged_evict(c.pool, c.batch, weight, 50, 1, 1, kept, new_len)
        assert c.batch.poll() == rkv.ERR_PAGE
        assert new_len.tolist() == [50, 0, 50] and (kept[1] == -1).all()
        c = Cache(27, [200, 300, 100], qs, 4, 2, 16, max_q=max(qs))
        c.q_start[1] = c.rows + c.spare + 1  # rows outside the tensors
        c.attend(weight=torch.ones((3, 2, c.max_kv), device="cuda"))
        assert c.batch.poll() == rkv.ERR_PAGE
        for bad in (-1, c.k.shape[0], 1 << 30):
            c = Cache(28, [200, 300, 100], qs, 4, 2, 16, max_q=max(qs))
            c.table[1, 300 // 16] = bad  # the chunk's last page
            out, z = c.attend(weight=torch.ones((3, 2, c.max_kv), device="cuda"))
            assert c.batch.poll() == rkv.ERR_PAGE
            a, b = c.rows_of(0)
            want = paged.attend(f64(c.q[a:b]), f64(c.dk[0]), f64(c.dv[0]), True)
            assert (np.abs(f64(out[a:b]) - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 1.25 * 2.0 ** -8 * want[3]).all()
            rkv.paged_write(c.pool, c.batch, k, k)
            assert c.batch.poll() == rkv.ERR_PAGE


@pytest.mark.parametrize("qs", [[2, 1, 2, 1], [40, 9, 130, 3]])
def test_row_ranges_that_decrease_are_reported(qs):
    """q_start falls back in the middle: reported by every call, and what lies outside the streams' tokens and the
    tensors' rows stays as it was."""
    c = Cache(33, [200, 300, 100, 260], qs, 4, 2, 16, max_q=sum(qs))
    weight = torch.ones((4, 2, c.max_kv), device="cuda")
    c.q_start.copy_(torch.tensor([0, c.rows, 1, 3, 3 + qs[3]], dtype=torch.int32))
    out, z = c.attend(weight=weight)
    assert c.batch.poll() == rkv.ERR_PAGE
    assert (out[c.rows:] == 7.0).all() and (z[c.rows:] == 7.0).all()
    for s, n in enumerate(c.kvs):
        assert (weight[s, :, n:] == 1).all()
    k = c.normal(c.rows + c.spare, 2, 128)
    spare = [p for p in range(c.k.shape[0]) if p not in set(c.table.flatten().tolist())]
    rkv.paged_write(c.pool, c.batch, k, k)
    assert c.batch.poll() == rkv.ERR_PAGE
    assert torch.isnan(c.k[spare]).all()
    for s, n in enumerate(c.kvs):  # the places behind a stream's last token on its last page
        if n % 16:
            assert torch.isnan(c.k[c.table[s, n // 16].long(), :, n % 16:]).all()


@pytest.mark.parametrize("qs", [[1, 2, 1], [20, 3, 9], [70, 140, 1]])
def test_rows_from_the_middle_and_pages_in_two_streams(qs):
    """The chunk's rows start behind the tensors' first, and two streams hold the same pages at their start; the
    page lists are columns of a wider tensor."""
    c = Cache(34, [290, 330, 50], qs, 6, 2, 32)
    same = 64  # tokens of two pages
    wide = torch.full((3, c.table.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
    wide[:, :-3] = c.table
    wide[1, :2] = wide[0, :2]
    c.dk[1][:same], c.dv[1][:same] = c.dk[0][:same], c.dv[0][:same]
    skip = c.spare - 1  # rows before the chunk's; one is left behind it
    c.q_start += skip
    q = torch.full_like(c.q, NAN)
    q[skip:skip + c.rows] = c.q[:c.rows]
    c.batch = rkv.PagedBatch(wide[:, :-3], c.kv_len, c.q_start, c.max_q, c.max_kv, c.status)
    old = torch.rand((3, 2, c.max_kv), device="cuda")
    weight = old.clone()
    out, z = c.attend(weight=weight, q=q)
    for t in (out, z):
        assert (t[:skip] == 7.0).all() and (t[skip + c.rows:] == 7.0).all()
    c.check(out[skip:], z[skip:], True, weight, old)
    k, v = c.normal(c.rows + c.spare, 2, 128), c.normal(c.rows + c.spare, 2, 128)
    rkv.paged_write(c.pool, c.batch, k, v)
    assert c.batch.poll() == rkv.OK
    c.table = wide
    for s, n in enumerate(c.kvs):
        a, b = c.rows_of(s)
        assert torch.equal(c.tokens(c.k, s, n)[n - c.qs[s]:], k[skip + a:skip + b])
        assert torch.equal(c.tokens(c.v, s, n)[n - c.qs[s]:], v[skip + a:skip + b])


@pytest.mark.parametrize("qs", [[1, 1, 1], [20, 3, 9], [70, 140, 1]])
def test_two_graphs_of_one_workspace(qs):
    """Two captured calls of different pages and rows share a workspace and are replayed in turn."""
    c = [Cache(35 + i, [500 - 90 * i, 300, 40 + 60 * i], qs, 8, 2, 16) for i in range(2)]
    size = max(rkv.paged_workspace_bytes(x.pool, x.batch, x.rows + x.spare, 8, True) for x in c)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    weight = [torch.zeros((3, 2, x.max_kv), device="cuda") for x in c]
    outs = [torch.full_like(x.q, 7.0) for x in c]
    graphs = []
    torch.cuda.synchronize()
    for x, w, o in zip(c, weight, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.attend(lse=False, weight=w, out=o, workspace=ws)
        graphs.append(g)
    ws.fill_(255)
    for i in (0, 1, 1, 0):
        old = weight[i].clone()
        graphs[i].replay()
        c[i].check(outs[i], None, True, weight[i], old)


def test_refusals_on_the_device():
    c = Cache(29, [200, 300], [1, 1], 4, 2, 16)
    out = torch.empty_like(c.q)
    small = torch.empty(0, dtype=torch.uint8, device="cuda")
    weight = torch.zeros((2, 2, 300), device="cuda")

    def refused(code, f, *a, **kw):
        with pytest.raises(rkv.RkvError) as e:
            f(*a, **kw)
        assert e.value.code == code

    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q, c.q)
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q.float(), out)
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q[:, :3], out[:, :3])
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q, out[:-1])
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q, out, weight=weight[:, :, :299].contiguous())
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q, out, weight=weight[:, :, ::2])
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, c.batch, c.q, out, lse=torch.zeros((3, 4), device="cuda"))
    refused(rkv.ERR_CAPACITY, rkv.paged_attention, c.pool, c.batch, c.q, out, weight=weight, workspace=small)
    refused(rkv.ERR_ARG, rkv.paged_write, c.pool, c.batch, c.q, c.q)
    refused(rkv.ERR_ARG, rkv.PagePool, c.k, c.v[:-1])
    refused(rkv.ERR_ARG, rkv.PagePool, c.k.transpose(1, 2), c.v.transpose(1, 2))
    refused(rkv.ERR_ARG, rkv.PagedBatch, c.table.long(), c.kv_len, c.q_start, 1, 300)
    refused(rkv.ERR_ARG, rkv.PagedBatch, c.table, c.kv_len, c.q_start[:-1], 1, 300)
    kept = torch.empty((2, 2, 10), dtype=torch.int32, device="cuda")
    refused(rkv.ERR_ARG, rkv.paged_evict, c.pool, c.batch, weight, 11, 1, 1, kept, torch.empty_like(c.kv_len))
    refused(rkv.ERR_ARG, rkv.paged_evict, c.pool, c.batch, weight, 10, 6, 5, kept, torch.empty_like(c.kv_len))
    none = rkv.PagedBatch(c.table, c.kv_len, None, 1, 300)
    refused(rkv.ERR_ARG, rkv.paged_attention, c.pool, none, c.q, out)
    empty = rkv.PagedBatch(c.table[:0], c.kv_len[:0], c.q_start[:1], 0, 300)
    rkv.paged_attention(c.pool, empty, c.q[:0], out[:0])
    rkv.paged_write(c.pool, empty, c.q[:0, :2], c.q[:0, :2])
    torch.cuda.synchronize()


def test_weights_without_columns_are_refused():
    c = Cache(37, [200, 300], [1, 1], 4, 2, 16)
    with pytest.raises(rkv.RkvError) as e:
        c.attend(weight=torch.zeros((2, 2, 0), device="cuda"))
    assert e.value.code == rkv.ERR_ARG


def test_poll_follows_its_stream():
    """A report that comes after the poll on the same stream is not wiped out by the poll's clear."""
    c = Cache(38, [200, 300], [1, 1], 4, 2, 16)
    c.kv_len[1] = 301
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(50):
            c.attend()
            assert c.batch.poll() == rkv.ERR_PAGE


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kvs,qs,hq,hk", [
    ([2], [3], 1, 1),
    ([3, 40], [5, 4], 4, 2),               # 10 rows of a KV head: scores kept
    ([9, 2, 100], [16, 3, 1], 2, 2),       # 16
    ([0, 1, 700], [4, 4, 4], 12, 3),       # 16, a stream without tokens
    ([3, 40], [20, 11], 2, 2),             # 20: scores formed again
    ([5, 3000], [9, 16], 4, 2),            # 32
    ([260, 40], [300, 7], 4, 2),           # tiles of 128 rows
])
def test_weights_of_rows_that_see_nothing(kvs, qs, hq, hk, causal):
    """Chunks longer than the cache: their first rows see no key and give none weight, twice in a row."""
    c = Cache(40, kvs, qs, hq, hk, 16)
    weight = torch.rand((len(kvs), hk, c.max_kv + 2), device="cuda")
    for _ in range(2):
        old = weight.clone()
        out, z = c.attend(causal, weight=weight)
        c.check(out, z, causal, weight, old)


def test_a_page_table_too_narrow_for_the_bound_is_refused():
    """A column slice of a wider table: its stride would reach max_kv, its columns do not."""
    c = Cache(41, [30, 20], [1, 1], 4, 2, 16)
    wide = torch.zeros((2, 5), dtype=torch.int32, device="cuda")
    wide[:, :2] = c.table
    weight = torch.zeros((2, 2, 64), device="cuda")
    kept = torch.empty((2, 2, 8), dtype=torch.int32, device="cuda")
    k = c.normal(c.rows, 2, 128)
    out = torch.empty_like(c.q)

    def calls(b):
        yield lambda: rkv.paged_write(c.pool, b, k, k)
        yield lambda: rkv.paged_attention(c.pool, b, c.q, out)
        yield lambda: rkv.paged_workspace_bytes(c.pool, b, c.rows, 4)
        yield lambda: rkv.paged_evict(c.pool, b, weight, 8, 1, 1, kept, torch.empty_like(c.kv_len))

    for call in calls(rkv.PagedBatch(wide[:, :2], c.kv_len, c.q_start, 1, 33)):
        with pytest.raises(rkv.RkvError) as e:
            call()
        assert e.value.code == rkv.ERR_ARG
    for call in calls(rkv.PagedBatch(wide[:, :2], c.kv_len, c.q_start, 1, 32)):  # all of the columns
        call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("hq,n", [(4, 8), (8, 16), (128, 1000)])  # 16 and 32 rows of a KV head, and blocks of two tokens
def test_row_ranges_whose_differences_pass_31_bits(hq, n):
    """q_start falls by so much that every difference wraps to a positive number, and the same rows come twice: reported,
    and neither rows outside the streams' nor anything behind the workspace is touched."""
    c = Cache(46, [1000] * 10, [n] + [0] * 9, hq, 2 if hq < 128 else 1, 16, max_q=n)
    far = (1 << 31) - 1
    c.q_start.copy_(torch.tensor([0, n, far, -far - 1, -1] * 2 + [0], dtype=torch.int64).to(torch.int32))
    weight = torch.ones((10, c.hk, 1003), device="cuda")
    size = rkv.paged_workspace_bytes(c.pool, c.batch, c.rows + c.spare, hq, True)
    ws = torch.full((size + 65536,), 85, dtype=torch.uint8, device="cuda")
    out, z = c.attend(weight=weight, workspace=ws)
    assert c.batch.poll() == rkv.ERR_PAGE
    assert (ws[size:] == 85).all()
    assert (out[n:] == 7.0).all() and (z[n:] == 7.0).all() and (weight[:, :, 1000:] == 1).all()
    k = c.normal(c.rows + c.spare, c.hk, 128)
    rkv.paged_write(c.pool, c.batch, k, k)
    assert c.batch.poll() == rkv.ERR_PAGE


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("qs", [[1, 1, 1], [5, 2, 3], [9, 30, 16], [70, 140, 1]])
def test_calls_that_feed_each_other_without_a_pause(qs, captured):
    """Each call reads what the one before it wrote (queries, weights, pages), the launches overlapping: the same
    bits as with every call waited for."""
    results = []
    for paused in (True, False):
        c = Cache(43, [900, 1500, 333], qs, 4, 2, 16)
        weight = torch.rand((3, 2, c.max_kv), generator=c.g, device="cuda")
        bufs = [c.q.clone(), torch.zeros_like(c.q), torch.zeros_like(c.q)]
        kept = torch.empty((3, 2, 300), dtype=torch.int32, device="cuda")
        new_len = torch.empty(3, dtype=torch.int32, device="cuda")
        ws = torch.empty(rkv.paged_workspace_bytes(c.pool, c.batch, c.q.shape[0], 4, True), dtype=torch.uint8, device="cuda")

        def steps():
            for i in range(12):
                a, b = bufs[i % 3], bufs[(i + 1) % 3]
                for call in (lambda: rkv.paged_attention(c.pool, c.batch, a, b, weight=weight, workspace=ws),
                             lambda: rkv.paged_write(c.pool, c.batch, b[:, :2], b[:, 2:]),
                             lambda: rkv.paged_evict(c.pool, c.batch, weight, 300, 2, 100, kept, new_len)):
                    call()
                    if paused:
                        torch.cuda.synchronize()

        torch.cuda.synchronize()
        if captured and not paused:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps()
            for _ in range(4):
                graph.replay()
        else:
            for _ in range(4):
                steps()
        torch.cuda.synchronize()
        assert c.batch.poll() == rkv.OK
        results.append([t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).clone()
                        for t in (c.k, c.v, weight, kept, *(b[:c.rows] for b in bufs))])
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kvs,qs", [([2], [3]), ([3, 40, 0], [5, 4, 2]), ([130, 20], [140, 33])])
def test_write_of_a_chunk_longer_than_its_stream(kvs, qs):
    """Rows at places before the first are left out, the others written, and none of it is an error: as in the
    attention, where those rows see nothing."""
    c = Cache(42, kvs, qs, 2, 2, 16)
    want_k, want_v = c.k.clone(), c.v.clone()
    k, v = c.normal(c.rows, 2, 128), c.normal(c.rows, 2, 128)
    rkv.paged_write(c.pool, c.batch, k, v)
    for s, (n, m) in enumerate(zip(kvs, qs)):
        a, _ = c.rows_of(s)
        for i in range(max(0, m - n), m):
            pos = n - m + i
            for pages, x in ((want_k, k), (want_v, v)):
                pages[c.table[s, pos // 16].long(), :, pos % 16] = x[a + i]
    assert torch.equal(c.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), want_v.view(torch.int16))
    assert c.batch.poll() == rkv.OK


@pytest.mark.parametrize("hq,hk,qs,spare", [(16, 1, [1, 1], 5), (4, 4, [3, 16], 40), (3, 1, [5, 2], 300)])
def test_weights_without_kept_scores(hq, hk, qs, spare):
    """Host bounds for which the scores would pass what a call keeps: the weights come from K again, in a workspace of
    ordinary size."""
    bound = (1 << 30) // ((sum(qs) + spare) * hq) + 64
    c = Cache(47, [700, 90], qs, hq, hk, 128, max_kv=bound, spare_rows=spare)
    assert rkv.paged_workspace_bytes(c.pool, c.batch, c.rows + spare, hq, True) < 1 << 27
    weight = torch.rand((2, hk, bound), device="cuda")
    for causal in (True, False):
        old = weight.clone()
        out, z = c.attend(causal, weight=weight)
        c.check(out, z, causal, weight, old)


def test_host_numbers_past_31_bits_are_refused():
    c = Cache(44, [200, 300], [1, 1], 4, 2, 16)
    weight = torch.zeros((2, 2, 300), device="cuda")
    kept = torch.empty((2, 2, 10), dtype=torch.int32, device="cuda")
    for far in (1 << 31, (1 << 32) + 1, -(1 << 32)):
        for call in (lambda: rkv.PagedBatch(c.table, c.kv_len, c.q_start, far, 300),
                     lambda: rkv.PagedBatch(c.table, c.kv_len, c.q_start, 1, far),
                     lambda: rkv.paged_evict(c.pool, c.batch, weight, 10, far, 1, kept, torch.empty_like(c.kv_len)),
                     lambda: rkv.paged_evict(c.pool, c.batch, weight, 10, 1, far, kept, torch.empty_like(c.kv_len)),
                     lambda: rkv.paged_workspace_bytes(c.pool, c.batch, far, 4),
                     lambda: rkv.paged_workspace_bytes(c.pool, c.batch, 2, far)):
            with pytest.raises(rkv.RkvError) as e:
                call()
            assert e.value.code in (rkv.ERR_ARG, rkv.ERR_UNSUPPORTED)
    torch.cuda.synchronize()


def test_a_failed_call_leaves_no_error_for_the_next():
    """A poll inside a capture is refused by CUDA; calls of the rolling window after it do not report that."""
    import ctypes
    rt = ctypes.CDLL("libcudart.so.12")
    c = Cache(45, [200], [1], 4, 2, 16)
    x = [torch.zeros(1024, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    st, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert rt.cudaStreamBeginCapture(st, 1) == 0  # this thread's calls only
    assert c.batch.poll(side) == rkv.ERR_CUDA
    assert rt.cudaStreamEndCapture(st, ctypes.byref(graph)) != 0  # the poll has spoilt it
    rt.cudaGetLastError()
    rkv.flow_x0_renoise(*x[:3], 0.5, 0.25, x[3], x[4])
    torch.cuda.synchronize()
    assert c.batch.poll() == rkv.OK


def test_thousands_of_units_of_one_tile():
    """Odd chunks of two query tiles and one, of one key tile each or none: 2000 units a call, again and again, every
    wait answered and the same bits each time."""
    kvs = [0, 1, 9, 14, 20, 18, 0, 11, 2, 16, 33, 128, 127, 100] * 3
    qs = [1, 249, 9, 97, 20, 144, 287, 193, 41, 101, 33, 127, 3, 55] * 3
    c = Cache(48, kvs, qs, 127, 1, 16, spare_rows=1)
    old = torch.rand((len(kvs), 1, c.max_kv), device="cuda")
    weight = old.clone()
    first = c.attend(False, weight=weight)
    c.check(*first, False, weight, old)
    w = torch.empty_like(weight)
    for _ in range(300):
        w.copy_(old)
        out, z = c.attend(False, weight=w)
        assert torch.equal(out[:c.rows], first[0][:c.rows]) and torch.equal(w, weight)
    assert c.batch.poll() == rkv.OK
