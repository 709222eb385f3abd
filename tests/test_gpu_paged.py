"""The paged K/V cache on the GPU, through the binding: append, decode and prompt attention against the FP64
oracle, the operations on pages against the oracle's list walks, and all of them together.

Tolerance of the attention, element by element (u = half a step of the 16-bit type, 2^-11 or 2^-8):
    |got - want| <= u |want| + A (u + e),   A = sum_c p_c |v_c|
the output's rounding, and the rounding of every weight p_c to 16 bits.  e bounds the relative error of
a weight and of the sum: exp2 (2^-21 for the two), the FP32 sums (n 2^-24), and an error of the score,
2^-23 hd scale max_c sum_d |q_d k_cd|, in exponent and maximum, so twice.  FP16 values below 2^-14 are
spaced 2^-24: 2^-25 more for the output, and n 2^-25 max |v| for the weights (the largest is at least 1).
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from store_kv_attention_b200 import build_lib
    build_lib.build()
    import store_kv_attention_b200 as m
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


def _check(got, res, dtype, hd, scale, n, vmax=None):
    want, mag, reach = res
    got = _np(got) if isinstance(got, torch.Tensor) else got
    u = 2.0 ** -11 if dtype == FP16 else 2.0 ** -8
    e = 2.0 ** -21 + n * 2.0 ** -24 + 2 * 2.0 ** -23 * hd * scale * np.nan_to_num(reach)[..., None]
    tol = u * np.abs(want) + mag * (u + e) * 1.01
    if dtype == FP16:
        tol = tol + 2.0 ** -25 * (1 + n * vmax)
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / np.maximum(tol, 1e-30)).max()
    assert worst <= 1.0, f"{worst:.3g} of the tolerance"


class Rig:
    """A cache whose sequences hold random K and V in pages of a random order; everything else is NaN."""

    def __init__(self, tl, lens, *, kv, group, hd, page, dtype, layers=2, seed=0, spare=0, seqs=None, n_lanes=None, split=0):
        self.tl, self.hd, self.dtype, self.kv, self.heads, self.page = tl, hd, dtype, kv, kv * group, page
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        max_pages = max(1, max(need)) + spare
        n_pages = sum(need) + 3
        n_seqs = len(lens) if seqs is None else max(seqs) + 2
        desc = tl.PagedDesc(layers, n_pages, page, kv, hd, n_seqs, max_pages, tl.TL_KV_FP16 if dtype == FP16 else tl.TL_KV_BF16)
        self.cache = tl.PagedCache(desc, self.heads, n_lanes or len(lens), split_rows=split)
        self.cache.k.fill_(float("nan"))
        self.cache.v.fill_(float("nan"))
        order = rng.permutation(n_pages).astype(np.int32)
        self.seqs = list(range(len(lens))) if seqs is None else seqs
        table = np.full((n_seqs, max_pages), -1, np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        at = 0
        for b, n in enumerate(lens):
            table[self.seqs[b], :need[b]] = order[at:at + need[b]]
            for j in range(need[b]):
                m = min(page, n - j * page)
                for pool in (self.cache.k, self.cache.v):
                    pool[:, int(order[at + j]), :, :m] = torch.randn((layers, kv, m, hd), generator=g, device="cuda").to(dtype)
            at += need[b]
        self.table = table
        self.cache.table.copy_(torch.from_numpy(table))
        self.cache.refs[torch.from_numpy(order[:at].astype(np.int64)).cuda()] = 1
        self.lens, self.g = list(lens), g

    def queries(self, n, sharp=1.0):
        return (torch.randn((n, self.heads, self.hd), generator=self.g, device="cuda") * sharp).to(self.dtype)

    def pools(self, layer):
        return _np(self.cache.k[layer]), _np(self.cache.v[layer])

    def vmax(self, layer):
        return float(np.nanmax(np.abs(self.pools(layer)[1])))

    def check_decode(self, layer, q, out, lens=None, scale=None):
        lens = self.lens if lens is None else lens
        scale = scale or self.hd ** -0.5
        res = paged_oracle.decode(*self.pools(layer), self.table, _np(q), lens, self.seqs, scale)
        _check(out, res, self.dtype, self.hd, scale, max(max(lens), 1), self.vmax(layer))

    def check_prompt(self, layer, q, cu, out, kv=None, scale=None):
        kv = self.lens if kv is None else kv
        scale = scale or self.hd ** -0.5
        res = paged_oracle.prompt(*self.pools(layer), self.table, _np(q), cu, kv, self.seqs, scale)
        inside = ~np.isnan(res[0]).any(axis=(1, 2))
        got = _np(out)
        assert np.isnan(got[~inside]).all(), "rows outside every lane were written"
        _check(got[inside], [r[inside] for r in res], self.dtype, self.hd, scale, max(max(kv), 1), self.vmax(layer))

    def ok(self):
        assert self.tl.poll_status(self.cache) == self.tl.TL_OK


# ---------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("kv,hd,page,dtype", [(8, 128, 16, BF16), (1, 64, 128, FP16), (3, 128, 32, FP16), (16, 64, 64, BF16)])
def test_append_writes_rows_where_the_table_says(tl, kv, hd, page, dtype):
    lens = [40, 0, 129, 7, 300]
    rig = Rig(tl, [n + 20 for n in lens], kv=kv, group=1, hd=hd, page=page, dtype=dtype)
    start = [3, 0, 17, 20, 0]
    cu = np.cumsum([2] + lens)            # the first two rows and the last three belong to nobody
    rows = int(cu[-1]) + 3
    wide = torch.randn((rows, 3, kv, hd), generator=rig.g, device="cuda").to(dtype)   # K and V inside a wider row
    k, v = wide[:, 1], wide[:, 2]
    want = [rig.cache.k.clone(), rig.cache.v.clone()]
    for b, n in enumerate(lens):
        for i in range(n):
            pos = start[b] + i
            for pool, x in zip(want, (k, v)):
                pool[1, rig.table[b, pos // page], :, pos % page] = x[cu[b] + i]
    tl.paged_append(rig.cache, 1, k, v, _i32(start), cu_rows=_i32(cu.tolist()))
    rig.ok()
    for a, b in zip((rig.cache.k, rig.cache.v), want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_append_skips_what_it_may_not_write(tl):
    """Out of range, no page, a shared page: not written and reported; the other lanes' rows are."""
    rig = Rig(tl, [20, 20, 20, 20, 20, 20], kv=2, group=1, hd=64, page=16, dtype=FP16)
    rig.cache.refs[int(rig.table[3, 1])] = 2
    rig.cache.table[4, 1] = -1
    x = torch.randn((6, 2, 64), generator=rig.g, device="cuda").to(FP16)
    want = rig.cache.k.clone()
    want[0, rig.table[0, 1], :, 1] = x[0]
    want[0, rig.table[5, 0], :, 4] = x[5]
    tl.paged_append(rig.cache, 0, x, x, _i32([17, -1, 32, 17, 17, 4]), seqs=_i32([0, 1, 2, 3, 4, 5]))
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
    assert torch.equal(rig.cache.k.view(torch.int16), want.view(torch.int16))
    tl.paged_append(rig.cache, 0, x[:2], x[:2], _i32([0, 0]), seqs=_i32([6, -1]))
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
    assert torch.equal(rig.cache.k.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("cu,written", [
    ([0, 3, 8, 8], (0,)),             # lane 1 claims rows that there are not
    ([0, 3, 6, 9], (0, 1)),           # lane 2 has none of its rows
    ([-2, 2, 4, 6], (1, 2)),          # lane 0 begins before the first row
    ([0, 4, 2, 6], ()),               # lane 1 ends before it begins: rows 2 and 3 have two owners
])
def test_append_reports_lanes_whose_rows_are_out_of_range(tl, cu, written):
    """Such a lane's rows are not written, the other lanes' are, and the call reports it."""
    rig = Rig(tl, [20, 20, 20], kv=2, group=1, hd=64, page=16, dtype=FP16)
    x = torch.randn((6, 2, 64), generator=rig.g, device="cuda").to(FP16)
    before = rig.cache.k.clone()
    tl.paged_append(rig.cache, 0, x, x, _i32([2, 2, 2]), cu_rows=_i32(cu))
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    for b in range(3):
        for i in range(max(0, min(6, cu[b + 1]) - cu[b])):
            at = (0, int(rig.table[b, 0]), slice(None), 2 + i)
            if b in written:
                assert same(rig.cache.k[at], x[cu[b] + i])
            elif written:
                assert same(rig.cache.k[at], before[at])
    assert same(rig.cache.k[1], before[1])


# ---------------------------------------------------------------------------------------- decode
@pytest.mark.parametrize("kv,group,hd,page,dtype,lens,split", [
    (4, 1, 128, 16, FP16, [0, 1, 15, 16, 17, 63, 64, 65], 0),
    (2, 4, 64, 32, BF16, [127, 128, 129, 1000, 2], 0),
    (1, 8, 128, 64, BF16, [5000], 0),
    (2, 5, 128, 128, FP16, [300, 1, 2049], 128),
    (1, 20, 64, 16, FP16, [513, 40], 256),       # two tiles of query heads, the second one partly filled
    (3, 16, 128, 16, BF16, [4097, 31], 0),
    (16, 1, 64, 16, FP16, [2049], 0),
])
def test_decode_matches_oracle(tl, kv, group, hd, page, dtype, lens, split):
    rig = Rig(tl, lens, kv=kv, group=group, hd=hd, page=page, dtype=dtype, split=split)
    q = rig.queries(len(lens))
    out = torch.full_like(q, float("nan"))
    tl.paged_attn_decode(rig.cache, 1, q, _i32(lens), out)
    rig.ok()
    rig.check_decode(1, q, out)


def test_decode_sharp_scores_scale_and_strided_queries(tl):
    """Large scores (one weight near 1), a scale of the caller's, queries inside wider rows, chosen sequences."""
    lens = [700, 64, 33]
    rig = Rig(tl, lens, kv=2, group=4, hd=128, page=32, dtype=BF16, seqs=[4, 0, 2])
    wide = rig.queries(6, sharp=6.0).view(3, 2, 8, 128)
    q, out = wide[:, 1], torch.full((3, 8, 128), float("nan"), dtype=BF16, device="cuda")
    tl.paged_attn_decode(rig.cache, 0, q, _i32(lens), out, seqs=_i32(rig.seqs), scale=0.31)
    rig.ok()
    rig.check_decode(0, q, out, scale=float(np.float32(0.31)))


def test_decode_lanes_do_not_depend_on_each_other(tl):
    """With a split length given, a lane's bits are those of its solo run, whatever lies beside it."""
    lens = [900, 3, 4000, 257]
    rig = Rig(tl, lens, kv=2, group=2, hd=128, page=16, dtype=FP16, split=256)
    q = rig.queries(4)
    out, solo = torch.empty_like(q), torch.empty_like(q)
    tl.paged_attn_decode(rig.cache, 0, q, _i32(lens), out)
    for b in range(4):
        tl.paged_attn_decode(rig.cache, 0, q[b:b + 1], _i32(lens[b:b + 1]), solo[b:b + 1], seqs=_i32([b]))
    rig.ok()
    assert torch.equal(out, solo)


@pytest.mark.parametrize("hd,dtype", [(64, FP16), (128, BF16)])
def test_decode_joins_many_splits(tl, hd, dtype):
    """Lanes of 64, 65, 301, 1, no and 2 splits in one call; a lane's bits are those it has in a shorter table."""
    lens = [64 * 128, 64 * 128 + 1, 300 * 128 + 5, 1, 0, 129]
    rig = Rig(tl, lens, kv=1, group=2, hd=hd, page=64, dtype=dtype, layers=1, split=128)
    q = rig.queries(6)
    out = torch.full_like(q, float("nan"))
    tl.paged_attn_decode(rig.cache, 0, q, _i32(lens), out)
    rig.ok()
    rig.check_decode(0, q, out)
    c = rig.cache
    d = tl.PagedDesc(1, c.desc.n_pages, 64, 1, hd, c.desc.max_seqs, 128, c.desc.dtype)
    short = tl.PagedCache(d, 2, 1, split_rows=128, k=c.k, v=c.v, table=c.table[:, :128].contiguous(), refs=c.refs)
    solo = torch.empty_like(q[:1])
    tl.paged_attn_decode(short, 0, q[:1], _i32(lens[:1]), solo)
    assert tl.poll_status(short) == tl.TL_OK
    assert torch.equal(out[:1], solo)


def test_decode_skips_and_reports(tl):
    """Lanes out of range are not written; positions without a page are left out."""
    lens = [40, 40, 40, 40]
    rig = Rig(tl, lens, kv=1, group=2, hd=64, page=16, dtype=FP16, spare=1)
    rig.cache.table[3, 1] = rig.cache.desc.n_pages
    q = rig.queries(4)
    out = torch.full_like(q, float("nan"))
    tl.paged_attn_decode(rig.cache, 0, q, _i32([40, -1, 65, 40]), out)
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
    assert torch.isnan(out[1:3]).all()
    k, v = rig.pools(0)
    for b, keep in ((0, np.arange(40)), (3, np.r_[0:16, 32:40])):
        for h in range(2):
            kk, vv = (np.concatenate([p[pg, 0] for pg in np.maximum(rig.table[b, :3], 0)])[keep] for p in (k, v))
            res = paged_oracle.attend(_np(q[b, h])[None], kk, vv, 0.125)
            _check(_np(out[b, h])[None], res, FP16, 64, 0.125, 40, rig.vmax(0))
    tl.paged_attn_decode(rig.cache, 0, q[:2], _i32([40, 40]), out[:2], seqs=_i32([4, -1]))
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE


def test_decode_offsets_past_32_bits(tl):
    """Pages whose elements lie past 2^32 bytes and 2^31 elements into the pool."""
    page, kv, hd, n_pages = 128, 16, 128, 9000           # 2.36e9 elements a layer
    desc = tl.PagedDesc(1, n_pages, page, kv, hd, 2, 4, tl.TL_KV_FP16)
    k = torch.zeros((1, n_pages, kv, page, hd), dtype=FP16, device="cuda")
    v = torch.zeros_like(k)
    cache = tl.PagedCache(desc, kv, 2, k=k, v=v)
    far = [n_pages - 1, 8300]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((200, kv, hd), generator=g, device="cuda").to(FP16)
    cache.table[1, :2] = _i32(far)
    tl.paged_append(cache, 0, rows, rows, _i32([0]), cu_rows=_i32([0, 200]), seqs=_i32([1]))
    q = torch.randn((200, kv, hd), generator=g, device="cuda").to(FP16)
    out, tok = torch.empty_like(q), torch.empty_like(q[:1])
    tl.paged_prompt_attn(cache, 0, q, _i32([0, 200]), _i32([200]), out, seqs=_i32([1]))
    tl.paged_attn_decode(cache, 0, q[199:], _i32([200]), tok, seqs=_i32([1]))
    cache.refs[far[1]] = 1
    tl.paged_copy(cache, _i32([far[1]]), _i32([far[0]]))
    assert tl.poll_status(cache) == tl.TL_OK
    assert torch.equal(k[0, far[0], :, :72], rows[128:].transpose(0, 1)) and torch.equal(k[0, far[0]], k[0, far[1]])
    x = _np(rows)
    for h in (0, kv - 1):
        res = paged_oracle.attend(_np(q[:, h]), x[:, h], x[:, h], hd ** -0.5, np.arange(200))
        _check(_np(out[:, h]), res, FP16, hd, hd ** -0.5, 200, np.abs(x).max())
        _check(_np(tok[:, h]), [r[199:] for r in res], FP16, hd, hd ** -0.5, 200, np.abs(x).max())


# ---------------------------------------------------------------------------------------- prompts
@pytest.mark.parametrize("kv,group,hd,page,dtype,lens,cached", [
    (2, 1, 64, 16, FP16, [1], [0]),
    (1, 4, 128, 16, FP16, [130, 1, 0, 257, 64], [0, 0, 5, 0, 0]),
    (2, 2, 128, 128, BF16, [300, 128], [0, 0]),
    (2, 3, 64, 32, BF16, [200, 33], [0, 100]),
    (1, 12, 128, 64, FP16, [70, 5], [600, 127]),          # four heads of each twelve packed
    (1, 1, 128, 16, BF16, [513], [0]),
    (2, 8, 64, 16, FP16, [40, 41, 39], [1000, 0, 88]),
    (1, 128, 64, 16, BF16, [3, 2], [0, 50]),              # one token a tile
    (1, 4, 128, 64, FP16, [70, 5, 0, 200], [3000, 100, 9, 5000]),   # blocks cut into pieces, up to eight
    (2, 1, 64, 128, BF16, [700], [900]),
])
def test_prompt_matches_oracle(tl, kv, group, hd, page, dtype, lens, cached):
    total = [a + b for a, b in zip(lens, cached)]
    rig = Rig(tl, total, kv=kv, group=group, hd=hd, page=page, dtype=dtype)
    cu = np.cumsum([1] + lens).tolist()                    # a row before and two behind that belong to nobody
    q = rig.queries(cu[-1] + 2)
    out = torch.full_like(q, float("nan"))
    tl.paged_prompt_attn(rig.cache, 1, q, _i32(cu), _i32(total), out)
    rig.ok()
    rig.check_prompt(1, q, cu, out)


@pytest.mark.parametrize("hd", [64, 128])
def test_prompt_growing_maxima_and_strided_queries(tl, hd):
    """Keys that grow along the sequence, so that every tile raises the maxima by far more than the rescale's
    threshold; scores up to about 60; a scale of the caller's; queries inside wider rows."""
    n = 600
    rig = Rig(tl, [n], kv=1, group=2, hd=hd, page=64, dtype=BF16, layers=1)
    ramp = torch.linspace(0.1, 6.0, 640, device="cuda").view(10, 64)
    for j in range(10):
        rig.cache.k[0, int(rig.table[0, j])] *= ramp[j].view(1, 64, 1).to(BF16)
    wide = rig.queries(3 * n).view(n, 3, 2, hd)
    q = wide[:, 2]
    out = torch.full((n, 2, hd), float("nan"), dtype=BF16, device="cuda")
    tl.paged_prompt_attn(rig.cache, 0, q, _i32([0, n]), _i32([n]), out, scale=0.25)
    rig.ok()
    rig.check_prompt(0, q, [0, n], out, scale=0.25)


def test_prompt_rows_that_attend_nothing(tl):
    """Queries at negative positions give zeros, a lane without cached positions too."""
    rig = Rig(tl, [20, 0], kv=1, group=2, hd=64, page=16, dtype=FP16)
    cu = [0, 150, 153]
    q = rig.queries(153)
    out = torch.full_like(q, float("nan"))
    tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32([20, 0]), out)
    rig.ok()
    assert not out[:130].any() and not out[150:].any()
    rig.check_prompt(0, q, cu, out)


@pytest.mark.parametrize("hd,page,dtype,before", [(128, 16, BF16, 0), (64, 128, FP16, 0), (128, 32, FP16, 2500)])
def test_prompt_is_causal_whatever_later_positions_hold(tl, hd, page, dtype, before):
    """NaN and infinities in K and V of later positions reach only the queries that attend them; with positions
    cached before, in blocks that are cut into pieces too."""
    n, at = 390, 301
    rig = Rig(tl, [n + before], kv=1, group=2, hd=hd, page=page, dtype=dtype, layers=1)
    q = rig.queries(n)
    out, clean = torch.empty_like(q), torch.empty_like(q)
    tl.paged_prompt_attn(rig.cache, 0, q, _i32([0, n]), _i32([n + before]), clean)
    slot = lambda i: (0, int(rig.table[0, (before + i) // page]), 0, (before + i) % page)  # noqa: E731
    rig.cache.v[slot(at)][3] = float("inf")
    rig.cache.v[slot(at + 20)][5] = float("nan")
    tl.paged_prompt_attn(rig.cache, 0, q, _i32([0, n]), _i32([n + before]), out)
    rig.ok()
    assert torch.equal(out[:at], clean[:at])
    assert torch.isinf(out[at:, :, 3]).all() and (out[at:, :, 3] > 0).all()
    assert torch.isnan(out[at + 20:, :, 5]).all() and torch.equal(out[:at + 20, :, 5], clean[:at + 20, :, 5])
    rest = [d for d in range(hd) if d not in (3, 5)]
    assert torch.equal(out[..., rest], clean[..., rest])
    rig.cache.k[slot(at)] = float("nan")
    tl.paged_prompt_attn(rig.cache, 0, q, _i32([0, n]), _i32([n + before]), out)
    assert torch.equal(out[:at], clean[:at]) and torch.isnan(out[at:]).all()


def test_prompt_chunks_repeat_bit_for_bit(tl):
    """Chunks over long caches, many CTAs with several tiles whose V is cleaned: the same bits every time."""
    new = [512, 401, 300, 450]
    total = [n + 4000 - 37 * b for b, n in enumerate(new)]
    rig = Rig(tl, total, kv=4, group=4, hd=128, page=16, dtype=BF16, layers=1)
    cu = np.cumsum([0] + new).tolist()
    q = rig.queries(cu[-1])
    first, out = torch.empty_like(q), torch.empty_like(q)
    tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32(total), first)
    for _ in range(40):
        out.fill_(float("nan"))
        tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32(total), out)
        assert torch.equal(out, first)
    rig.ok()


def _check_repeats(rig, q, cu, kv, times=30):
    """One call against the oracle, then the same bits from `times` more."""
    first, out = torch.full_like(q, float("nan")), torch.empty_like(q)
    args = _i32(cu), _i32(kv)
    rig.tl.paged_prompt_attn(rig.cache, 0, q, *args, first, seqs=_i32(rig.seqs))
    rig.ok()
    rig.check_prompt(0, q, cu, first, kv=kv)
    for _ in range(times):
        out.fill_(float("nan"))
        rig.tl.paged_prompt_attn(rig.cache, 0, q, *args, out, seqs=_i32(rig.seqs))
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    rig.ok()


@pytest.mark.parametrize("hd,group,dtype", [(64, 4, FP16), (128, 4, BF16), (128, 1, FP16)])
def test_prompt_full_blocks_before_a_few_rows_that_attend_nothing(tl, hd, group, dtype):
    """Blocks whose rows are all stored at once, each followed by a lane of a few queries without positions: more blocks
    than SMs, so that a CTA writes the one's outputs while the other's are still on their way."""
    block = 256 // group
    rig = Rig(tl, [block, 0], kv=1, group=group, hd=hd, page=16, dtype=dtype, layers=1)
    new = [block, 3] * 200
    rig.seqs = [0, 1] * 200
    cu = np.cumsum([0] + new).tolist()
    _check_repeats(rig, rig.queries(cu[-1]), cu, [block, 0] * 200)


@pytest.mark.parametrize("hd,group,n", [(64, 2, 128), (128, 2, 128), (128, 1, 256), (64, 4, 97), (128, 2, 192)])
def test_prompt_tiles_of_a_block_that_need_different_steps(tl, hd, group, n):
    """The first tile's scores end before the second's and the next block's queries follow at once: many short blocks
    a CTA, of different queries."""
    rig = Rig(tl, [n], kv=1, group=group, hd=hd, page=32, dtype=FP16, layers=1)
    lanes = 600 // -(-n * group // 256)
    rig.seqs = [0] * lanes
    _check_repeats(rig, rig.queries(n * lanes), list(range(0, n * lanes + 1, n)), [n] * lanes)


@pytest.mark.parametrize("empty", [1, 2, 3])
def test_prompt_lanes_without_positions_before_others(tl, empty):
    """Blocks that attend nothing, one to three in a row, then one with scores: the scores are of its own queries."""
    rig = Rig(tl, [0, 70], kv=1, group=2, hd=128, page=64, dtype=BF16, layers=1)
    new = ([5] * empty + [70]) * 250
    rig.seqs = ([0] * empty + [1]) * 250
    cu = np.cumsum([0] + new).tolist()
    _check_repeats(rig, rig.queries(cu[-1]), cu, ([0] * empty + [70]) * 250)


def _sink(tl, n, dtype, split=0):
    """One position of all the weight, n - 1 others 17.6 (natural units) below it, whose V alone is not zero."""
    rig = Rig(tl, [n], kv=1, group=1, hd=64, page=128, dtype=dtype, layers=1, split=split, n_lanes=148)
    rig.cache.k.zero_()
    rig.cache.v.abs_().clamp_(max=1)      # of one sign: what is lost does not cancel
    rig.cache.k[0, int(rig.table[0, 0]), 0, 0] = 2.2
    rig.cache.v[0, int(rig.table[0, 0]), 0, 0] = 0
    return rig


def _check_sink(rig, got, q, n, least):
    """The module's bound, with `least` in place of 2^-25: half the spacing of the smallest weights, relative to the
    largest one."""
    k, v = (paged_oracle.rows_of(p, rig.table[0], 0, n) for p in rig.pools(0))
    want, mag, reach = paged_oracle.attend(_np(q), k, v, 0.125)
    u = 2.0 ** -11 if rig.dtype == FP16 else 2.0 ** -8
    e = 2.0 ** -21 + n * 2.0 ** -24 + 2 * 2.0 ** -23 * 64 * 0.125 * reach[:, None]
    tol = u * np.abs(want) + mag * (u + e) * 1.01 + 2.0 ** -25 + n * least * np.nanmax(np.abs(v))
    worst = (np.abs(_np(got) - want) / tol).max()
    assert worst <= 1.0, f"{worst:.3g} of the tolerance"


@pytest.mark.parametrize("lanes,dtype", [(1, FP16), (148, FP16), (148, BF16)])   # cut into pieces, and not
def test_prompt_small_weights_behind_a_large_one(tl, lanes, dtype):
    """The first step sets the base of the exponents, from which the weights of 60000 positions are small.  They are
    held 2^7 times as large in FP16, spaced 2^-24 at the least: half of that is 2^-32 of the largest weight."""
    n = 60000
    rig = _sink(tl, n, dtype)
    q = torch.ones((lanes, 1, 64), dtype=dtype, device="cuda")
    out = torch.full_like(q, float("nan"))
    lane = torch.zeros(lanes, dtype=torch.int32, device="cuda")
    tl.paged_prompt_attn(rig.cache, 0, q, torch.arange(lanes + 1, dtype=torch.int32, device="cuda"), lane + n, out, seqs=lane)
    rig.ok()
    assert torch.equal(out, out[:1].expand_as(out))
    _check_sink(rig, out[:1, 0], q[:1, 0], n, 2.0 ** -32)


@pytest.mark.parametrize("split,dtype", [(0, FP16), (4096, FP16), (4096, BF16)])
def test_decode_small_weights_beside_a_large_one(tl, split, dtype):
    """The same for the decode, whose FP16 weights are held 2^15 times as large: half a spacing is 2^-40."""
    n = 60000
    rig = _sink(tl, n, dtype, split)
    q = torch.ones((1, 1, 64), dtype=dtype, device="cuda")
    out = torch.full_like(q, float("nan"))
    tl.paged_attn_decode(rig.cache, 0, q, _i32([n]), out)
    rig.ok()
    _check_sink(rig, out[:, 0], q[:, 0], n, 2.0 ** -40)


def test_prompt_call_of_seconds_with_nothing_to_clean(tl):
    """A thousand single queries over 2^22 positions each (eight pages, entered over and over): the warps that clean V
    wait for the whole call, which is no reason to give up.  Every position counts as often as the others, so the
    result is that of the eight pages once."""
    kv, hd, page, lanes, n = 16, 64, 128, 1024, 1 << 22
    cache = tl.PagedCache(tl.PagedDesc(1, 8, page, kv, hd, 1, n // page, tl.TL_KV_FP16), kv, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    for pool in (cache.k, cache.v):
        pool.copy_(torch.randn(pool.shape, generator=g, device="cuda"))
    cache.table[0] = torch.arange(n // page, device="cuda") % 8
    q = torch.randn((1, kv, hd), generator=g, device="cuda").to(FP16).expand(lanes, kv, hd).contiguous()
    out = torch.full_like(q, float("nan"))
    lane = torch.zeros(lanes, dtype=torch.int32, device="cuda")
    cu = torch.arange(lanes + 1, dtype=torch.int32, device="cuda")
    tl.paged_prompt_attn(cache, 0, q, cu, lane + n, out, seqs=lane)
    assert tl.poll_status(cache) == tl.TL_OK
    res = paged_oracle.decode(_np(cache.k[0]), _np(cache.v[0]), np.arange(8)[None], _np(q[:1]), [8 * page], [0], hd ** -0.5)
    _check(out[:1], res, FP16, hd, hd ** -0.5, n, float(cache.v.abs().max()))
    assert torch.equal(out[:-lanes // 8], out[:1].expand(lanes - lanes // 8, kv, hd))   # the last blocks are cut into pieces


def test_prompt_skips_and_reports(tl):
    rig = Rig(tl, [40, 40, 40, 40], kv=1, group=1, hd=64, page=16, dtype=FP16)
    rig.cache.table[1, 2] = -1
    q = rig.queries(160)
    cu = [0, 40, 80, 120, 160]
    for lens, seqs, lanes in (([40, 40, 49, 40], [0, 1, 2, 3], (1, 2)), ([40, 40, -1, 40], [0, 4, 2, -1], (1, 2, 3))):
        out = torch.full_like(q, float("nan"))
        tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32(lens), out, seqs=_i32(seqs))
        assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
        for b in range(4):
            assert torch.isnan(out[cu[b]:cu[b + 1]]).all() == (b in lanes)
    for bad in ([0, 40, 30, 120, 161], [-1, 40, 80, 120, 160]):
        out = torch.full_like(q, float("nan"))
        tl.paged_prompt_attn(rig.cache, 0, q, _i32(bad), _i32([30, 30, 30, 30]), out, seqs=_i32([0, 0, 2, 3]))
        assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE


@pytest.mark.parametrize("cu", [[0, 40, 30, 120, 161], [-1, 40, 80, 120, 160], [0, 40, 80, 70, 160], [5, 45, 200, 60, 90]])
@pytest.mark.parametrize("group,hd", [(1, 64), (8, 128)])
def test_prompt_lanes_whose_rows_are_out_of_range(tl, cu, group, hd):
    """A lane that begins before row 0, ends before it begins or ends past the rows is skipped: the rows of no other
    lane stay as they were, and those of one other lane alone are its results."""
    rows, lens = 160, [30, 40, 60, 100]
    rig = Rig(tl, lens, kv=1, group=group, hd=hd, page=16, dtype=FP16)
    q = rig.queries(rows)
    out = torch.full_like(q, float("nan"))
    tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32(lens), out)
    assert tl.poll_status(rig.cache) == tl.TL_ERR_DEVICE_RANGE
    valid = [b for b in range(4) if 0 <= cu[b] <= cu[b + 1] <= rows]
    owners = np.zeros(rows, int)
    for b in valid:
        owners[cu[b]:cu[b + 1]] += 1
    assert 0 < len(valid) < 4
    assert torch.isnan(out[torch.from_numpy(owners == 0)]).all()
    for b in valid:
        mine = np.arange(cu[b], cu[b + 1])
        alone = owners[mine] == 1
        k, v = (paged_oracle.rows_of(p, rig.table[b], 0, lens[b]) for p in rig.pools(0))
        last = lens[b] - len(mine) + np.arange(len(mine))
        for h in range(group):
            res = paged_oracle.attend(_np(q)[mine, h], k, v, hd ** -0.5, last)
            _check(_np(out)[mine, h][alone], [r[alone] for r in res], FP16, hd, hd ** -0.5, lens[b], rig.vmax(0))


def test_prompt_row_equals_decode_of_the_same_position(tl):
    """The last row of a prompt and the decode of its token agree within the roundings of both."""
    lens = [500, 77]
    rig = Rig(tl, lens, kv=2, group=4, hd=128, page=32, dtype=FP16)
    q = rig.queries(577)
    out, tok = torch.empty_like(q), torch.empty_like(q[:2])
    tl.paged_prompt_attn(rig.cache, 0, q, _i32([0, 500, 577]), _i32(lens), out)
    tl.paged_attn_decode(rig.cache, 0, q[[499, 576]], _i32(lens), tok)
    rig.check_decode(0, q[[499, 576]], tok)
    rig.check_decode(0, q[[499, 576]], out[[499, 576]])


def test_a_thousand_lanes(tl):
    """As many lanes as a call may have, some empty, in a table that would hold 2^22 positions each."""
    rng = np.random.default_rng(5)
    new = rng.integers(0, 4, 1024)
    total = (new + rng.integers(0, 60, 1024)).tolist()
    rig = Rig(tl, total, kv=1, group=2, hd=64, page=16, dtype=FP16, layers=1, n_lanes=1024, seqs=rng.permutation(1024).tolist())
    wide = tl.PagedDesc(1, rig.cache.desc.n_pages, 16, 1, 64, 1025, 262144, tl.TL_KV_FP16)
    table = torch.full((1025, 262144), -1, dtype=torch.int32, device="cuda")
    table[:, :rig.table.shape[1]] = torch.from_numpy(rig.table[:1025]).cuda()
    rig.cache = tl.PagedCache(wide, 2, 1024, k=rig.cache.k, v=rig.cache.v, table=table, refs=rig.cache.refs)
    cu = np.cumsum([0] + new.tolist()).tolist()
    q, tok = rig.queries(cu[-1]), rig.queries(1024)
    out, o1 = torch.full_like(q, float("nan")), torch.full_like(tok, float("nan"))
    tl.paged_prompt_attn(rig.cache, 0, q, _i32(cu), _i32(total), out, seqs=_i32(rig.seqs))
    tl.paged_attn_decode(rig.cache, 0, tok, _i32(total), o1, seqs=_i32(rig.seqs))
    rig.ok()
    rig.check_prompt(0, q, cu, out)
    rig.check_decode(0, tok, o1)


def test_two_streams_with_a_workspace_each(tl):
    """Calls that overlap on the GPU, each on a workspace of its own over the same pool: the bits of calls alone."""
    lens = [3000, 500, 1200]
    rig = Rig(tl, lens, kv=2, group=4, hd=128, page=16, dtype=BF16, layers=1)
    c = rig.cache
    other = tl.PagedCache(c.desc, rig.heads, 3, k=c.k, v=c.v, table=c.table, refs=c.refs)
    cu, n, kv = _i32([0, 200, 300, 700]), 700, _i32(lens)
    q = rig.queries(n)
    want, w1 = torch.empty_like(q), torch.empty_like(q[:3])
    tl.paged_prompt_attn(c, 0, q, cu, kv, want)
    tl.paged_attn_decode(c, 0, q[:3], kv, w1)
    outs = [(torch.empty_like(q), torch.empty_like(q[:3])) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for cache, (a, b), st in zip((c, other), outs, streams):
            tl.paged_prompt_attn(cache, 0, q, cu, kv, a, stream=st)
            tl.paged_attn_decode(cache, 0, q[:3], kv, b, stream=st)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, w1)
    assert tl.poll_status(c) == tl.TL_OK and tl.poll_status(other) == tl.TL_OK


# ---------------------------------------------------------------------------------------- pages
class Twin:
    """A cache beside the oracle's list walks: each operation on both, then everything compared."""

    def __init__(self, tl, n_pages, page, max_seqs, max_pages, layers=3, kv=2, hd=64):
        self.tl = tl
        self.o = paged_oracle.Pages(n_pages, page, max_seqs, max_pages)
        self.cache = tl.PagedCache(tl.PagedDesc(layers, n_pages, page, kv, hd, max_seqs, max_pages), kv, min(max_seqs, 1024))
        n = self.cache.k.numel()
        self.cache.k.view(torch.int16).copy_(torch.arange(n, device="cuda").view(self.cache.k.shape))
        self.cache.v.view(torch.int16).copy_((torch.arange(n, device="cuda") * 7 + 1).view(self.cache.k.shape))
        self.k, self.v = self.cache.k.clone(), self.cache.v.clone()

    def do(self, op, *lists):
        self.o.flags = set()
        moves = getattr(self.o, op)(*lists)
        getattr(self.tl, "paged_" + op)(self.cache, *[None if x is None else _i32(x) for x in lists])
        for pool in (self.k, self.v):
            was = pool.clone()
            for a, b in moves:
                pool[:, b] = was[:, a]
        want = self.tl.TL_ERR_DEVICE_RANGE if "range" in self.o.flags else \
            self.tl.TL_ERR_DEVICE_CAPACITY if "full" in self.o.flags else self.tl.TL_OK
        assert self.tl.poll_status(self.cache) == want, op
        assert np.array_equal(self.cache.table.cpu().numpy(), self.o.table), op
        assert np.array_equal(self.cache.refs.cpu().numpy(), self.o.refs), op
        assert torch.equal(self.cache.k.view(torch.int16), self.k.view(torch.int16)), op
        assert torch.equal(self.cache.v.view(torch.int16), self.v.view(torch.int16)), op


def test_pages_of_a_serving_loop(tl):
    t = Twin(tl, n_pages=70, page=16, max_seqs=12, max_pages=9)
    t.do("reserve", [3, 0, 7], [0, 0, 0], [100, 16, 33])
    t.do("fork", [3, 3, 0], [4, 5, 9], [100, 64, 16])
    t.do("reserve", [4, 3, 5, 9], [100, 100, 64, 16], [1, 1, 1, 20])   # all sharers of a last page copy it
    t.do("free", [3], [30])
    t.do("free", [7, 4, 7], None)                                      # one listed twice
    t.do("reserve", [7, 11], [0, 0], [1, 144])
    t.do("compact")
    t.do("copy", [0, 5, 1], [60, 61, 62])
    t.do("free", [3, 5, 9], [17, 0, 16])
    t.do("compact")
    t.do("compact")
    t.do("free", list(range(12)), None)
    t.do("compact")
    assert not t.o.refs.any()


def test_pages_refusals(tl):
    t = Twin(tl, n_pages=24, page=32, max_seqs=6, max_pages=4)
    t.do("reserve", [0, 1, 0, 6, -1, 2, 3], [0, 0, 0, 0, 0, -1, 100], [64, 1, 5, 1, 1, 1, 40])  # listed twice, out of range, too long
    t.do("reserve", [3], [7], [2 ** 31 - 8])
    t.do("fork", [0, 0, 1, 2, 9, 0, 4], [2, 2, 0, 3, 4, 5, 5], [64, 1, 1, 1, 1, 65, 0])         # dst twice, src a dst, lacking pages
    t.do("free", [6, 2, -3, 0], [0, -1, 0, 31])
    t.do("copy", [0, 1, 2, 24, 3, -1, 8], [10, 11, 10, 12, 0, 13, 8])
    t.do("reserve", [0, 3, 4, 5], [0, 0, 0, 0], [0, 128, 128, 128])
    t.do("reserve", [1, 2, 4], [0, 0, 0], [128, 128, 128])                                      # the last is not covered
    t.do("reserve", [4, 1], [0, 0], [128, 1])


def test_poll_tells_a_lack_of_pages_and_what_was_out_of_range(tl):
    """Both recorded, by one call or by a step of two: each is returned once, the lack of pages first."""
    c = tl.PagedCache(tl.PagedDesc(1, 3, 16, 1, 64, 4, 4), 1, 4)
    x = torch.zeros((2, 1, 64), dtype=FP16, device="cuda")
    polls = lambda: [tl.poll_status(c) for _ in range(3)]  # noqa: E731
    tl.paged_reserve(c, _i32([9, 0, 1]), _i32([0, 0, 0]), _i32([1, 32, 32]))
    assert polls() == [tl.TL_ERR_DEVICE_CAPACITY, tl.TL_ERR_DEVICE_RANGE, tl.TL_OK]
    tl.paged_reserve(c, _i32([1, 2]), _i32([0, 0]), _i32([16, 16]))      # sequence 2 gets no page for its token
    tl.paged_append(c, 0, x, x, _i32([0, 0]), seqs=_i32([1, 2]))
    assert polls() == [tl.TL_ERR_DEVICE_CAPACITY, tl.TL_ERR_DEVICE_RANGE, tl.TL_OK]
    tl.paged_reserve(c, _i32([2]), _i32([0]), _i32([16]))
    assert polls() == [tl.TL_ERR_DEVICE_CAPACITY, tl.TL_OK, tl.TL_OK]
    tl.paged_append(c, 0, x, x, _i32([0, 0]), seqs=_i32([1, 2]))
    assert polls() == [tl.TL_ERR_DEVICE_RANGE, tl.TL_OK, tl.TL_OK]


@pytest.mark.parametrize("n_pages,max_pages", [(20001, 400), (40000, 3000)])
def test_pages_at_size(tl, n_pages, max_pages):
    """Several scan rounds over the pool and over the candidates of one call, odd sizes, random lists."""
    rng = np.random.default_rng(n_pages)
    t = Twin(tl, n_pages=n_pages, page=16, max_seqs=200, max_pages=max_pages, layers=1, kv=1)
    hi = max_pages * 16
    lens = [0] * 200
    for i in range(90):
        lens[i] = int(min(rng.integers(1, hi), n_pages * 16 // 120))
    lens[50] = hi                                   # one long prompt beside the others
    t.do("reserve", list(range(90)), [0] * 90, lens[:90])
    t.do("free", [int(i) for i in rng.permutation(90)[:45]], None)
    src = [i for i in range(90) if (t.o.table[i] >= 0).any()][:40]
    t.do("fork", src, list(range(100, 100 + len(src))), [min(lens[i], int(rng.integers(0, hi))) for i in src])
    t.do("compact")
    t.do("reserve", list(range(100, 100 + len(src))), [int(rng.integers(0, lens[i])) for i in src], [3] * len(src))
    t.do("compact")


def test_pages_with_counts_that_are_not_the_tables(tl):
    """A table entered by hand without counts, then freed (counts below 0) and compacted: no page is lost or copied
    to where there is none, and what is not counted is free."""
    t = Twin(tl, n_pages=40, page=16, max_seqs=4, max_pages=6)
    t.do("reserve", [0], [0], [40])
    t.cache.table[1, :3] = _i32([30, 20, 39])
    tl.paged_free(t.cache, _i32([1]))
    assert t.cache.refs[[20, 30, 39]].tolist() == [-1] * 3
    tl.paged_compact(t.cache)
    tl.paged_reserve(t.cache, _i32([2]), _i32([0]), _i32([96]))
    assert tl.poll_status(t.cache) == tl.TL_OK
    assert t.cache.table[0].tolist() == [0, 1, 2, -1, -1, -1] and t.cache.table[2].tolist() == [3, 4, 5, 6, 7, 8]


def test_reserve_a_thousand_sequences(tl):
    t = Twin(tl, n_pages=1500, page=16, max_seqs=1030, max_pages=2, layers=1, kv=1)
    order = np.random.default_rng(0).permutation(1030)[:1024].tolist()
    t.do("reserve", order, [0] * 1024, [1 + i % 16 for i in range(1024)])
    t.do("reserve", order, [16] * 1024, [1] * 1024)          # 476 of them are covered
    t.do("free", order, [16] * 1024)
    t.do("compact")


# ---------------------------------------------------------------------------------------- together
def _serve(tl, cache, layers, x, out):
    """Prompts into the cache, forks, three tokens each, a rejected token taken back, compaction, one more token."""
    kv, heads = cache.desc.n_kv_heads, cache.n_heads
    n_prompt = [50, 7, 130]
    cu = _i32([0, 50, 57, 187])
    seqs, zero = _i32([0, 1, 2]), _i32([0, 0, 0])
    tl.paged_reserve(cache, seqs, zero, _i32(n_prompt))
    for la in range(layers):
        q, k, v = x[la, :187, :heads], x[la, :187, heads:heads + kv], x[la, :187, heads + kv:]
        tl.paged_append(cache, la, k, v, zero, cu_rows=cu, seqs=seqs)
        tl.paged_prompt_attn(cache, la, q, cu, _i32(n_prompt), out[la, :187], seqs=seqs)
    tl.paged_fork(cache, _i32([0, 2]), _i32([3, 4]), _i32([50, 130]))
    lanes, at = _i32([0, 1, 2, 3, 4]), 187
    lens = [50, 7, 130, 50, 130]
    for step in range(4):
        if step == 3:                                  # the last token is taken back, then the pool compacted
            lens = [n - 1 for n in lens]
            tl.paged_free(cache, lanes, _i32(lens))
            tl.paged_compact(cache)
        tl.paged_reserve(cache, lanes, _i32(lens), _i32([1] * 5))
        for la in range(layers):
            row = x[la, at:at + 5]
            tl.paged_append(cache, la, row[:, heads:heads + kv], row[:, heads + kv:], _i32(lens), seqs=lanes)
            tl.paged_attn_decode(cache, la, row[:, :heads], _i32([n + 1 for n in lens]), out[la, at:at + 5], seqs=lanes)
        lens = [n + 1 for n in lens]
        at += 5
    return lens


@pytest.mark.parametrize("dtype,page", [(FP16, 16), (BF16, 64)])
def test_serving_run_matches_plain_attention(tl, dtype, page):
    """The operators as they are used together, against attention over plainly kept K and V."""
    layers, kv, heads, hd = 2, 2, 6, 64
    cache = tl.PagedCache(tl.PagedDesc(layers, 60, page, kv, hd, 6, 12, tl.TL_KV_FP16 if dtype == FP16 else tl.TL_KV_BF16), heads, 5)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((layers, 207, heads + 2 * kv, hd), generator=g, device="cuda").to(dtype)
    out = torch.empty((layers, 207, heads, hd), dtype=dtype, device="cuda")
    _serve(tl, cache, layers, x, out)
    assert tl.poll_status(cache) == tl.TL_OK
    # rows of each sequence at each step, as indices into x
    hist = [list(range(0, 50)), list(range(50, 57)), list(range(57, 187))]
    hist += [hist[0], hist[2]]
    want = [(b, i, hist[b][: i + 1], hist[b][i]) for b in range(3) for i in range(len(hist[b]))]
    at = 187
    for step in range(4):
        if step == 3:
            hist = [h[:-1] for h in hist]
        hist = [h + [at + b] for b, h in enumerate(hist)]
        want += [(b, len(h) - 1, h, h[-1]) for b, h in enumerate(hist)]
        at += 5
    xs, got = _np(x), _np(out)
    vmax = np.abs(xs).max()
    for la in range(layers):
        for b, i, rows, r in want[::7] + want[-20:]:
            for h in range(heads):
                kk, vv = xs[la, rows, heads + h // 3], xs[la, rows, heads + kv + h // 3]
                res = paged_oracle.attend(xs[la, r, h][None], kk, vv, hd ** -0.5)
                _check(got[la, r, h][None], res, dtype, hd, hd ** -0.5, len(rows), vmax)


def test_graph_replay_on_a_side_stream_equals_eager(tl):
    """The calls captured, replayed twice from the same start, on another stream: the bits of the eager run.  Two
    graphs share the workspace, replayed one after the other."""
    rig = Rig(tl, [0, 40, 700, 129], kv=2, group=4, hd=128, page=16, dtype=BF16, spare=2)
    lens, one = _i32([0, 40, 700, 129]), _i32([1] * 4)
    after = _i32([1, 41, 701, 130])
    seqs = _i32([0, 1, 2, 3])
    rows = torch.randn((4, 12, 128), generator=rig.g, device="cuda").to(BF16)
    start = [t.clone() for t in (rig.cache.k, rig.cache.v, rig.cache.table, rig.cache.refs)]
    cu = _i32([0, 1, 2, 3, 4])
    out, pr = torch.empty_like(rows[:, :8]), torch.empty_like(rows[:, :8])

    def step():
        tl.paged_reserve(rig.cache, seqs, lens, one)
        tl.paged_append(rig.cache, 1, rows[:, 8:10], rows[:, 10:], lens)
        tl.paged_attn_decode(rig.cache, 1, rows[:, :8], after, out)

    def step2():
        tl.paged_prompt_attn(rig.cache, 1, rows[:, :8], cu, after, pr)
        tl.paged_attn_decode(rig.cache, 0, rows[:, :8], lens, out2)
    out2 = torch.empty_like(out)

    def reset():
        for a, b in zip((rig.cache.k, rig.cache.v, rig.cache.table, rig.cache.refs), start):
            a.copy_(b)
        for o in (out, pr, out2):
            o.fill_(float("nan"))
    step()
    step2()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, pr, out2, rig.cache.table, rig.cache.refs, rig.cache.k.view(torch.int16))]
    side = torch.cuda.Stream()
    reset()
    torch.cuda.synchronize()
    graphs = []
    with torch.cuda.stream(side):
        for f in (step, step2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                f()
            graphs.append(g)
        for _ in range(2):
            reset()
            for g in graphs:
                g.replay()
    side.synchronize()
    rig.ok()
    for a, b in zip((out, pr, out2, rig.cache.table, rig.cache.refs, rig.cache.k.view(torch.int16)), want):
        assert torch.equal(a.view(torch.int16) if a.is_floating_point() else a, b.view(torch.int16) if b.is_floating_point() else b)
