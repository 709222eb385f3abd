"""The paged K/V cache on the host (no GPU): sizes, refusals before any launch, the binding's checks of its
arguments, and the CPU oracle's pins."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_oracle


@pytest.fixture(scope="module")
def tl():
    from store_kv_attention_b200 import build_lib
    build_lib.build()
    import store_kv_attention_b200 as m
    return m


def _desc(tl, **kw):
    base = dict(n_layers=3, n_pages=40, page_size=16, n_kv_heads=4, head_dim=128, max_seqs=8, max_pages=20, dtype=0)
    base.update(kw)
    return tl.PagedDesc(**base)


def test_cache_bytes_match_layout(tl):
    assert tl.paged_cache_bytes(_desc(tl)) == (3 * 40 * 4 * 16 * 128 * 2, 8 * 20 * 4, 40 * 4)
    assert tl.paged_cache_bytes(_desc(tl, head_dim=64, dtype=tl.TL_KV_BF16))[0] == 3 * 40 * 4 * 16 * 64 * 2


@pytest.mark.parametrize("kw,status", [
    (dict(page_size=24), 4), (dict(page_size=256), 4), (dict(head_dim=96), 4), (dict(n_kv_heads=257), 4),
    (dict(max_pages=(1 << 18) + 1), 4), (dict(n_pages=(1 << 22) + 1), 4), (dict(max_seqs=65537), 4),
    (dict(n_pages=1 << 22, n_kv_heads=64), 4), (dict(dtype=2), 1), (dict(n_layers=0), 1), (dict(n_pages=-1), 1),
])
def test_desc_validation(tl, kw, status):
    with pytest.raises(tl.TLError) as e:
        tl.paged_cache_bytes(_desc(tl, **kw))
    assert e.value.status == status


@pytest.mark.parametrize("max_pages", [1, 20, 4096, 262144])
@pytest.mark.parametrize("heads", [4, 12, 128])
def test_workspace_covers_every_smaller_call(tl, max_pages, heads):
    """The workspace of n lanes is enough for every call of fewer: the launch's own need, from its refusal."""
    d = _desc(tl, max_pages=max_pages, max_seqs=1024)
    for split in (0, 256):
        for n in (1, 7, 64, 1024):
            have = tl.paged_workspace_bytes(d, heads, n, split)
            for m in {m for m in (1, 2, 3, n // 2, n - 1, n) if 0 < m <= n}:
                assert _decode_need(tl, d, heads, m, split) <= have, (n, m, split)


def _decode_need(tl, d, heads, n, split):
    fake = 1 << 20
    st = tl.lib.tl_paged_attn_decode(ctypes.byref(d.c()), tl.PagedCacheC(fake, fake, fake, fake), 0, heads, fake, 0, fake,
                                     None, 0.0, split, fake, n, fake, 0, None)
    assert st == tl.TL_ERR_CAPACITY
    return int(tl.lib.tl_last_error_message().decode().split("<")[1].split()[0])


def test_calls_rejected_before_launch(tl):
    L, d = tl.lib, _desc(tl)
    fake, odd = 1 << 20, (1 << 20) + 8
    c = tl.PagedCacheC(fake, fake, fake, fake)
    ws = tl.paged_workspace_bytes(d, 8, 4)
    dc = ctypes.byref(d.c())

    def append(desc=dc, cache=c, layer=0, k=fake, ks=0, rows=4, cu=None, start=fake, seqs=None, n=4, w=fake, wb=ws):
        return L.tl_paged_append(desc, cache, layer, k, ks, fake, 0, rows, cu, start, seqs, n, w, wb, None)
    assert append(desc=None) == tl.TL_ERR_INVALID_ARG
    assert append(cache=tl.PagedCacheC(odd, fake, fake, fake)) == tl.TL_ERR_INVALID_ARG
    assert append(cache=tl.PagedCacheC(fake, fake, None, fake)) == tl.TL_ERR_INVALID_ARG
    assert append(layer=3) == tl.TL_ERR_CAPACITY and append(layer=-1) == tl.TL_ERR_CAPACITY
    assert append(k=odd) == tl.TL_ERR_INVALID_ARG and append(k=None) == tl.TL_ERR_INVALID_ARG
    assert append(ks=511) == tl.TL_ERR_INVALID_ARG and append(ks=516) == tl.TL_ERR_INVALID_ARG
    assert append(rows=5) == tl.TL_ERR_INVALID_ARG              # one row per lane without cu_rows
    assert append(rows=-1, cu=fake) == tl.TL_ERR_INVALID_ARG
    assert append(n=9, rows=9) == tl.TL_ERR_CAPACITY            # more lanes than sequences
    assert append(n=1025, rows=1025, seqs=fake) == tl.TL_ERR_UNSUPPORTED
    assert append(w=None) == tl.TL_ERR_INVALID_ARG and append(wb=128) == tl.TL_ERR_CAPACITY
    assert append(rows=0, cu=fake) == tl.TL_OK and append(rows=0, k=None, start=None) == tl.TL_OK
    assert append(rows=0, layer=3) == tl.TL_ERR_CAPACITY

    def decode(layer=0, heads=8, q=fake, qs=0, lens=fake, scale=0.0, split=0, out=fake, n=4, w=fake, wb=ws):
        return L.tl_paged_attn_decode(dc, c, layer, heads, q, qs, lens, None, scale, split, out, n, w, wb, None)
    assert decode(heads=6) == tl.TL_ERR_SHAPE and decode(heads=0) == tl.TL_ERR_INVALID_ARG
    assert decode(heads=1028) == tl.TL_ERR_UNSUPPORTED
    assert decode(qs=8 * 128 - 8) == tl.TL_ERR_INVALID_ARG and decode(qs=8 * 128 + 4) == tl.TL_ERR_INVALID_ARG
    for scale in (-1.0, float("nan"), float("inf")):
        assert decode(scale=scale) == tl.TL_ERR_INVALID_ARG
    for split in (-128, 100, 8192):
        assert decode(split=split) == tl.TL_ERR_INVALID_ARG
    assert decode(out=odd) == tl.TL_ERR_INVALID_ARG and decode(lens=None) == tl.TL_ERR_INVALID_ARG
    assert decode(n=0) == tl.TL_ERR_INVALID_ARG and decode(n=9) == tl.TL_ERR_CAPACITY
    assert decode(w=odd) == tl.TL_ERR_INVALID_ARG and decode(wb=0) == tl.TL_ERR_CAPACITY

    def prompt(heads=8, rows=10, cu=fake, lens=fake, scale=0.0, n=4, wb=ws):
        return L.tl_paged_prompt_attn(dc, c, 0, heads, fake, 0, rows, cu, lens, None, scale, fake, n, fake, wb, None)
    assert prompt(heads=6) == tl.TL_ERR_SHAPE and prompt(cu=None) == tl.TL_ERR_INVALID_ARG
    assert prompt(rows=-1) == tl.TL_ERR_INVALID_ARG and prompt(rows=(1 << 24) + 1) == tl.TL_ERR_UNSUPPORTED
    assert prompt(scale=-0.5) == tl.TL_ERR_INVALID_ARG and prompt(wb=0) == tl.TL_ERR_CAPACITY
    assert prompt(rows=0) == tl.TL_OK

    no_refs = tl.PagedCacheC(fake, fake, fake, None)
    for name, args in (("copy", (fake, fake)), ("fork", (fake, fake, fake)), ("reserve", (fake, fake, fake)),
                       ("free", (fake, None))):
        f = getattr(L, "tl_paged_" + name)
        assert f(dc, no_refs, *args, 1, fake, ws, None) == tl.TL_ERR_INVALID_ARG
        assert f(dc, c, *args, -1, fake, ws, None) == tl.TL_ERR_INVALID_ARG
        assert f(dc, c, *args, 1025, fake, ws, None) == tl.TL_ERR_UNSUPPORTED
        assert f(dc, c, *args, 1, fake, 256, None) == tl.TL_ERR_CAPACITY
        assert f(dc, c, None, *args[1:], 1, fake, ws, None) == tl.TL_ERR_INVALID_ARG
        assert f(dc, c, *args, 0, fake, ws, None) == tl.TL_OK
        assert f(dc, c, *[None] * len(args), 0, fake, ws, None) == tl.TL_OK   # an empty list has no address
    assert L.tl_paged_compact(dc, no_refs, None, fake, ws, None) == tl.TL_ERR_INVALID_ARG
    assert L.tl_paged_compact(dc, c, None, fake, 256, None) == tl.TL_ERR_CAPACITY


def test_binding_checks_tensors(tl):
    """Types, shapes, layouts and devices that the library cannot see are refused by the binding."""
    d = _desc(tl)
    c = tl.PagedCache(d, n_heads=8, n_lanes=4, device="cpu")
    q, lens = torch.zeros(4, 8, 128, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    out = torch.zeros_like(q)
    for bad in (q.bfloat16(), q[:, :, :64], q.transpose(0, 1), q[0], q[:1].expand(4, 8, 128)):
        with pytest.raises(ValueError):
            tl.paged_attn_decode(c, 0, bad, lens, out)
    for bad in (lens.long(), lens[:3], torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            tl.paged_attn_decode(c, 0, q, bad, out)
    with pytest.raises(ValueError):
        tl.paged_attn_decode(c, 0, q, lens, torch.zeros(4, 16, 128, dtype=torch.float16)[:, ::2])
    with pytest.raises(ValueError):
        tl.paged_prompt_attn(c, 0, q, lens, lens, out)          # cu_q has n_lanes + 1 entries
    with pytest.raises(ValueError):
        tl.paged_append(c, 0, q[:, :4], q[:3, :4], lens)
    with pytest.raises(ValueError):
        tl.paged_fork(c, lens, lens[:2], lens)
    with pytest.raises(ValueError):
        tl.PagedCache(d, n_heads=8, n_lanes=4, k=c.k[:, :10])
    with pytest.raises(ValueError):
        tl.paged_attn_decode(c, 0, q, lens, out)                # a cache on the host


def test_oracle_attend_against_torch():
    """The oracle's attention equals the library's, causal at the right end, in FP64."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 64, generator=g, dtype=torch.float64) for n in (5, 9, 9))
    mask = torch.arange(9)[None] <= torch.arange(5)[:, None] + 4
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask[None])[0]
    got, mag, _ = paged_oracle.attend(q.numpy(), k.numpy(), v.numpy(), 0.125, last=np.arange(5) + 4)
    assert np.abs(got - want.numpy()).max() < 1e-13 and (mag >= np.abs(got) - 1e-15).all()
    empty, _, _ = paged_oracle.attend(q.numpy(), k.numpy(), v.numpy(), 0.125, last=np.array([-3, -1, 0, 1, 2]))
    assert not empty[:2].any() and np.allclose(empty[2], v[0].numpy())


def test_oracle_pages_by_hand():
    p = paged_oracle.Pages(n_pages=6, page=16, max_seqs=4, max_pages=3)
    assert p.reserve([2, 0], [0, 0], [17, 5]) == [] and p.table.tolist()[0] == [2, -1, -1]
    assert p.table.tolist()[2] == [0, 1, -1] and p.refs.tolist() == [1, 1, 1, 0, 0, 0]
    p.fork([2], [1], [17])
    assert p.refs.tolist() == [2, 2, 1, 0, 0, 0]
    assert p.reserve([1], [17], [1]) == [(1, 3)] and p.table.tolist()[1] == [0, 3, -1]
    p.free([0, 2])
    assert p.refs.tolist() == [1, 0, 0, 1, 0, 0]
    assert p.compact() == [(3, 1)] and p.table.tolist()[1] == [0, 1, -1] and not p.flags
    p.reserve([0, 1, 2], [0, 32, 0], [40, 1, 32])
    assert p.flags == {"full"} and (p.table[2] < 0).all() and p.table[0].tolist() == [2, 3, 4]
