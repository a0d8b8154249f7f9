"""The paged-cache calls on the host, without a GPU: refusals come back as codes before any
device work, and the workspace size is a host computation."""
import ctypes

import pytest

rkv = pytest.importorskip("rolling_kv_chunked_b200")

A = 0x10000  # an aligned address that no refused call follows


def pool(**kw):
    p = dict(k=A, v=A, page_stride=2 * 16 * 128, n_pages=4, kv_heads=2, page_tokens=16)
    p.update(kw)
    return rkv._PagePool(*p.values())


def batch(**kw):
    b = dict(page_table=A, kv_len=A, q_start=A, status=None, table_stride=4, n_seqs=2, max_q=8, max_kv=64)
    b.update(kw)
    return rkv._PagedBatch(*b.values())


def write(p=None, b=None, k=A, v=A, rows=8, ks=256, vs=256):
    return rkv._lib.rkv_paged_write(p or pool(), b or batch(), k, v, rows, ks, vs, None)


def attend(p=None, b=None, q=A, heads=4, rows=8, qs=512, out=2 * A, os_=512, lse=None, weight=None, width=0, ws=A,
           size=1 << 40):
    return rkv._lib.rkv_paged_attention(p or pool(), b or batch(), q, heads, rows, qs, out, os_, 1, lse, weight, width,
                                        ws, size, None)


def evict(p=None, b=None, weight=A, width=64, keep=8, sinks=1, recent=2, kept=A, out=A):
    return rkv._lib.rkv_paged_evict(p or pool(), b or batch(), weight, width, keep, sinks, recent, kept, out, None)


POOLS = [(dict(k=None), rkv.ERR_ARG), (dict(v=A + 8), rkv.ERR_ARG), (dict(n_pages=0), rkv.ERR_ARG),
         (dict(kv_heads=0), rkv.ERR_ARG), (dict(page_tokens=0), rkv.ERR_ARG), (dict(page_tokens=8), rkv.ERR_UNSUPPORTED),
         (dict(page_tokens=48), rkv.ERR_UNSUPPORTED), (dict(page_tokens=256), rkv.ERR_UNSUPPORTED),
         (dict(page_stride=2 * 16 * 128 - 8), rkv.ERR_ARG), (dict(page_stride=2 * 16 * 128 + 4), rkv.ERR_ARG),
         (dict(page_stride=1 << 38), rkv.ERR_UNSUPPORTED)]
BATCHES = [(dict(page_table=None), rkv.ERR_ARG), (dict(kv_len=A + 2), rkv.ERR_ARG), (dict(status=A + 1), rkv.ERR_ARG),
           (dict(n_seqs=-1), rkv.ERR_ARG), (dict(max_q=-1), rkv.ERR_ARG), (dict(max_kv=-1), rkv.ERR_ARG),
           (dict(max_kv=65), rkv.ERR_ARG), (dict(table_stride=3), rkv.ERR_ARG),
           (dict(n_seqs=(1 << 16) + 1), rkv.ERR_UNSUPPORTED)]


@pytest.mark.parametrize("call", [write, attend, evict])
def test_pool_and_batch_refusals(call):
    for kw, code in POOLS:
        assert call(p=pool(**kw)) == code, kw
    for kw, code in BATCHES:
        assert call(b=batch(**kw)) == code, kw
    if call is not evict:
        assert call(b=batch(q_start=None)) == rkv.ERR_ARG
    assert call(b=batch(n_seqs=0, page_table=None, kv_len=None, q_start=None)) == rkv.OK  # nothing to do


def test_write_refusals():
    for kw in (dict(k=None), dict(v=None), dict(k=A + 2), dict(rows=-1), dict(ks=255), dict(ks=248), dict(vs=0),
               dict(vs=-256), dict(vs=260)):
        assert write(**kw) == rkv.ERR_ARG, kw
    assert write(rows=0, k=None, v=None) == rkv.OK
    assert write(rows=1 << 30) == rkv.ERR_UNSUPPORTED


def test_attention_refusals():
    for kw in (dict(q=None), dict(out=None), dict(q=A + 4), dict(out=2 * A + 4), dict(heads=0), dict(heads=3),
               dict(rows=-1), dict(qs=504), dict(qs=516), dict(os_=0), dict(out=A), dict(out=A + 7 * 1024),
               dict(q=A + 1024, out=A), dict(lse=A + 2), dict(weight=A, width=63), dict(weight=A + 2, width=64)):
        assert attend(**kw) == rkv.ERR_ARG, kw
    assert attend(heads=2 * 129, qs=258 * 128, os_=258 * 128, out=1 << 30) == rkv.ERR_UNSUPPORTED
    assert attend(rows=0, q=None, out=None) == rkv.OK
    assert attend(weight=A, width=64, size=0) == rkv.ERR_CAPACITY
    assert attend(weight=A, width=64, ws=None) == rkv.ERR_ARG
    assert attend(weight=A, width=64, ws=A + 4) == rkv.ERR_ARG


def test_workspace_is_a_host_computation():
    def size(p=None, b=None, heads=4, rows=8, weight=0):
        n = ctypes.c_longlong(-1)
        rc = rkv._lib.rkv_paged_workspace(p or pool(k=None, v=None), b or batch(page_table=None, kv_len=None), heads, rows,
                                          weight, ctypes.byref(n))
        return rc, n.value

    assert size()[0] == rkv.OK and size()[1] >= 0
    assert size(weight=1)[1] >= size()[1] + 8 * 4 * 4 - 255
    assert size(rows=0)[0] == rkv.OK
    assert size(heads=3)[0] == rkv.ERR_ARG
    assert size(rows=-1)[0] == rkv.ERR_ARG
    assert size(p=pool(page_tokens=17))[0] == rkv.ERR_UNSUPPORTED
    assert rkv._lib.rkv_paged_workspace(pool(), batch(), 4, 8, 0, None) == rkv.ERR_ARG
    # scores of 2^28 rows of 4 heads over 2^24 tokens: past any memory, and 64 bits where both grow further
    far = batch(max_q=1, table_stride=1 << 20, max_kv=1 << 24)
    assert size(b=far, rows=1 << 28)[0] == rkv.OK
    assert size(b=far, rows=1 << 28, weight=1)[0] == rkv.ERR_UNSUPPORTED
    assert size(b=far, rows=2, weight=1)[0] == rkv.OK


def test_evict_refusals():
    for kw in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(keep=8, sinks=4, recent=5), dict(weight=None),
               dict(weight=A + 2), dict(width=63), dict(kept=None), dict(out=None),
               dict(keep=2, sinks=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert evict(**kw) == rkv.ERR_ARG, kw
    for keep in ((1 << 30) + 1, (1 << 31) - 1):
        assert evict(keep=keep) == rkv.ERR_UNSUPPORTED
    assert rkv._lib.rkv_paged_poll_status(None, None) == rkv.ERR_ARG
    assert rkv._lib.rkv_paged_poll_status(A + 2, None) == rkv.ERR_ARG
    assert "page" in rkv.status_string(rkv.ERR_PAGE)


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    with pytest.raises(rkv.RkvError) as e:  # not on a GPU
        rkv.PagePool(torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16))
    assert e.value.code == rkv.ERR_ARG
    with pytest.raises(rkv.RkvError):
        rkv.PagedBatch(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), None, 1, 64)


def test_workspace_of_kept_scores_is_bounded():
    """Scores go by max_kv, up to 2^32 bytes; past that none are kept."""
    def size(weight, kv, rows=8, max_q=8, heads=4):
        n = ctypes.c_longlong(-1)
        b = batch(max_q=max_q, table_stride=kv // 16, max_kv=kv)
        assert rkv._lib.rkv_paged_workspace(pool(), b, heads, rows, weight, ctypes.byref(n)) == rkv.OK
        return n.value

    most = (1 << 32) // (4 * 8 * 4)
    extra = [size(1, kv) - size(0, kv) for kv in (most, most + 64, 16 * most)]
    assert extra[0] >= 1 << 32 and extra[0] < (1 << 32) + 1024
    assert extra[1] == extra[2] < 1024
    assert size(1, most, max_q=20) - size(0, most, max_q=20) < 1024  # more rows: never
