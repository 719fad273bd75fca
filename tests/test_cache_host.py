"""Host side of the cache operators (include/vas.h: vas_pool_compact, vas_seq_fork_tail,
vas_build_prefix_groups, and what paged_kv_append, paged_kv_copy and paged_kv_keep_path
refuse before any CUDA call).  CPU only."""
import ctypes

import numpy as np
import pytest

P_ = ctypes.c_void_p
FAKE, NULL = P_(1 << 20), P_(0)  # never dereferenced: the checks come first


# ---- pool ----------------------------------------------------------------------------
def _content(pool, ids, maxp, store):
    """What each sequence reads through its table from a page-number-indexed store."""
    bt, lens = pool.block_table(ids, maxp)
    P = pool.page_size
    return [store[bt[r, :(n + P - 1) // P]].reshape(-1)[:n].copy() for r, n in enumerate(lens)]


def test_compact_keeps_every_sequence(vas_lib):
    rng = np.random.default_rng(3)
    P, N = 16, 120
    pool = vas_lib.PagePool(N, P, seed=11)
    ids = []
    for i in range(30):
        if pool.admit(i, int(rng.integers(1, 100))) == vas_lib.VAS_OK:
            ids.append(i)
    for i in list(ids)[::3]:
        assert pool.free(i) == vas_lib.VAS_OK
        ids.remove(i)
    n = min(pool.seq_len(ids[1]), 40)
    assert pool.fork(ids[1], 99, n) == vas_lib.VAS_OK
    ids.append(99)
    store = rng.integers(0, 1 << 30, (N, P))
    before = _content(pool, ids, 8, store)
    counts = sorted(pool.refcount(p) for p in range(N))
    free, used = pool.free_pages, N - pool.free_pages
    src, dst = pool.compact()
    assert len(set(src)) == len(src) == len(set(dst)) and not set(src) & set(dst)
    store[dst] = store[src]
    for a, b in zip(before, _content(pool, ids, 8, store)):
        np.testing.assert_array_equal(a, b)
    assert pool.free_pages == free and counts == sorted(pool.refcount(p) for p in range(N))
    assert all(pool.refcount(p) > 0 for p in range(used))
    assert all(pool.refcount(p) == 0 for p in range(used, N))
    # compact again: nothing to move; the next page handed out is the lowest free one
    assert len(pool.compact()[0]) == 0
    assert pool.admit(1000, 1) == vas_lib.VAS_OK
    assert pool.block_table([1000], 1)[0][0, 0] == used


def test_compact_refusals_change_nothing(vas_lib):
    pool = vas_lib.PagePool(8, 16, seed=0)
    pool.admit(1, 32)
    pool.admit(2, 32)
    pool.free(1)
    h, buf = pool._h, (ctypes.c_int32 * 8)()
    fn = vas_lib._lib.vas_pool_compact
    assert fn(h, None, None, 0) == 2
    assert fn(h, buf, buf, 1) == vas_lib.VAS_E_INVALID_ARG   # no room for the moves
    assert fn(h, buf, buf, -1) == vas_lib.VAS_E_INVALID_ARG
    assert fn(NULL, buf, buf, 8) == vas_lib.VAS_E_INVALID_ARG
    assert list(pool.block_table([2], 2)[0][0]) == [2, 3]
    empty = vas_lib.PagePool(0, 16)
    assert len(empty.compact()[0]) == 0


def test_fork_tail(vas_lib):
    pool = vas_lib.PagePool(32, 16, seed=5)
    pool.admit(1, 70)
    assert pool.fork(1, 2, 70) == 0
    bt, _ = pool.block_table([1, 2], 5)
    assert pool.fork_tail(1, 2, 70) == (bt[0, 4], bt[1, 4], 6)
    assert pool.fork(1, 3, 64) == 0
    assert pool.fork_tail(1, 3, 64) is None            # whole pages only: nothing to copy
    assert pool.fork_tail(1, 1, 70) is None            # one page, no copy of itself
    assert pool.fork_tail(1, 3, 0) is None
    for bad in [(1, 9, 70), (9, 2, 70)]:
        with pytest.raises(vas_lib.VasError):
            pool.fork_tail(*bad)
    with pytest.raises(vas_lib.VasError):
        pool.fork_tail(1, 2, 71)                       # past either length
    with pytest.raises(vas_lib.VasError):
        pool.fork_tail(1, 2, -1)


def test_prefix_groups(vas_lib):
    P = 16
    pool = vas_lib.PagePool(400, P, seed=9)
    pool.admit(0, 200)
    for i in (1, 2, 3):
        assert pool.fork(0, i, 200) == 0               # 12 whole pages shared
    pool.admit(10, 50)
    pool.admit(20, 100)
    assert pool.fork(20, 21, 96) == 0                  # 6 pages
    pool.grow(21, 1)
    start, lens = pool.prefix_groups([0, 1, 2, 3, 10, 20, 21])
    assert list(start) == [0, 4, 5, 7] and list(lens) == [192, 0, 96]
    # The query tokens are never shared: a window that reaches into the common pages
    # shortens the prefix.
    start, lens = pool.prefix_groups([0, 1, 2, 3], [1, 9, 1, 1])
    assert list(start) == [0, 4] and list(lens) == [176]
    # A sequence that shares one page only would cost the group before it eleven.
    assert pool.fork(0, 4, 16) == 0
    pool.grow(4, 100)
    start, lens = pool.prefix_groups([0, 1, 4])
    assert list(start) == [0, 2, 3] and list(lens) == [192, 0]
    # ... and two that share only a little still make a group of their own.
    start, lens = pool.prefix_groups([4, 0])
    assert list(start) == [0, 2] and list(lens) == [16]
    assert [list(x) for x in pool.prefix_groups([])] == [[0], []]
    with pytest.raises(vas_lib.VasError):
        pool.prefix_groups([77])
    with pytest.raises(vas_lib.VasError):
        pool.prefix_groups([0], [201])                 # a window longer than its sequence
    with pytest.raises(vas_lib.VasError):
        pool.prefix_groups([0], [-1])


# ---- refusals of the device entry points --------------------------------------------------
def _append(v, *, ptrs=None, **kw):
    d = dict(num_seqs=4, total_tokens=10, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16,
             num_pages=100, max_pages_per_seq=10, kv_dtype=v.VAS_BF16, rotary_dim=128, interleaved=0,
             max_position=500, q_stride=32 * 128, k_stride=8 * 128, v_stride=8 * 128, eps=1e-6)
    d.update(kw)
    quant = d["kv_dtype"] in (v.VAS_FP8_E4M3, v.VAS_INT8)
    at = lambda i: P_((1 << 30) + (i << 24))
    p = dict(q=at(0), k=at(1), v=at(2), qw=at(3), kw=at(4), cs=at(5), pos=at(6), bt=at(7), lens=at(8),
             ql=at(9), out=at(10), kp=at(11), vp=at(12), ks=at(13) if quant else NULL,
             vs=at(14) if quant else NULL)
    p.update(ptrs or {})
    return v._lib.paged_kv_append(*p.values(), ctypes.byref(v.vas_append_dims(**d)), NULL)


def test_append_refusals(vas_lib):
    v = vas_lib
    bad, uns = v.VAS_E_INVALID_ARG, v.VAS_E_UNSUPPORTED
    for kw in [dict(head_dim=96), dict(page_size=8), dict(kv_dtype=4), dict(kv_dtype=-1),
               dict(rotary_dim=8), dict(rotary_dim=144), dict(interleaved=2)]:
        assert _append(v, **kw) == uns, kw
    for kw in [dict(num_seqs=-1), dict(total_tokens=-1), dict(num_kv_heads=0), dict(num_q_heads=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(num_pages=0),
               dict(max_pages_per_seq=0), dict(q_stride=32 * 128 - 8), dict(k_stride=8 * 128 + 4),
               dict(v_stride=-1024), dict(rotary_dim=-16), dict(max_position=-1),
               dict(num_pages=1 << 28)]:
        assert _append(v, **kw) == bad, kw
    for name in ["q", "k", "v", "cs", "bt", "lens", "ql", "out", "kp", "vp"]:
        assert _append(v, ptrs={name: NULL}) == bad, name
    for name in ["q", "k", "v", "qw", "kw", "cs", "out", "kp", "vp"]:
        assert _append(v, ptrs={name: P_((1 << 31) + 8)}) == bad, name
    for name in ["pos", "bt", "lens", "ql"]:
        assert _append(v, ptrs={name: P_((1 << 31) + 2)}) == bad, name
    # scales with quantised pools, and only with them
    assert _append(v, ptrs={"ks": FAKE}) == bad
    assert _append(v, kv_dtype=v.VAS_INT8, ptrs={"vs": NULL}) == bad
    # q_out over q in another layout, or over k
    q = P_(1 << 30)
    assert _append(v, q_stride=48 * 128, ptrs={"out": q}) == bad
    assert _append(v, ptrs={"out": P_((1 << 30) + 256)}) == bad
    assert _append(v, ptrs={"out": P_((1 << 30) + (1 << 24))}) == bad
    # an empty step does nothing
    assert _append(v, num_seqs=0) == v.VAS_OK and _append(v, total_tokens=0) == v.VAS_OK


def _pool(v, **kw):
    d = dict(num_layers=2, num_pages=100, page_size=16, num_kv_heads=8, head_dim=128,
             kv_dtype=v.VAS_BF16)
    d.update(kw)
    return ctypes.byref(v.vas_pool_dims(**d))


def _copy(v, src, dst, tokens=None, ptrs=(FAKE, FAKE, NULL, NULL), n=None, **kw):
    arr = lambda x: None if x is None else (ctypes.c_int32 * max(1, len(x)))(*x)
    return v._lib.paged_kv_copy(*ptrs, arr(src), arr(dst), arr(tokens), len(src) if n is None else n,
                                _pool(v, **kw), NULL)


def test_copy_refusals(vas_lib):
    v = vas_lib
    bad, uns = v.VAS_E_INVALID_ARG, v.VAS_E_UNSUPPORTED
    assert _copy(v, [1, 2], [3, 3]) == bad            # one target twice
    assert _copy(v, [1, 2], [2, 3]) == bad            # a target that is also a source
    assert _copy(v, [1], [1]) == bad
    for pages in (100, 100000):                       # the pairs in a map of the pool, or sorted
        assert _copy(v, [1, 2, 9], [3, 4, 3], num_pages=pages) == bad
        assert _copy(v, [1, 2, 9], [3, 9, 5], num_pages=pages) == bad
        assert _copy(v, [1, 2, 9], [3, 4, pages], num_pages=pages) == bad
    assert _copy(v, [1], [100]) == bad and _copy(v, [-1], [4]) == bad
    assert _copy(v, [1], [2], tokens=[0]) == bad and _copy(v, [1], [2], tokens=[17]) == bad
    assert _copy(v, [1], [2], n=-1) == bad
    assert _copy(v, [], []) == v.VAS_OK
    assert _copy(v, [1], [2], num_layers=0) == v.VAS_OK
    assert _copy(v, [1], [2], ptrs=(NULL, FAKE, NULL, NULL)) == bad
    assert _copy(v, [1], [2], ptrs=(P_((1 << 20) + 8), FAKE, NULL, NULL)) == bad
    assert _copy(v, [1], [2], ptrs=(FAKE, FAKE, FAKE, NULL)) == bad     # scales of a bf16 pool
    assert _copy(v, [1], [2], kv_dtype=v.VAS_FP8_E4M3) == bad           # none of an FP8 pool
    for kw in [dict(head_dim=80), dict(page_size=64), dict(kv_dtype=9), dict(num_layers=40000)]:
        assert _copy(v, [1], [2], **kw) == uns, kw
    for kw in [dict(num_pages=-1), dict(num_kv_heads=0), dict(num_layers=-1)]:
        assert _copy(v, [1], [2], **kw) == bad, kw
    assert v._lib.paged_kv_copy(FAKE, FAKE, NULL, NULL, None, None, None, 1, _pool(v), NULL) == bad


def test_copy_refuses_pages_past_32_bits(vas_lib):
    """Byte offsets in a page are 32 bits, up to the end of the 16 KB segment that the page
    ends in: pages that end less than a segment below 2^31 are refused like larger ones."""
    v = vas_lib
    for heads in (262143, 262142, 262144, 1 << 30):   # 8192 bytes a head and page of 16 fp32 tokens
        assert _copy(v, [1], [2], num_kv_heads=heads, kv_dtype=v.VAS_F32) == v.VAS_E_UNSUPPORTED, heads


def test_keep_path_refusals(vas_lib):
    v = vas_lib
    bad = v.VAS_E_INVALID_ARG

    def keep(B=2, n=4, N=2, maxp=10, ptrs=None, **kw):
        p = dict(k=FAKE, v=FAKE, ks=NULL, vs=NULL, bt=FAKE, lens=FAKE, ql=FAKE)
        q = dict(index=NULL, path=FAKE, acc=FAKE)
        for name, x in (ptrs or {}).items():
            (p if name in p else q)[name] = x
        return v._lib.paged_kv_keep_path(*p.values(), N, maxp, *q.values(), B, n, _pool(v, **kw), NULL)

    for kw in [dict(B=-1), dict(n=0), dict(n=256), dict(N=-1), dict(maxp=-1), dict(B=3)]:
        assert keep(**kw) == bad, kw                   # B=3: more rows than sequences
    for name in ["k", "v", "bt", "lens", "ql", "path", "acc"]:
        assert keep(ptrs={name: NULL}) == bad, name
    assert keep(ptrs={"path": P_((1 << 20) + 2)}) == bad
    assert keep(ptrs={"ks": FAKE}) == bad
    assert keep(head_dim=72) == v.VAS_E_UNSUPPORTED
    assert keep(B=0) == v.VAS_OK and keep(num_layers=0) == v.VAS_OK


def test_prefix_attention_refusals(vas_lib):
    v = vas_lib
    d = dict(num_seqs=4, total_q_tokens=10, num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16,
             num_pages=100, max_pages_per_seq=10, kv_dtype=v.VAS_BF16, scale=0.0)

    def call(start=FAKE, lens=FAKE, groups=2, nbytes=1 << 30, q=FAKE, ks=NULL, share=0, **kw):
        dims = v.vas_attn_dims(**{**d, **kw})
        return v._lib.paged_attn_fwd_prefix(q, FAKE, FAKE, ks, NULL, FAKE, FAKE, FAKE, start, lens, NULL,
                                            FAKE, FAKE, ctypes.byref(dims), groups, share, FAKE, nbytes, NULL)

    bad, uns = v.VAS_E_INVALID_ARG, v.VAS_E_UNSUPPORTED
    assert call(share=2) == bad and call(share=-1) == bad
    assert call(groups=-1) == bad and call(start=NULL) == bad and call(lens=NULL) == bad
    assert call(start=P_((1 << 20) + 2)) == bad and call(q=NULL) == bad and call(ks=FAKE) == bad
    assert call(num_q_heads=30) == bad and call(kv_dtype=v.VAS_FP8_E4M3) == bad
    assert call(kv_dtype=v.VAS_F32) == uns and call(head_dim=80) == uns
    assert call(nbytes=64) == v.VAS_E_WORKSPACE
    assert call(num_seqs=0) == v.VAS_OK
    dims = v.vas_attn_dims(**d)
    sizes = [v.paged_attn_prefix_workspace_min(dims, g) for g in (0, 1, 1000)]
    assert 0 < sizes[0] <= sizes[1] < sizes[2]
    assert v.paged_attn_prefix_workspace_size(dims, 3) > v.paged_attn_prefix_workspace_min(dims, 3)
    assert v.paged_attn_prefix_workspace_size(dims, -1) == 0
    assert v.paged_attn_prefix_workspace_min(v.vas_attn_dims(**{**d, "kv_dtype": v.VAS_F32}), 1) == 0


def test_prefix_binding_refuses_dims_of_other_tensors(vas_lib):
    """dims kept from another batch, pool, table or code type are refused before anything is
    looked at on a device: the kernels take their extents from them."""
    import torch
    v = vas_lib
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)
    q, kv = z(6, 8, 64, t=torch.bfloat16), z(20, 16, 2, 64, t=torch.bfloat16)
    bt, lens = z(3, 10), z(3)
    base = v.attn_dims(q, kv, bt, lens)

    def call(dims, q=q, kv=kv, bt=bt, lens=lens, **kw):
        v.paged_attn_fwd_prefix(q, kv, kv, bt, lens, z(3), z(2), z(1), q, z(6, 8, t=torch.float32), z(64),
                                dims=dims, **kw)

    def refused(dims, **kw):
        with pytest.raises(ValueError, match="dims"):
            call(dims, **kw)

    for name, value in dict(num_seqs=2, total_q_tokens=5, num_q_heads=4, num_kv_heads=4, head_dim=128,
                            page_size=32, num_pages=21, max_pages_per_seq=11, kv_dtype=v.VAS_F32).items():
        d = v.attn_dims(q, kv, bt, lens)
        setattr(d, name, value)
        refused(d)
    refused(base, bt=z(3, 9))                            # a narrower table than that of the dims
    refused(base, q=z(6, 16, 64, t=torch.bfloat16))
    refused(base, kv=z(20, 32, 2, 64, t=torch.bfloat16))
    codes = z(20, 16, 2, 64, t=torch.uint8)
    refused(v.attn_dims(q, codes, bt, lens, quant="fp8"), kv=codes, quant="int8")
    refused(v.attn_dims(q, codes, bt, lens, quant="fp8"), kv=codes)


def test_append_binding_refuses_tokens_of_no_sequence(vas_lib):
    """The C entry point does nothing for an empty batch; with tokens in hand that would leave
    their q_out rows as they were."""
    import torch
    v = vas_lib
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)
    bf = torch.bfloat16
    kv, x = z(20, 16, 2, 64, t=bf), z(5, 2, 64, t=bf)
    with pytest.raises(ValueError, match="5 tokens of no sequence"):
        v.paged_kv_append(x, x, x, z(0, 4), z(0), z(0), x.clone(), kv, kv)


def test_append_in_place_of_one_token_with_any_stride(vas_lib):
    """One row is contiguous whatever its stride (a slice of one packed projection): q_out may
    be q.  Without a device the call goes on to fail there.  Several rows may not."""
    import torch
    v = vas_lib
    q = P_(1 << 30)
    if not torch.cuda.is_available():  # the addresses are not those of any memory
        assert _append(v, total_tokens=1, q_stride=48 * 128, ptrs={"out": q}) == v.VAS_E_CUDA
        assert _append(v, total_tokens=1, ptrs={"out": q}) == v.VAS_E_CUDA
    assert _append(v, total_tokens=2, q_stride=48 * 128, ptrs={"out": q}) == v.VAS_E_INVALID_ARG
    assert _append(v, total_tokens=1, q_stride=48 * 128, ptrs={"out": P_((1 << 30) + 256)}) == v.VAS_E_INVALID_ARG
