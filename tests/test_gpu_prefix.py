"""GPU parity of attention over shared prefixes (include/vas.h: paged_attn_fwd_prefix)
against the float64 oracle on the same tables, where every sequence stands for itself."""
import numpy as np
import pytest
import torch

from verify_attention_spec_gb300 import workloads as wl

from gpu_common import (add_sink, ancestor_masks, check_quant_rel_l2, compare_attention,
                        oracle_attention, to_device)

pytestmark = pytest.mark.gpu


def shared_inputs(groups, Hq, Hkv, D, P, kv, seed):
    """groups: a list of (prefix tokens, [(suffix, ql), ...]); the whole pages of a prefix are
    one set of pages for the group.  A sequence's length is prefix + suffix."""
    lens, qlens, start, prefix = [], [], [0], []
    for pre, members in groups:
        for suf, ql in members:
            lens.append(pre + suf)
            qlens.append(ql)
        start.append(len(lens))
        prefix.append(pre)
    a = wl.attention_inputs(lens, qlens, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=P,
                            kv_dtype=kv, seed=seed)
    bt = a.block_table.numpy()
    for g, (pre, members) in enumerate(groups):
        bt[start[g]:start[g + 1], :pre // P] = bt[start[g], :pre // P]
    return a, np.asarray(start, np.int32), np.asarray(prefix, np.int32)


def run_prefix(vas, a, start, prefix, masks=None, workspace_bytes=None, out=None, lse=None, ws=None,
               share="always"):
    d = a.q.device
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(d)
    out = torch.empty_like(a.q) if out is None else out
    lse = torch.empty(a.q.shape[:2], dtype=torch.float32, device=d) if lse is None else lse
    quant = a.kv_dtype if a.kv_dtype in wl.QUANTIZED else None
    dims = vas.attn_dims(a.q, a.k_pages, a.block_table, a.seq_lens, quant=quant)
    if ws is None:
        ws = vas.alloc_prefix_workspace(dims, len(prefix), nbytes=workspace_bytes)
    tm = None if masks is None else torch.from_numpy(np.ascontiguousarray(masks).view(np.int64)).to(d)
    vas.paged_attn_fwd_prefix(a.q, a.k_pages, a.v_pages, a.block_table, a.seq_lens, a.query_lens,
                              t(start), t(prefix), out, lse, ws, k_scale=a.k_scale, v_scale=a.v_scale,
                              quant=quant, tree_mask=tm, share=share, dims=dims)
    torch.cuda.synchronize()
    return out, lse


def check(vas, groups, Hq, Hkv, D, P, kv, seed=1, parents=None, hide=True):
    a, start, prefix = shared_inputs(groups, Hq, Hkv, D, P, kv, seed)
    ref_o, ref_l = oracle_attention(a, parents=parents)
    masks = None if parents is None else ancestor_masks(parents, a.query_lens.numpy())
    ad = to_device(a)
    if hide:
        # Only the first member with query tokens has its shared pages read: the others'
        # entries name no page at all.
        for g, (pre, members) in enumerate(groups):
            first = next((j for j, m in enumerate(members) if m[1] > 0), None)
            if first is None or pre < 256 or sum(m[1] > 0 for m in members) < 2:
                continue
            rows = [start[g] + j for j in range(len(members)) if j != first]
            ad.block_table[rows, :pre // P] = -1
    out, lse = run_prefix(vas, ad, start, prefix, masks)
    assert vas.vas_last_device_error() == 0
    compare_attention(out, lse, ref_o, ref_l, kv)
    return ad, start, prefix, out, lse


D1 = (1, 1)
SHAPES = [(64, 8, 128, 32), (32, 8, 128, 16), (4, 4, 64, 16), (16, 2, 64, 32), (3, 1, 128, 16)]
KV = [wl.BF16, wl.FP8, wl.INT8]


@pytest.mark.parametrize("Hq,Hkv,D,P", SHAPES)
@pytest.mark.parametrize("kv", KV)
def test_groups_of_every_kind(vas_lib, Hq, Hkv, D, P, kv):
    """Decode rows and windows; prefixes that end in a page, at a page, one page past the
    smallest shared length; a group with idle members first, in the middle and last; one
    member; a short prefix; none; an empty group."""
    groups = [(300, [(1, 1), (40, 5), (7, 7), (200, 1)]),
              (256, [(9, 0), (64, 1), (3, 0), (1, 1), (0, 0)]),
              (1000, [(5, 5)]),
              (512, []),
              (64, [(3, 1), (80, 2)]),
              (0, [(30, 1), (1, 1)]),
              (1024 + 31, [(1, 1)] * 9 + [(100, 17)])]
    check(vas_lib, groups, Hq, Hkv, D, P, kv, seed=Hq + D)


@pytest.mark.parametrize("kv", [wl.BF16, wl.FP8])
@pytest.mark.parametrize("members", [2, 15, 16, 17, 31, 33, 48, 64, 65])
def test_row_counts(vas_lib, members, kv):
    """Rows of a group around the tile sizes: 8 a member and KV head."""
    check(vas_lib, [(768, [D1] * members)], 16, 2, 128, 16, kv, seed=members)


@pytest.mark.parametrize("pre", [256, 272, 383, 384, 400, 511, 513, 1023, 2500, 9000])
@pytest.mark.parametrize("P", [16, 32])
def test_prefix_lengths(vas_lib, pre, P):
    check(vas_lib, [(pre, [(20, 3), (1, 1), (5, 2), (33, 33), (9, 1)])], 32, 4, 128, P, wl.BF16, seed=pre)
    check(vas_lib, [(pre, [(20, 3), (1, 1), (5, 2)])], 2, 2, 64, P, wl.INT8, seed=pre)


def test_prompt_chunks_on_a_prefix(vas_lib):
    """Long query windows: many row blocks of one group, the suffix on the chunk path."""
    check(vas_lib, [(2048, [(300, 300), (700, 257), (64, 64)])], 32, 8, 128, 16, wl.BF16, seed=3)
    check(vas_lib, [(600, [(129, 129), (300, 200)])], 16, 2, 64, 32, wl.FP8, seed=4)


@pytest.mark.parametrize("kv", [wl.BF16, wl.FP8])
def test_last_blocks_of_every_size(vas_lib, kv):
    """Groups of more rows than a block, whose last block has one row's heads, half a block,
    a little more, and all: 256 rows a block, 4 a token.  Odd and even numbers of tiles, so
    that heads begin behind padding, and groups one behind another."""
    def members(tokens):
        return [(40, tokens - 34)] + [(21, 17)] * 2 if tokens < 74 else [(90, tokens - 50), (60, 50)]
    for pre in (400, 1024):
        check(vas_lib, [(pre, members(t)) for t in (65, 96, 97, 128, 129)], 12, 3, 128, 16, kv, seed=pre)
    check(vas_lib, [(640, members(70)), (300, [(1, 1)] * 4), (2000, members(120))], 32, 8, 64, 32, kv, seed=12)


def test_many_groups(vas_lib):
    rng = np.random.default_rng(5)
    groups = [(int(rng.integers(256, 700)), [(int(rng.integers(1, 60)), 1) for _ in range(int(rng.integers(2, 6)))])
              for _ in range(90)]
    check(vas_lib, groups, 8, 2, 64, 16, wl.BF16, seed=6)


def test_many_members(vas_lib):
    """More members than the planner has threads."""
    check(vas_lib, [(320, [D1] * 400), (288, [(2, 2)] * 200)], 4, 1, 64, 16, wl.BF16, seed=7)


@pytest.mark.parametrize("kv", [wl.BF16, wl.INT8])
def test_trees_behind_a_prefix(vas_lib, kv):
    groups = [(512, [(20, 9), (33, 17), (64, 64), (4, 1)]), (0, [(50, 5)])]
    qlens = [m[1] for g in groups for m in g[1]]
    parents = wl.draft_tree_parents(qlens, seed=8, extra_roots=0.1)
    check(vas_lib, groups, 32, 8, 128, 16, kv, seed=8, parents=parents)


def test_large_scores(vas_lib):
    """Scores that grow along the prefix by hundreds: the running maximum moves in every
    tile; and a prefix that weighs nothing against the suffix, and the other way round."""
    for sign in (1.0, -1.0):
        a, start, prefix = shared_inputs([(2000, [(17, 1), (40, 3), (1, 1)])], 8, 2, 128, 16, wl.BF16, 9)
        bt = a.block_table.numpy()
        ramp = torch.arange(2048, dtype=torch.float32) / 2048 * 60 * sign
        q = torch.zeros_like(a.q)
        q[..., 0] = 100.0
        for i in range(3):
            for pg in range((int(a.seq_lens[i]) + 15) // 16):
                a.k_pages[bt[i, pg], :, :, 0] = ramp[pg * 16:pg * 16 + 16, None].to(torch.bfloat16)
        a.q = q
        ref_o, ref_l = oracle_attention(a)
        out, lse = run_prefix(vas_lib, to_device(a), start, prefix)
        # lse reaches 530, where half a step of fp32 is 2^-15 and the dot product's rounding
        # D times that at most: within the tolerance of 2e-3 times 4.
        assert np.abs(lse.double().cpu().numpy() - ref_l).max() <= 8e-3
        compare_attention(out, lse * 0, ref_o, ref_l * 0, wl.BF16)


def test_slots_past_the_end_are_not_read(vas_lib):
    """NaN in every slot behind the last token of each sequence, and in every page that no
    table names."""
    for kv in (wl.BF16, wl.FP8):
        a, start, prefix = shared_inputs([(300, [(17, 2), (5, 1), (40, 4)])], 8, 2, 128, 16, kv, 10)
        bt, lens = a.block_table.numpy(), a.seq_lens.numpy()
        used = np.zeros((a.num_pages, 16), bool)
        for i, L in enumerate(lens):
            for t in range(L):
                used[bt[i, t // 16], t % 16] = True
        dead = torch.from_numpy(~used)
        ref_o, ref_l = oracle_attention(a)
        for t in (a.k_pages, a.v_pages):
            t[dead] = 0x7F if kv == wl.FP8 else float("nan")
        if kv == wl.FP8:
            for t in (a.k_scale, a.v_scale):
                t.permute(0, 2, 1)[dead] = float("nan")
        out, lse = run_prefix(vas_lib, to_device(a), start, prefix)
        compare_attention(out, lse, ref_o, ref_l, kv)


def test_workspaces(vas_lib):
    """The smallest workspace (no room for partials: every member by itself), one with room
    for a few, the recommended; the same result within the tolerance, and the same bits
    again on a dirty workspace."""
    v = vas_lib
    a, start, prefix = shared_inputs([(3000, [D1] * 12), (700, [(9, 5)] * 3)], 32, 8, 128, 16, wl.BF16, 11)
    ref_o, ref_l = oracle_attention(a)
    ad = to_device(a)
    dims = v.attn_dims(ad.q, ad.k_pages, ad.block_table, ad.seq_lens)
    small, full = (f(dims, 2) for f in (v.paged_attn_prefix_workspace_min, v.paged_attn_prefix_workspace_size))
    assert 0 < v.paged_attn_workspace_min(dims) < small < full
    for n in (small, small + 27 * 32 * 516 * 2 + 4096, small + 27 * 32 * 516 * 3 + 4096, full, 4 * full):
        out, lse = run_prefix(v, ad, start, prefix, workspace_bytes=n)
        compare_attention(out, lse, ref_o, ref_l, wl.BF16)
    with pytest.raises(v.VasError):
        run_prefix(v, ad, start, prefix, workspace_bytes=small - 256)
    ws = v.alloc_prefix_workspace(dims, 2)
    o1, l1 = run_prefix(v, ad, start, prefix, ws=ws)
    ws.fill_(0xFF)
    o2, l2 = run_prefix(v, ad, start, prefix, ws=ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert v.vas_last_device_error() == 0


def test_ungrouped_sequences_and_no_groups(vas_lib):
    """Sequences before the first and behind the last group, and a call without groups, are
    paged_attn_fwd."""
    v = vas_lib
    a, _, _ = shared_inputs([(400, [(5, 1)] * 4)], 8, 2, 128, 16, wl.BF16, 12)
    ref_o, ref_l = oracle_attention(a)
    ad = to_device(a)
    for start, prefix in ([1, 3], [400]), ([0], []), ([2, 2], [400]), ([4, 4], [9]):
        out, lse = run_prefix(v, ad, np.array(start), np.array(prefix, np.int32))
        assert v.vas_last_device_error() == 0
        compare_attention(out, lse, ref_o, ref_l, wl.BF16)


def test_bad_groups_and_pages(vas_lib):
    v = vas_lib
    a, start, prefix = shared_inputs([(400, [(5, 1), (9, 2), (1, 1)]), (300, [(8, 3), (20, 1)])], 8, 2, 128, 16,
                                     wl.BF16, 13)
    ref_o, ref_l = oracle_attention(a)
    ad = to_device(a)

    def outcome(bits, bad, **kw):
        out, lse = run_prefix(v, kw.get("a", ad), kw.get("start", start), kw.get("prefix", prefix))
        assert v.vas_last_device_error() == bits
        ok = [r for r in range(8) if r not in bad]
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        compare_attention(out, lse, ref_o[ok], ref_l[ok], wl.BF16, rows=ok)

    # a prefix that reaches into a member's window: that member alone is refused
    outcome(v.VAS_DEV_BAD_LENGTHS, [3], prefix=np.array([401, 300]))
    outcome(v.VAS_DEV_BAD_LENGTHS, [0, 1, 2, 3], prefix=np.array([100000, 300]))
    # groups out of order, out of the batch, a negative prefix: nothing shared, all computed
    outcome(v.VAS_DEV_BAD_LENGTHS, [], start=np.array([0, 4, 2]))
    outcome(v.VAS_DEV_BAD_LENGTHS, [], start=np.array([-1, 3, 5]))
    outcome(v.VAS_DEV_BAD_LENGTHS, [], start=np.array([0, 3, 6]))
    outcome(v.VAS_DEV_BAD_LENGTHS, [], prefix=np.array([-1, 300]))
    # a sequence with bad lengths is refused as paged_attn_fwd does, the others computed
    b = to_device(a)
    b.seq_lens[4] = 1 << 29
    outcome(v.VAS_DEV_BAD_LENGTHS, [7], a=b)
    # a bad page in a shared prefix takes its group, in a suffix its sequence
    b = to_device(a)
    b.block_table[0:3, 7] = a.num_pages
    outcome(v.VAS_DEV_BAD_PAGE, [0, 1, 2, 3], a=b)
    b = to_device(a)
    b.block_table[1, 25] = -5
    outcome(v.VAS_DEV_BAD_PAGE, [1, 2], a=b)
    # a clean call afterwards
    outcome(0, [])


def test_binding_refusals(vas_lib):
    v = vas_lib
    a, start, prefix = shared_inputs([(300, [D1] * 3)], 8, 2, 128, 16, wl.BF16, 14)
    ad = to_device(a)
    with pytest.raises(ValueError):
        run_prefix(v, ad, start, np.array([300, 1]))
    with pytest.raises(ValueError):
        run_prefix(v, ad, start, prefix, out=torch.empty_like(ad.q)[:2])
    other = v.attn_dims(ad.q[:2], ad.k_pages, ad.block_table[:2], ad.seq_lens[:2])
    with pytest.raises(ValueError):
        v.paged_attn_fwd_prefix(ad.q, ad.k_pages, ad.v_pages, ad.block_table, ad.seq_lens, ad.query_lens,
                                torch.zeros(1, dtype=torch.int32, device="cuda"),
                                torch.zeros(0, dtype=torch.int32, device="cuda"), ad.q.clone(),
                                torch.empty(3, 8, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda"),
                                dims=other)
    with pytest.raises(ValueError):
        run_prefix(v, ad, start, prefix, share="sometimes")
    f = to_device(wl.attention_inputs([300] * 2, [1] * 2, num_q_heads=4, num_kv_heads=2, head_dim=64,
                                      page_size=16, kv_dtype=wl.F32, seed=1))
    with pytest.raises(v.VasError) as e:
        run_prefix(v, f, np.array([0, 2]), np.array([256]), workspace_bytes=1 << 20)
    assert e.value.status == v.VAS_E_UNSUPPORTED


def test_streams_and_graphs(vas_lib):
    """On a side stream behind the copy of its inputs, and captured: a replay with other
    inputs gives their result."""
    v = vas_lib
    a, start, prefix = shared_inputs([(900, [D1] * 10 + [(30, 5)])], 16, 2, 128, 16, wl.BF16, 15)
    ad = to_device(a)
    o1, l1 = run_prefix(v, ad, start, prefix)
    q = ad.q.clone()
    ad.q.zero_()
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
    st, pl = t(start), t(prefix)
    out, lse = torch.empty_like(o1), torch.empty_like(l1)
    dims = v.attn_dims(ad.q, ad.k_pages, ad.block_table, ad.seq_lens)
    ws = v.alloc_prefix_workspace(dims, 1)
    call = lambda: v.paged_attn_fwd_prefix(ad.q, ad.k_pages, ad.v_pages, ad.block_table, ad.seq_lens,
                                           ad.query_lens, st, pl, out, lse, ws, share="always", dims=dims)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
            call()
        torch.cuda._sleep(20_000_000)
        ad.q.copy_(q)
        g.replay()
    s.synchronize()
    assert torch.equal(out, o1) and torch.equal(lse, l1)
    assert v.vas_last_device_error() == 0


def test_groups_from_the_pool(vas_lib):
    """Forked sequences grouped by the pool, the batch as a scheduler builds it."""
    v = vas_lib
    P, Hq, Hkv, D = 16, 8, 2, 128
    pool = v.PagePool(400, P, seed=16)
    pool.admit(0, 1000)
    for i in range(1, 6):
        assert pool.fork(0, i, 1000) == 0
    pool.admit(50, 77)
    ids, qlens = [0, 1, 2, 3, 4, 5, 50], [1, 1, 5, 1, 1, 1, 2]
    for i, n in zip(ids, qlens):
        pool.grow(i, n)
    start, prefix = pool.prefix_groups(ids, qlens)
    assert list(start) == [0, 6, 7] and list(prefix) == [992, 0]
    bt, lens = pool.block_table(ids, 70)
    g = torch.Generator().manual_seed(17)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32))
    a = wl.AttentionInputs(mk(sum(qlens), Hq, D), mk(400, P, Hkv, D), mk(400, P, Hkv, D), t(bt), t(lens),
                           t(qlens), Hq, Hkv, D, P, wl.BF16)
    ref_o, ref_l = oracle_attention(a)
    out, lse = run_prefix(v, to_device(a), start, prefix)
    compare_attention(out, lse, ref_o, ref_l, wl.BF16)


def test_shared70b_full_size(vas_lib):
    """The 70B batch with 2048-token prompts shared by groups of 8, against
    paged_attn_fwd's result on the same tables."""
    from gpu_common import run_gpu_attention
    v = vas_lib
    ad = to_device(wl.workload_attention("shared70b", pool_device="cuda"))
    o1, l1 = run_gpu_attention(v, ad)
    out, lse = run_prefix(v, ad, np.arange(0, 513, 8), np.full(64, 2048))
    assert v.vas_last_device_error() == 0
    # Both are within the tolerance of the exact values: twice it apart at most, and lse too.
    assert float((out.float() - o1.float()).abs().max()) <= 2e-2
    assert float((lse - l1).abs().max()) <= 4e-3
    assert float((out.float() - o1.float()).norm() / o1.float().norm()) <= 1e-2


def test_auto_shares_where_it_pays(vas_lib):
    """Little to save: paged_attn_fwd's bits, and every member's own table is read.  Enough
    (100 members on 2048 tokens, 8 KV heads: 198 Mi elements of K), or a long prefix in a small
    batch: the prefix pages are the leader's."""
    from gpu_common import run_gpu_attention
    v = vas_lib
    a, start, prefix = shared_inputs([(600, [(9, 1)] * 5), (300, [(40, 5), (1, 1)])], 32, 8, 128, 16, wl.BF16, 18)
    ad = to_device(a)
    o1, l1 = run_gpu_attention(v, ad)
    o2, l2 = run_prefix(v, ad, start, prefix, share="auto")
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    for groups in ([(2048, [D1] * 100)], [(2048, [(9, 1)] * 2)], [(1024, [(9, 9)] * 3)]):
        a, start, prefix = shared_inputs(groups, 16, 8, 128, 16, wl.BF16, 19)
        ref_o, ref_l = oracle_attention(a)
        ad = to_device(a)
        ad.block_table[1:, :groups[0][0] // 16] = -1
        out, lse = run_prefix(v, ad, start, prefix, share="auto")
        assert v.vas_last_device_error() == 0
        compare_attention(out, lse, ref_o, ref_l, wl.BF16)


@pytest.mark.parametrize("kv", [wl.FP8, wl.INT8])
def test_queries_beyond_the_f16_range(vas_lib, kv):
    """|q| near 2^18 with the softmax scale divided by 2^16, behind a shared prefix of
    quantised pages: the queries are brought into f16's range by a power of two."""
    import oracle
    v = vas_lib
    a, start, prefix = shared_inputs([(500, [(20, 3), (1, 1), (7, 2)])], 32, 8, 128, 16, kv, 20)
    a.q = (a.q.float() * 65536.0).to(torch.bfloat16)  # exact: a power of two
    a.q[0] /= 65536.0                                 # one row of ordinary size among them
    scale = 1.0 / (65536.0 * np.sqrt(128))
    ref_o, ref_l = oracle.paged_attn_quant(
        wl.bf16_bits(a.q), a.k_pages.numpy(), a.v_pages.numpy(), a.k_scale.numpy(), a.v_scale.numpy(),
        a.block_table.numpy(), a.seq_lens.numpy(), a.query_lens.numpy(),
        fmt=oracle.Q_E4M3 if kv == wl.FP8 else oracle.Q_INT8, scale=scale)
    ad = to_device(a)
    dims = v.attn_dims(ad.q, ad.k_pages, ad.block_table, ad.seq_lens, scale=scale, quant=kv)
    out, lse = torch.empty_like(ad.q), torch.empty(ad.q.shape[:2], device="cuda")
    ws = v.alloc_prefix_workspace(dims, 1)
    t = lambda x: torch.from_numpy(x).cuda()
    v.paged_attn_fwd_prefix(ad.q, ad.k_pages, ad.v_pages, ad.block_table, ad.seq_lens, ad.query_lens, t(start),
                            t(prefix), out, lse, ws, k_scale=ad.k_scale, v_scale=ad.v_scale, quant=kv,
                            share="always", dims=dims)
    torch.cuda.synchronize()
    compare_attention(out, lse, ref_o, ref_l, kv)


def test_two_layers_share_a_workspace_in_a_graph(vas_lib):
    """Two captured calls on one workspace, one behind the other, and two graphs replayed in
    turn: each gives its own result."""
    v = vas_lib
    cases = []
    for seed, members in ((21, 9), (22, 30)):
        a, start, prefix = shared_inputs([(800, [D1] * members + [(30, 5)])], 16, 2, 128, 16, wl.BF16, seed)
        ad = to_device(a)
        want = run_prefix(v, ad, start, prefix)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        cases.append((ad, t(start), t(prefix), torch.empty_like(want[0]), torch.empty_like(want[1]), want))
    dims = [v.attn_dims(c[0].q, c[0].k_pages, c[0].block_table, c[0].seq_lens) for c in cases]
    ws = torch.empty(max(v.paged_attn_prefix_workspace_size(d, 1) for d in dims), dtype=torch.uint8, device="cuda")

    def call(c, d):
        a = c[0]
        v.paged_attn_fwd_prefix(a.q, a.k_pages, a.v_pages, a.block_table, a.seq_lens, a.query_lens, c[1], c[2],
                                c[3], c[4], ws, share="always", dims=d)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs = []
        for order in ((0, 1), (1, 0, 1)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for i in order:
                    call(cases[i], dims[i])
            graphs.append(g)
        for c in cases:
            c[3].zero_()
        for k in (0, 1, 0, 0, 1):
            graphs[k].replay()
    s.synchronize()
    for c in cases:
        assert torch.equal(c[3], c[5][0]) and torch.equal(c[4], c[5][1])
    assert v.vas_last_device_error() == 0


@pytest.mark.parametrize("kv", [wl.FP8, wl.INT8])
@pytest.mark.parametrize("weight,sink_v,amplitude", [(0.55, 0.02, 1.0), (0.9, 0.02, 0.25), (0.55, 0.02, 0.05),
                                                     (0.9, 0.02, 0.05), (0.9, 0.02, 1e-12), (0.55, 0.02, 1e6)])
def test_weights_far_below_the_largest(vas_lib, kv, weight, sink_v, amplitude):
    """A first token, in the shared prefix, that takes most of the softmax and has a small V:
    the output is made by the many small weights.  One stream of rows and two."""
    for members in (3, 12):
        a, start, prefix = shared_inputs([(4000, [(17, 1), (40, 5), (3, 3)] * (members // 3))], 32, 4, 128, 16, kv, 31)
        add_sink(a, weight, sink_v, amplitude, 4000)
        ref_o, ref_l = oracle_attention(a)
        out, lse = run_prefix(vas_lib, to_device(a), start, prefix)
        check_quant_rel_l2(out, lse, ref_o, ref_l)
    assert vas_lib.vas_last_device_error() == 0


@pytest.mark.parametrize("kv", [wl.FP8, wl.INT8])
@pytest.mark.parametrize("D,P", [(128, 32), (64, 16)])
def test_v_scales_that_change_along_a_prefix(vas_lib, kv, D, P):
    """Pages of a prefix whose V is up to 2^30 larger or smaller than their neighbours',
    growing, falling, at random and all small, some all zero."""
    rng = np.random.default_rng(33)
    n = 1500 // P
    for e in (np.linspace(-30, 0, n), np.linspace(0, -30, n), rng.integers(-30, 1, n), np.full(n, -30.0)):
        for groups in ([(1500, [(20, 1)] * 3)], [(1500, [(20, 7)] * 5)]):
            a, start, prefix = shared_inputs(groups, 16, 2, D, P, kv, 32)
            for c in range(n):
                a.v_scale[int(a.block_table[0, c])] *= float(2.0 ** np.round(e[c]))
            a.v_scale[int(a.block_table[0, n // 2])] = 0.0
            for i in range(len(a.seq_lens)):  # what follows the prefix is as small as its last page
                for c in range(n, -(-int(a.seq_lens[i]) // P)):
                    a.v_scale[int(a.block_table[i, c])] *= float(2.0 ** np.round(e[-1]))
            ref_o, ref_l = oracle_attention(a)
            out, lse = run_prefix(vas_lib, to_device(a), start, prefix)
            check_quant_rel_l2(out, lse, ref_o, ref_l)
    assert vas_lib.vas_last_device_error() == 0


@pytest.mark.parametrize("kv", [wl.FP8, wl.INT8])
@pytest.mark.parametrize("size", [2.0 ** 17, 2.0 ** 60])
def test_large_queries_of_one_member(vas_lib, kv, size):
    """Queries of one member far outside f16's range, along an element that no K has, beside
    ordinary ones of the other members: those keep all their bits."""
    for members in ([(17, 1), (40, 5), (3, 3)], [(17, 1), (40, 5), (3, 3)] * 5):
        a, start, prefix = shared_inputs([(700, members)], 32, 4, 128, 16, kv, 34)
        a.k_pages[..., 0] = 0
        a.q[0] = 0
        a.q[0, :, 0] = size
        ref_o, ref_l = oracle_attention(a)
        out, lse = run_prefix(vas_lib, to_device(a), start, prefix)
        check_quant_rel_l2(out, lse, ref_o, ref_l)
    assert vas_lib.vas_last_device_error() == 0


def test_more_groups_than_threads_and_uncached_lengths(vas_lib):
    """600 groups, and 5000 sequences, whose lengths the planner reads from memory each time
    it needs them; groups with idle members among them."""
    rng = np.random.default_rng(35)
    groups = [(int(rng.integers(250, 330)), [(int(rng.integers(1, 40)), 1)] * int(rng.integers(1, 4)))
              for _ in range(600)]
    check(vas_lib, groups, 4, 1, 64, 16, wl.BF16, seed=35)
    groups = [(256, [(2, int(q)) for q in rng.integers(0, 3, 50)]) for _ in range(100)]
    check(vas_lib, groups, 2, 1, 64, 16, wl.FP8, seed=36)
