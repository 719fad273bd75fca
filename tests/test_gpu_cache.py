"""GPU tests of the operators that write and move the paged KV cache (include/vas.h:
paged_kv_append, paged_kv_copy, paged_kv_keep_path) against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

from verify_attention_spec_gb300 import workloads as wl

from gpu_common import compare_attention, oracle_attention, run_gpu_attention

pytestmark = pytest.mark.gpu

KV_TYPES = ["f32", "bf16", "fp8", "int8"]
EPS32 = 2.0 ** -24   # half a step of fp32, relative


def _act(kv):
    return torch.float32 if kv == "f32" else torch.bfloat16


def _cos_sin(rows, rot, theta=10000.0):
    ang = np.arange(rows)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)[None, :]
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))


def _pools(kv, pages, P, Hkv, D, lead=(), seed=1):
    g = torch.Generator().manual_seed(seed)
    shape = (*lead, pages, P, Hkv, D)
    if kv in ("f32", "bf16"):
        mk = lambda: torch.randn(shape, generator=g).to(_act(kv)).cuda()
        return mk(), mk(), None, None
    mk = lambda: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
    sc = lambda: torch.rand((*lead, pages, Hkv, P), generator=g).cuda()
    return mk(), mk(), sc(), sc()


class Case:
    """One append step: inputs on the device, and the definition in float64."""

    def __init__(self, lens, qlens, Hq, Hkv, D, P, kv, *, rot=None, inter=False, norm=True,
                 positions=None, seed=0, extra=0, packed=True):
        self.lens, self.qlens = np.asarray(lens), np.asarray(qlens)
        self.Hq, self.Hkv, self.D, self.P, self.kv = Hq, Hkv, D, P, kv
        self.rot, self.inter = D if rot is None else rot, inter
        g = torch.Generator().manual_seed(seed)
        T = int(self.qlens.sum())
        self.T = T
        act = _act(kv)
        # Values over several binades; one all-zero head row and one large one.
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g) * torch.exp2(
            torch.randint(-6, 7, (T, Hq + 2 * Hkv, 1), generator=g).float())
        if T:
            qkv[0, -1] = 0
            qkv[T // 2, Hq] = 0
        self.qkv = qkv.to(act).cuda()
        self.q, self.k, self.v = (self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:])
        if not packed:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.wq = (1 + 0.3 * torch.randn(D, generator=g)).to(act).cuda() if norm else None
        self.wk = (1 + 0.3 * torch.randn(D, generator=g)).to(act).cuda() if norm else None
        bt, pages = wl.build_pool(self.lens, P, seed + 5, int((-(-self.lens // P)).sum()) + extra)
        self.bt_np = bt
        self.kp, self.vp, self.ks, self.vs = _pools(kv, pages, P, Hkv, D, seed=seed + 9)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
        self.bt, self.lens_t, self.ql_t = t(bt), t(self.lens), t(self.qlens)
        self.pos_np = None if positions is None else np.asarray(positions)
        self.positions = None if positions is None else t(positions)
        top = int(max(self.lens.max(initial=0), 1 if positions is None else self.pos_np.max() + 1))
        self.cs = _cos_sin(top, self.rot).cuda() if self.rot else None
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=act, device="cuda")

    def call(self, vas, **kw):
        a = dict(cos_sin=self.cs, positions=self.positions, q_weight=self.wq, k_weight=self.wk,
                 interleaved=self.inter, eps=1e-5, k_scale=self.ks, v_scale=self.vs,
                 quant=self.kv if self.kv in wl.QUANTIZED else None)
        a.update(kw)
        vas.paged_kv_append(self.q, self.k, self.v, self.bt, self.lens_t, self.ql_t, self.q_out,
                            self.kp, self.vp, **a)

    def places(self):
        """(sequence, cache position) of every packed token."""
        seq = np.repeat(np.arange(len(self.qlens)), self.qlens)
        pos = np.concatenate([np.arange(L - q, L) for L, q in zip(self.lens, self.qlens)] or [[]])
        return seq, pos.astype(np.int64)

    def head(self, x, w):
        """(y, |u| + |v|): the transformed rows and the pair magnitudes that the fp32
        error bound goes by."""
        x = x.double().cpu().numpy()
        if w is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w.double().cpu().numpy()
        mag, y = np.abs(x), x.copy()
        if self.rot:
            at = self.places()[1] if self.pos_np is None else self.pos_np
            cs = self.cs.double().cpu().numpy()[at][:, None, :]
            cos, sin = cs[..., :self.rot // 2], cs[..., self.rot // 2:]
            h = self.rot // 2
            e, o = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.inter else (
                slice(0, h), slice(h, self.rot))
            y[..., e], y[..., o] = (x[..., e] * cos - x[..., o] * sin,
                                    x[..., o] * cos + x[..., e] * sin)
            s = mag[..., e] + mag[..., o]
            mag[..., e], mag[..., o] = s, s
        return y, mag


def _decode(codes, kv):
    return (codes.view(torch.float8_e4m3fn) if kv == "fp8" else codes.view(torch.int8)).double().cpu().numpy()


# Computation in fp32 (unit EPS32): the sum of D <= 128 squares as 16 fused terms a lane and
# 3 exchanges, its mean, the addition of eps, root and reciprocal leave a factor within
# (19 / 2 + 3) units; two products and the rotation (a product, a fused product, a sum) add 5
# more, relative to |u| + |v| of the pair.  24 units cover all of it.  Then one rounding to
# the stored type: half a step.
FP32_UNITS = 24


def _check_stored(c, got, y, mag, what):
    slack = FP32_UNITS * EPS32 * mag
    half = EPS32 if c.kv == "f32" else 2.0 ** -8
    err = np.abs(got.double().cpu().numpy() - y)
    bound = slack + half * (np.abs(y) + slack)
    assert np.all(err <= bound), (what, float((err - bound).max()))


def _check_codes(c, codes, scales, y, mag, what):
    """Dequantised rows against y.  The scale is max |y| / qmax: the maximum is off by
    FP32_UNITS of |u| + |v| <= 2 max |y| (a rotation keeps a pair's norm, which is at most
    sqrt 2 max |y| and at least (|u| + |v|) / sqrt 2), plus half a step of the division."""
    qmax = 448.0 if c.kv == "fp8" else 127.0
    amax = np.abs(y).max(-1)
    sc = scales.double().cpu().numpy()
    want = np.where(amax > 0, amax / qmax, 1.0)
    assert np.all(np.abs(sc - want) <= (2 * FP32_UNITS + 2) * EPS32 * want), what
    got = _decode(codes, c.kv) * sc[..., None]
    # A code is the rounding of y / scale: half a step (relative 2^-4, or 2^-10 scales below
    # the smallest normal, in E4M3; half a scale in INT8), the value itself being off by
    # slack and the scale's error, and by the division's half step.
    slack = FP32_UNITS * EPS32 * mag + (2 * FP32_UNITS + 4) * EPS32 * np.abs(y)
    # A largest element computed above its exact value saturates at qmax: covered by slack.
    half = np.maximum(2.0 ** -4 * (np.abs(y) + slack), 2.0 ** -10 * sc[..., None]) if c.kv == "fp8" \
        else 0.5 * sc[..., None] * (1 + 4 * EPS32)
    err = np.abs(got - y)
    assert np.all(err <= slack + half), (what, float((err - slack - half).max()))


def _check(c, before):
    yq, mq = c.head(c.q, c.wq)
    _check_stored(c, c.q_out, yq, mq, "q")
    seq, pos = c.places()
    page, slot = c.bt_np[seq, pos // c.P], pos % c.P
    pg, sl = torch.from_numpy(page).long().cuda(), torch.from_numpy(slot).cuda()
    yk, mk = c.head(c.k, c.wk)
    yv = c.v.double().cpu().numpy()
    if c.kv in wl.QUANTIZED:
        _check_codes(c, c.kp[pg, sl], c.ks[pg, :, sl], yk, mk, "k")
        _check_codes(c, c.vp[pg, sl], c.vs[pg, :, sl], yv, np.abs(yv), "v")
        # V is not transformed: its codes and scales are those of the pool's format exactly
        codes, sc = wl.quantize_pool(c.v.cpu()[:, None], c.kv)
        assert torch.equal(codes[:, 0], c.vp[pg, sl].cpu())
        assert torch.equal(sc[:, :, 0], c.vs[pg, :, sl].cpu())
    else:
        _check_stored(c, c.kp[pg, sl], yk, mk, "k")
        assert torch.equal(c.vp[pg, sl], c.v)
    # Every other slot of the pool is as it was.
    for now, old in zip((c.kp, c.vp, c.ks, c.vs), before):
        if now is None:
            continue
        a, b = now.clone(), old.clone()
        if a.dim() == 4:
            a[pg, sl] = 0
            b[pg, sl] = 0
        else:
            a[pg, :, sl] = 0
            b[pg, :, sl] = 0
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _run(vas, c, **kw):
    before = [None if t is None else t.clone() for t in (c.kp, c.vp, c.ks, c.vs)]
    c.call(vas, **kw)
    torch.cuda.synchronize()
    assert vas.vas_last_device_error() == 0
    _check(c, before)


# One token, a window over a page border, empty windows first, in the middle and last, a
# window that is its whole sequence, a sequence that holds nothing.
LENS = [40, 1, 17, 33, 0, 64, 5, 200, 31]
QLENS = [0, 1, 2, 33, 0, 5, 1, 37, 0]


@pytest.mark.parametrize("kv", KV_TYPES)
@pytest.mark.parametrize("Hq,Hkv,D,P", [(64, 8, 128, 32), (32, 8, 128, 16), (4, 4, 64, 16), (3, 1, 64, 32),
                                        (5, 5, 128, 16)])
def test_append_shapes(vas_lib, kv, Hq, Hkv, D, P):
    _run(vas_lib, Case(LENS, QLENS, Hq, Hkv, D, P, kv, seed=D + Hq, extra=7))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (16, True), (48, False), (48, True),
                                       (112, False), (128, True)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_rotations(vas_lib, kv, rot, inter, norm):
    _run(vas_lib, Case(LENS, QLENS, 6, 2, 128, 16, kv, rot=rot, inter=inter, norm=norm, seed=rot))


@pytest.mark.parametrize("B", [1, 256, 257, 1000])
def test_append_many_sequences(vas_lib, B):
    """One token each for more sequences than a block has threads (the scan's steps), with
    empty windows between them."""
    rng = np.random.default_rng(B)
    ql = (rng.random(B) < 0.8).astype(np.int64) * rng.integers(1, 4, B)
    ql[0] = 2
    _run(vas_lib, Case(ql + rng.integers(0, 50, B), ql, 4, 2, 64, 16, "bf16", seed=B))


def test_append_prompt(vas_lib):
    """A long chunk takes several rows a lane; another one the same rows one a lane."""
    _run(vas_lib, Case([1500, 700], [1024, 700], 64, 8, 128, 32, "bf16", seed=4))
    _run(vas_lib, Case([1500, 700], [1024, 700], 64, 8, 128, 32, "fp8", seed=5, inter=True, rot=64))
    _run(vas_lib, Case([3000], [2999], 16, 2, 64, 16, "f32", seed=6))


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 64), (5, 1, 64), (33, 2, 128), (1, 1, 128)])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_append_heads_that_leave_a_group_empty(vas_lib, Hq, Hkv, D, kv):
    """Many tokens whose heads do not fill the last group of rows: a step of it has few heads
    or none."""
    _run(vas_lib, Case([2600, 901], [2560, 900], Hq, Hkv, D, 16, kv, rot=32, inter=Hq == 16, seed=Hq))


def test_append_positions_and_tree_depths(vas_lib):
    """Explicit positions turn the rows; the slots stay where the packing puts them."""
    pos = np.concatenate([[9], [500, 501, 501, 502, 0]])
    _run(vas_lib, Case([10, 60], [1, 5], 8, 2, 128, 16, "bf16", positions=pos, seed=8))


def test_append_in_place_and_without_queries(vas_lib):
    c = Case(LENS, QLENS, 8, 2, 128, 16, "bf16", seed=10, packed=False)
    d = Case(LENS, QLENS, 8, 2, 128, 16, "bf16", seed=10, packed=False)
    c.call(vas_lib)
    d.q_out = d.q
    d.call(vas_lib)
    assert torch.equal(c.q_out, d.q) and torch.equal(c.kp, d.kp)
    e = Case(LENS, QLENS, 8, 2, 128, 16, "bf16", seed=10)
    vas_lib.paged_kv_append(None, e.k, e.v, e.bt, e.lens_t, e.ql_t, None, e.kp, e.vp, cos_sin=e.cs,
                            k_weight=e.wk, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(c.kp, e.kp) and torch.equal(c.vp, e.vp)


def test_append_is_repeatable_and_captures(vas_lib):
    """The same bits again, from a side stream and from a replayed graph with new inputs."""
    c = Case(LENS, QLENS, 8, 2, 128, 16, "fp8", seed=12)
    d = Case(LENS, QLENS, 8, 2, 128, 16, "fp8", seed=12)
    c.call(vas_lib)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    keep = d.qkv.clone()
    d.qkv.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            d.call(vas_lib)
        d.qkv.copy_(keep)
        g.replay()
    s.synchronize()
    for x, y in ((c.q_out, d.q_out), (c.kp, d.kp), (c.vp, d.vp), (c.ks, d.ks), (c.vs, d.vs)):
        assert torch.equal(x, y)


def test_append_reports_bad_tokens(vas_lib):
    """Bad lengths, pages and positions: NaN queries, nothing stored, the bits set, every
    other token as if they were not there."""
    v = vas_lib
    c = Case([40, 20, 30, 25], [2, 1, 3, 2], 4, 2, 64, 16, "bf16", seed=14)
    good = Case([40, 20, 30, 25], [2, 1, 3, 2], 4, 2, 64, 16, "bf16", seed=14)
    good.call(v)
    torch.cuda.synchronize()
    old = c.kp.clone()

    def outcome(bits, bad_rows):
        torch.cuda.synchronize()
        assert v.vas_last_device_error() == bits
        ok = [r for r in range(8) if r not in bad_rows]
        assert torch.isnan(c.q_out[bad_rows]).all()
        assert torch.equal(c.q_out[ok], good.q_out[ok])
        seq, pos = good.places()
        for r in range(8):
            at = (int(c.bt_np[seq[r], pos[r] // 16]), int(pos[r] % 16))
            want = old if r in bad_rows else good.kp
            assert torch.equal(c.kp[at], want[at]), r
        c.kp.copy_(old)

    c.lens_t[1] = 0                        # a window longer than its sequence
    c.call(v)
    outcome(v.VAS_DEV_BAD_LENGTHS, [2])
    c.lens_t[1] = 20
    c.bt[2, 1] = c.kp.shape[0]             # a page outside the pool
    c.call(v)
    outcome(v.VAS_DEV_BAD_PAGE, [3, 4, 5])
    c.bt[2, 1] = -1
    c.call(v)
    outcome(v.VAS_DEV_BAD_PAGE, [3, 4, 5])
    c.bt[2, 1] = int(c.bt_np[2, 1])
    pos = torch.from_numpy(good.places()[1].astype(np.int32)).cuda()
    pos[7] = c.cs.shape[0]
    pos[0] = -1
    c.call(v, positions=pos)
    outcome(v.VAS_DEV_BAD_POSITION, [0, 7])
    c.lens_t[0] = 1 << 30                  # past the table
    c.call(v)
    outcome(v.VAS_DEV_BAD_LENGTHS, [0, 1])
    c.lens_t[0] = 40
    c.ql_t[3] = 1                          # seven tokens for eight rows
    c.call(v)
    torch.cuda.synchronize()
    assert v.vas_last_device_error() == v.VAS_DEV_BAD_LENGTHS
    assert torch.isnan(c.q_out[7]).all() and torch.equal(c.q_out[:6], good.q_out[:6])
    c.ql_t[3] = 9                          # more tokens than rows: a sequence that does not fit
    c.call(v)
    torch.cuda.synchronize()
    assert v.vas_last_device_error() == v.VAS_DEV_BAD_LENGTHS
    assert torch.isnan(c.q_out[6:]).all() and torch.equal(c.q_out[:6], good.q_out[:6])


@pytest.mark.parametrize("kv", ["fp8", "int8"])
def test_append_extremes_of_the_scales(vas_lib, kv):
    """A row with an infinity or a NaN reads back as NaN or infinity, the smallest
    magnitudes as themselves or zero, and no other row is touched by them."""
    c = Case([5], [5], 2, 2, 64, 16, kv, rot=0, norm=False, seed=15)
    c.v[0, 0, 3] = float("inf")
    c.v[1, 0, 3] = float("nan")
    c.v[2, 0] = 0
    c.v[2, 0, 5] = 2.0 ** -133          # the smallest bf16: its scale rounds to zero or below
    c.v[3, 0] = 3.0e38
    c.call(vas_lib)
    torch.cuda.synchronize()
    page = int(c.bt_np[0, 0])
    sc = c.vs[page].cpu()
    assert not torch.isfinite(sc[0, 0]) and not torch.isfinite(sc[0, 1])
    assert torch.isfinite(sc[:, 2:5]).all() and torch.isfinite(sc[1, :5]).all()
    with np.errstate(invalid="ignore"):
        got = _decode(c.vp[page], kv) * sc.double().numpy().T[..., None]
    assert np.abs(got[2, 0]).max() <= 2.0 ** -132 and np.all(got[2, 0, :5] == 0)
    # 3.0e38 throughout: the largest code, times a scale half a step off
    x = float(torch.tensor(3.0e38).to(torch.bfloat16))
    np.testing.assert_allclose(got[3, 0], x, rtol=2 * EPS32)


def test_append_binding_refusals(vas_lib):
    c = Case([4], [4], 4, 2, 64, 16, "bf16", seed=16)
    for name, x in [("q", c.q.float()), ("k", c.k[:, :1]), ("v", c.v.transpose(1, 2)), ("q", c.q.cpu()),
                    ("bt", c.bt.long()), ("cs", c.cs.double()), ("q_out", c.q_out[:, :3]), ("wq", c.wq[:32]),
                    ("kp", c.kp.float()), ("lens_t", c.lens_t.cpu())]:
        d = Case([4], [4], 4, 2, 64, 16, "bf16", seed=16)
        setattr(d, name, x)
        with pytest.raises(ValueError):
            d.call(vas_lib)
    with pytest.raises(ValueError):
        c.call(vas_lib, quant="fp8")
    with pytest.raises(vas_lib.VasError):
        c.call(vas_lib, k_scale=torch.ones(c.kp.shape[0], 2, 16, device="cuda"))


# ---- copies ------------------------------------------------------------------------------
@pytest.mark.parametrize("kv", KV_TYPES)
@pytest.mark.parametrize("P,Hkv,D,layers", [(16, 8, 128, 0), (32, 2, 64, 3), (16, 1, 64, 1)])
@pytest.mark.parametrize("pairs", [1, 64, 65, 2049])
def test_copy_pages(vas_lib, kv, P, Hkv, D, layers, pairs):
    rng = np.random.default_rng(pairs + P)
    pages = 2 * pairs + 5
    pools = _pools(kv, pages, P, Hkv, D, lead=(layers,) if layers else (), seed=pairs)
    perm = rng.permutation(pages)
    src, dst = perm[:pairs], perm[pairs:2 * pairs]
    if pairs > 2:
        src = src.copy()
        src[1] = src[0]                  # one source, two copies
    for tokens in (None, rng.integers(1, P + 1, pairs)):
        want = [None if t is None else t.clone() for t in pools]
        n = np.full(pairs, P) if tokens is None else tokens
        live = torch.from_numpy(np.arange(P)[None, :] < n[:, None]).cuda()
        s, d = torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda()
        for t in want:
            if t is None:
                continue
            x = t if layers else t[None]
            if t is want[0] or t is want[1]:
                x[:, d] = torch.where(live[None, :, :, None, None], x[:, s], x[:, d])
            else:
                x[:, d] = torch.where(live[None, :, None, :], x[:, s], x[:, d])
        vas_lib.paged_kv_copy(pools[0], pools[1], src, dst, tokens=tokens, k_scale=pools[2],
                              v_scale=pools[3])
        torch.cuda.synchronize()
        for a, b in zip(pools, want):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_copy_reads_its_lists_before_it_returns(vas_lib):
    pools = _pools("bf16", 200, 16, 8, 128)
    src, dst = np.arange(90, dtype=np.int32), np.arange(100, 190, dtype=np.int32)
    want = pools[0].clone()
    want[100:190] = want[:90]
    torch.cuda._sleep(20_000_000)
    vas_lib.paged_kv_copy(pools[0], pools[1], src, dst)
    src[:], dst[:] = 195, 196
    torch.cuda.synchronize()
    assert torch.equal(pools[0], want)


def test_copy_binding_refusals(vas_lib):
    k, v, _, _ = _pools("bf16", 8, 16, 2, 64)
    for src, dst, tok in [([0], [1, 2], None), ([0], [1], [1, 2]), ([0.5], [1], None), ([0], [2**32 + 1], None),
                          ([[0]], [[1]], None)]:
        with pytest.raises(ValueError):
            vas_lib.paged_kv_copy(k, v, src, dst, tokens=tok)
    with pytest.raises(vas_lib.VasError):
        vas_lib.paged_kv_copy(k, v, [0, 0], [1, 1])
    with pytest.raises(ValueError):
        vas_lib.paged_kv_copy(k, v.cpu(), [0], [1])
    with pytest.raises(ValueError):
        vas_lib.paged_kv_copy(k, v[:4], [0], [1])
    vas_lib.paged_kv_copy(k, v, [], [])


# ---- accepted paths ------------------------------------------------------------------------
def _keep_reference(t, is_scale, c):
    """The moves in order of definition: all sources read, then all targets written."""
    x = t if c["layers"] else t[None]
    old = x.clone()
    for b, i in enumerate(c["index"]):
        base = c["lens"][i] - c["ql"][i]
        for s in range(max(0, c["acc"][b])):
            p0, p1 = base + c["path"][b][s], base + 1 + s
            g0, g1 = c["bt"][i, p0 // c["P"]], c["bt"][i, p1 // c["P"]]
            if is_scale:
                x[:, g1, :, p1 % c["P"]] = old[:, g0, :, p0 % c["P"]]
            else:
                x[:, g1, p1 % c["P"]] = old[:, g0, p0 % c["P"]]


def _keep_case(kv, P, Hkv, D, layers, n, seed, index=None):
    rng = np.random.default_rng(seed)
    N = 9
    ql = rng.integers(n + 1, n + 9, N)
    lens = ql + rng.integers(0, 70, N)
    bt, pages = wl.build_pool(lens, P, seed)
    index = list(range(N)) if index is None else index
    path = np.full((len(index), n), -1, np.int32)
    acc = rng.integers(-1, n + 1, len(index))
    for b, i in enumerate(index):
        m = max(0, acc[b])
        path[b, :m] = np.sort(rng.choice(np.arange(1, ql[i]), m, replace=False))
    return dict(P=P, layers=layers, bt=bt, lens=lens, ql=ql, index=index, path=path, acc=acc,
                pools=_pools(kv, pages, P, Hkv, D, lead=(layers,) if layers else (), seed=seed))


def _keep_call(vas, c, index=True):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()
    k, v, ks, vs = c["pools"]
    vas.paged_kv_keep_path(k, v, t(c["bt"]), t(c["lens"]), t(c["ql"]), t(c["path"]), t(c["acc"]),
                           seq_index=t(c["index"]) if index else None, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv", KV_TYPES)
@pytest.mark.parametrize("P,Hkv,D,layers,n", [(16, 8, 128, 0, 16), (32, 2, 64, 3, 5), (16, 5, 128, 2, 1),
                                              (32, 1, 64, 0, 63), (16, 16, 128, 0, 255)])
def test_keep_path(vas_lib, kv, P, Hkv, D, layers, n):
    for index in (None, [4, 0, 7]):
        c = _keep_case(kv, P, Hkv, D, layers, n, seed=n + P, index=index)
        want = [None if t is None else t.clone() for t in c["pools"]]
        for j, t in enumerate(want):
            if t is not None:
                _keep_reference(t, j >= 2, c)
        _keep_call(vas_lib, c, index=index is not None)
        assert vas_lib.vas_last_device_error() == 0
        for a, b in zip(c["pools"], want):
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_keep_path_skips_bad_rows(vas_lib):
    v = vas_lib

    def outcome(change, bits, bad):
        c = _keep_case("bf16", 16, 2, 64, 0, 6, seed=3)
        c["acc"][:] = 3
        c["path"][:, :3] = [2, 3, 5]
        good = dict(c, index=[i for i in c["index"] if i not in bad], pools=None)
        good["path"], good["acc"] = c["path"][good["index"]].copy(), c["acc"][good["index"]].copy()
        change(c)
        want = c["pools"][0].clone()
        _keep_reference(want, False, good)
        _keep_call(v, c)
        assert v.vas_last_device_error() == bits
        assert torch.equal(c["pools"][0], want)

    def setter(name, at, x):
        def f(c):
            c[name][at] = x
        return f

    outcome(setter("path", (2, 1), 2), v.VAS_DEV_BAD_TREE, [2])          # the same node twice
    outcome(setter("path", (2, 0), 0), v.VAS_DEV_BAD_TREE, [2])          # the root
    outcome(setter("path", (2, 2), 600), v.VAS_DEV_BAD_TREE, [2])        # past the window
    outcome(setter("acc", 5, 7), v.VAS_DEV_BAD_TREE, [5])                # more nodes than columns
    outcome(setter("index", 8, 9), v.VAS_DEV_BAD_TREE, [8])              # no such sequence
    outcome(setter("index", 8, -1), v.VAS_DEV_BAD_TREE, [8])
    outcome(setter("index", 8, 2), v.VAS_DEV_BAD_TREE, [8])              # a sequence named twice
    outcome(setter("lens", 4, 3), v.VAS_DEV_BAD_LENGTHS, [4])
    outcome(setter("lens", 4, 1 << 30), v.VAS_DEV_BAD_LENGTHS, [4])
    outcome(setter("bt", 6, -1), v.VAS_DEV_BAD_PAGE, [6])



@pytest.mark.parametrize("row", [0, 1])
def test_keep_path_that_falls_in_a_full_table(vas_lib, row):
    """A path that falls and rises again, in a sequence that fills its table: its later nodes
    belong behind the last page, where no entry of the table is looked up (the next row's
    first is none of the pool's pages)."""
    v = vas_lib
    lens, ql = np.array([64, 64]), np.array([6, 40])
    bt, pages = wl.build_pool(lens, 16, 4)
    path = np.full((2, 40), -1, np.int32)
    path[0, :6] = [5, 1, 2, 3, 4, 5]                  # node 5 would go to position 64
    path[1] = [38, *range(1, 40)]                     # node 39 to position 64
    acc = np.array([6, 40]) * (np.arange(2) == row)
    bt[1, 0] = -1 if row == 0 else bt[1, 0]
    c = dict(bt=bt, lens=lens, ql=ql, path=path, acc=acc, index=[0, 1], pools=_pools("bf16", pages, 16, 2, 64))
    before = [c["pools"][i].clone() for i in (0, 1)]
    _keep_call(v, c)
    assert v.vas_last_device_error() == v.VAS_DEV_BAD_TREE
    assert torch.equal(c["pools"][0], before[0]) and torch.equal(c["pools"][1], before[1])


# ---- together -------------------------------------------------------------------------------
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_serving_step(vas_lib, kv):
    """A prompt appended, forked, its tail copied; the child brings a draft tree, keeps an
    accepted path and is rolled back; the pool is compacted: attention over the result is
    that of the same tokens appended one after the other."""
    v = vas_lib
    P, Hq, Hkv, D, N = 16, 8, 2, 128, 64
    quant = kv if kv in wl.QUANTIZED else None
    pool = v.PagePool(N, P, seed=21)
    kp, vp, ks, vs = _pools(kv, N, P, Hkv, D, seed=22)
    scales = dict(k_scale=ks, v_scale=vs)
    cs = _cos_sin(200, D).cuda()
    g = torch.Generator().manual_seed(23)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    rows = torch.randn(60, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()

    def append(ids, qlens, x, positions=None):
        bt, lens = pool.block_table(ids, 8)
        q = torch.empty(x.shape[0], Hq, D, dtype=torch.bfloat16, device="cuda")
        v.paged_kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], dev(bt), dev(lens), dev(qlens), q,
                          kp, vp, cos_sin=cs, positions=positions, q_weight=w, k_weight=w, quant=quant,
                          **scales)
        return q, bt, lens

    pool.admit(99, 37)                                   # pages that will be holes
    pool.admit(1, 41)
    append([1], [41], rows[:41])
    assert pool.fork(1, 2, 41) == 0
    src, dst, tokens = pool.fork_tail(1, 2, 41)
    v.paged_kv_copy(kp, vp, [src], [dst], tokens=[tokens], **scales)
    pool.grow(2, 7)                                      # the root and six drafts
    depth = np.array([0, 1, 1, 2, 2, 3, 3])
    _, bt, lens = append([2], [7], rows[41:48], positions=dev(41 + depth))
    v.paged_kv_keep_path(kp, vp, dev(bt), dev(lens), dev([7]), dev([[2, 4, 5, -1, -1, -1]]), dev([3]),
                         **scales)
    pool.rollback(2, 3)
    pool.free(99)
    src, dst = pool.compact()
    assert len(src) > 0
    v.paged_kv_copy(kp, vp, src, dst, **scales)
    pool.grow(2, 1)
    q, bt, lens = append([2], [1], rows[50:51])

    # The same 46 tokens in a row into another sequence.
    assert pool.admit(3, 46) == 0
    order = list(range(42)) + [43, 45, 46] + [50]
    q3, _, _ = append([3], [46], rows[order])
    assert torch.equal(q[0], q3[-1])
    bt, lens = pool.block_table([2, 3], 8)
    a = wl.AttentionInputs(torch.cat([q, q]), kp, vp, dev(bt), dev(lens), dev([1, 1]), Hq, Hkv, D, P,
                           kv, ks, vs)
    out, lse = run_gpu_attention(v, a)
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])
    ref_o, ref_l = oracle_attention(a)
    compare_attention(out, lse, ref_o, ref_l, kv)
    assert v.vas_last_device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_offsets_past_32_bits(vas_lib, kv):
    """The last pages of a pool of more than 2^32 elements: append, keep path, copy and
    attention on a shared prefix give the bits that they give on the first pages of a small one."""
    v = vas_lib
    P, Hq, Hkv, D, N = 32, 16, 8, 128, 64
    big = 2 ** 32 // (P * Hkv * D) + 512
    quant = kv if kv in wl.QUANTIZED else None
    g = torch.Generator().manual_seed(31)
    L, ql = [300, 311, 290], [4, 5, 1]
    # The members share 8 pages; each has two of its own behind them.
    bt = np.array([list(range(8)) + [20 + 3 * i, 40 - i] for i in range(3)])
    rows = torch.randn(sum(ql), Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    cs = _cos_sin(400, D).cuda()
    first = _pools(kv, N, P, Hkv, D, seed=32)
    if quant:  # no NaN codes
        for t in first[:2]:
            t[(t & 0x7F) == 0x7F] = 0x3A
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()

    def steps(pools, at):
        kp, vp, ks, vs = pools
        scales = dict(k_scale=ks, v_scale=vs)
        table, lens, qlens = dev(bt + at), dev(L), dev(ql)
        q = torch.empty(sum(ql), Hq, D, dtype=torch.bfloat16, device="cuda")
        v.paged_kv_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], table, lens, qlens, q,
                          kp, vp, cos_sin=cs, quant=quant, **scales)
        v.paged_kv_keep_path(kp, vp, table, lens, qlens, dev([[2, 3], [3, 4], [-1, -1]]), dev([2, 2, 0]),
                             **scales)
        v.paged_kv_copy(kp, vp, [at + 20, at + 1], [at + 50, at + N - 1], tokens=[P, 7], **scales)
        dims = v.attn_dims(q, kp, table, lens, quant=quant)
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        v.paged_attn_fwd_prefix(q, kp, vp, table, lens, qlens, dev([0, 3]), dev([256]), out, lse,
                                v.alloc_prefix_workspace(dims, 1), dims=dims, quant=quant,
                                share="always", **scales)
        assert v.vas_last_device_error() == 0
        assert torch.isfinite(lse).all()
        return [q, out, lse] + [t[at:at + N] for t in pools if t is not None]

    last = [None if t is None else torch.zeros((big, *t.shape[1:]), dtype=t.dtype, device="cuda")
            for t in first]
    for small, large in zip(first, last):
        if large is not None:
            large[big - N:] = small
    small, large = steps(first, 0), steps(last, big - N)
    for x, y in zip(small, large):
        assert torch.equal(x, y)
    for t in last:
        assert t is None or not t[:big - N].any()


@pytest.mark.parametrize("B", [1024, 1025, 3000, 5003])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_append_more_sequences_than_starts(vas_lib, B, kv):
    """The first rows of up to 1024 sequences lie in shared memory; of more, only every 2nd
    to 5th, the last chunk not filled evenly, with empty windows at the chunks' ends."""
    rng = np.random.default_rng(B)
    ql = (rng.random(B) < 0.6).astype(np.int64) * rng.integers(1, 4, B)
    step = -(-B // 1024)
    ql[0] = ql[step - 1::2 * step] = ql[2 * step::3 * step] = 0
    ql[-1] = 2
    _run(vas_lib, Case(ql + rng.integers(0, 20, B), ql, 3, 1, 64, 16, kv, seed=B))


@pytest.mark.parametrize("B", [900, 1025, 2500])
def test_append_bad_lengths_of_many_sequences(vas_lib, B):
    """A window longer than its sequence, a table too short for it, windows that are too few
    and too many for the rows: those tokens are refused, the rest stored."""
    v = vas_lib
    rng = np.random.default_rng(B)
    ql = rng.integers(0, 3, B)
    bad = [B // 3, B // 2]
    ql[bad] = 2
    c = Case(ql + rng.integers(0, 20, B), ql, 2, 1, 64, 16, "bf16", seed=B)
    seq, pos = c.places()

    def outcome(refused):
        before = c.kp.clone()
        c.q_out.fill_(7.0)
        c.call(v)
        assert v.vas_last_device_error() == v.VAS_DEV_BAD_LENGTHS
        nan = torch.isnan(c.q_out.float()).flatten(1)
        want = torch.from_numpy(refused).cuda()
        assert torch.equal(nan.all(1), want) and torch.equal(nan.any(1), want)
        page = torch.from_numpy(c.bt_np[seq[refused], pos[refused] // 16]).long().cuda()
        slot = torch.from_numpy(pos[refused] % 16).cuda()
        assert torch.equal(c.kp[page, slot], before[page, slot])

    c.lens_t[bad[0]] = 1                                  # shorter than its window
    c.lens_t[bad[1]] = 16 * c.bt.shape[1] + 1             # past the table
    outcome(np.isin(seq, bad))
    c.lens_t.copy_(torch.from_numpy(c.lens))
    last = int(np.flatnonzero(ql)[-1])
    c.ql_t[last] = 0                                      # the last rows have no sequence
    outcome(seq == last)
    c.ql_t[last] = int(ql[last]) + 1                      # a window past the last row
    c.lens_t[last] = max(int(c.lens[last]), int(ql[last]) + 1)
    outcome(seq == last)
