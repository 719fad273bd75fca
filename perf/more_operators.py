"""Timed cases of the block-scaled cache and of the logits: attention over 8-bit pages with
one scale per page and KV head, the append that quantises such pages as it writes them, the
read-back of cached tokens, and the penalties, biases, masks and softmax that turn a
verification window's logits into the probabilities the rejection rule takes.

Each case runs either in its plain form (torch operations in 32 bits) or, with ``own`` set,
through the package's entry points.  Shapes are those of the package's workloads: the
Llama-3-8B layer (32/8 heads of 128, 16-token pages), the 70B layer (64/8 heads of 128,
32-token pages), small layers of 64-wide heads, vocabularies of 128256 and 32000.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 500000.0


# ---- cases ----------------------------------------------------------------------------
def listed():
    return [
        # Four short chats on one step of the 8B layer: the latency of the smallest batch.
        dict(name="attend_four", op="attend", kv="fp8", seqs=4, lo=40, hi=500, verify=0.0, k=0,
             hq=32, hkv=8, d=128, page=16),
        # One decode step of 64 sequences of the 8B layer.
        dict(name="attend_decode64", op="attend", kv="fp8", seqs=64, lo=128, hi=4096, verify=0.0,
             k=0, hq=32, hkv=8, d=128, page=16),
        # A full batch of the 70B layer, one sequence in eight verifying four drafts.
        dict(name="attend_batch512", op="attend", kv="fp8", seqs=512, lo=256, hi=4096,
             verify=0.125, k=4, hq=64, hkv=8, d=128, page=32),
        # Ragged verify windows on INT8 pages.
        dict(name="attend_int8_windows", op="attend", kv="int8", seqs=61, lo=100, hi=2500,
             verify=0.5, k=4, hq=32, hkv=8, d=128, page=16),
        # Eight 1024-token prompt chunks behind cached context (chunked prefill, 70B layer).
        dict(name="attend_chunks", op="attend", kv="fp8", seqs=8, lo=4096, hi=4096, verify=1.0,
             k=1023, hq=64, hkv=8, d=128, page=32),
        # One decode step of 64 sequences: each token joins a partly filled page.
        dict(name="append_decode64", op="append", kv="fp8", seqs=64, ql_lo=1, ql_hi=1, ctx=1024,
             hq=32, hkv=8, d=128, page=16, rot=128, inter=False, norm=True),
        # Eight 1024-token prompt chunks of the 70B layer.
        dict(name="append_prefill8", op="append", kv="fp8", seqs=8, ql_lo=1024, ql_hi=1024,
             ctx=1024, hq=64, hkv=8, d=128, page=32, rot=128, inter=False, norm=True),
        # Ragged prompts on 64-wide heads into INT8 pages, keys stored as they come.
        dict(name="append_ragged_int8", op="append", kv="int8", seqs=37, ql_lo=1, ql_hi=511, ctx=77,
             hq=16, hkv=2, d=64, page=16, rot=0, inter=False, norm=False),
        # Cached prompts of 16 requests handed to another program: FP8 pages back to bf16.
        dict(name="read_prompts", op="read", kv="fp8", out="bf16", seqs=16, lo=1000, hi=8192,
             skip=100, hkv=8, d=128, page=32),
        # The last tokens of a few sequences, INT8 pages to fp32: latency.
        dict(name="read_tails", op="read", kv="int8", out="f32", seqs=5, lo=1, hi=77, skip=300, hkv=2,
             d=64, page=16),
        # One decode step of four sequences, vocabulary 32000: penalties, then temperature.
        dict(name="logits_four", op="logits", kind="probs", seqs=4, n=0, vocab=32000, pad=0,
             type="f32", hist=500, bias=0, mask=False, tree=False),
        # 64 windows of four drafts over a vocabulary of 128256: everything at once.
        dict(name="logits_windows", op="logits", kind="probs", seqs=64, n=4, vocab=128256, pad=0,
             type="bf16", hist=2048, bias=40, mask=True, tree=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "read", "logits", "logits"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32])
    hkv, g = rng.choice([(8, 4), (8, 8), (4, 1), (2, 8), (1, 5)])
    if op == "attend":
        verify = rng.choice([0.0, 0.0, 0.25, 1.0])
        k = 0 if verify == 0.0 else _log(rng, 1, 700)
        seqs = _log(rng, 1, max(1, min(500, 6000 // (k + 1))))
        # tokens of a padded batch, and scores of its rows
        most = min(16000, 1000000 // seqs, 200000000 // (seqs * (k + 1) * hkv * g))
        hi = _log(rng, k + 2, max(k + 2, most))
        return dict(op=op, kv=rng.choice(["fp8", "fp8", "int8"]), seqs=seqs, lo=rng.randint(k + 1, hi),
                    hi=hi, verify=verify, k=k, hq=hkv * g, hkv=hkv, d=d, page=page)
    if op == "append":
        kv = rng.choice(["fp8", "fp8", "int8"])
        seqs = _log(rng, 1, 600)
        hi = _log(rng, 1, max(1, min(2048, 8000 // seqs)))
        raw = kv == "int8"
        return dict(op=op, kv=kv, seqs=seqs, ql_lo=rng.randint(1, hi), ql_hi=hi, ctx=_log(rng, 1, 1500),
                    hq=hkv * g, hkv=hkv, d=d, page=page, rot=0 if raw else rng.choice([d, d, d // 2]),
                    inter=not raw and rng.random() < 0.3, norm=not raw and rng.random() < 0.7)
    if op == "read":
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 1, max(1, 60000 // seqs))
        return dict(op=op, kv=rng.choice(["fp8", "int8", "fp8_token", "int8_token", "bf16"]),
                    out=rng.choice(["bf16", "f32"]), seqs=seqs, lo=rng.randint(1, hi), hi=hi,
                    skip=_log(rng, 1, 400), hkv=hkv, d=d, page=page)
    vocab = rng.choice([128256, 32000, _log(rng, 1000, 150000)])
    n = rng.randint(0, 8)
    return dict(op=op, kind=rng.choice(["probs", "probs", "logits"]),
                seqs=_log(rng, 1, max(1, 40000000 // (vocab * (n + 1)))), n=n, vocab=vocab,
                pad=rng.choice([0, 0, rng.randint(1, 200)]), type=rng.choice(["bf16", "bf16", "f32"]),
                hist=rng.choice([0, _log(rng, 1, 3000)]), bias=rng.choice([0, rng.randint(1, 300)]),
                mask=rng.random() < 0.5, tree=n > 1 and rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------
_QMAX = {"fp8": 448.0, "int8": 127.0}
_GROW = {"fp8": 448.0, "int8": 127.5}  # the largest |value| / scale that a page's scale is kept for


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _cuda(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _codes(x, kv):
    """Codes of x, already divided by its scale, as bytes."""
    if kv == "fp8":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _power(x):
    """The smallest power of two at or above x > 0."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.ones_like(x), torch.where(m == 0.5, e - 1, e))


def _pool(c, gen, pages):
    """One operand of a block-scaled pool [pages, P, Hkv, D] and its scales [pages, Hkv].
    Heads and pages differ in magnitude, as layers' keys and values do."""
    x = _normal(gen, pages, c["page"], c["hkv"], c["d"])
    x *= torch.exp(0.3 * _normal(gen, pages, 1, c["hkv"], 1))
    m = x.abs().amax((1, 3))
    s = _power(m / 448.0) if c["kv"] == "fp8" else m / 127.0
    return _codes(x / s[:, None, :, None], c["kv"]), s


def _token_pool(c, gen, pages):
    """A pool of the other storage types: bf16, or codes with a scale per token and head."""
    x = _normal(gen, pages, c["page"], c["hkv"], c["d"])
    if c["kv"] == "bf16":
        return x.to(torch.bfloat16), None
    kv = c["kv"].split("_")[0]
    s = x.abs().amax(-1) / _QMAX[kv]
    return _codes(x / s[..., None], kv), s.transpose(-1, -2).contiguous()


def _tables(lens, page, rng):
    """Permuted pages for sequences of these lengths."""
    need = -(-np.asarray(lens, np.int64) // page)
    total = int(need.sum())
    perm = rng.permutation(total).astype(np.int32)
    col = np.arange(max(1, int(need.max())))[None, :]
    first = (np.cumsum(need) - need)[:, None]
    table = np.where(col < need[:, None], perm[np.minimum(first + col, total - 1)], -1)
    return table.astype(np.int32), total


def _sizes(c):
    """The generator of a case's lengths: they belong to the case, not to the seed."""
    return np.random.default_rng([v for v in c.values() if isinstance(v, int) and v >= 0])


def _attend_lengths(c):
    sizes = _sizes(c)
    ql = np.where(sizes.random(c["seqs"]) < c["verify"], c["k"] + 1, 1)
    return ql, np.maximum(sizes.integers(c["lo"], c["hi"] + 1, c["seqs"]), ql)


def _append_lengths(c):
    sizes = _sizes(c)
    ql = sizes.integers(c["ql_lo"], c["ql_hi"] + 1, c["seqs"])
    return ql, ql + sizes.integers(0, c["ctx"] + 1, c["seqs"])


def _read_lengths(c):
    sizes = _sizes(c)
    return (sizes.integers(0, c["skip"] + 1, c["seqs"]), sizes.integers(c["lo"], c["hi"] + 1, c["seqs"]))


def _prepare_attend(c, rng, gen):
    ql, lens = _attend_lengths(c)
    table, pages = _tables(lens, c["page"], rng)
    T = int(ql.sum())
    s = dict(case=c, q=_normal(gen, T, c["hq"], c["d"]).to(torch.bfloat16), bt=_cuda(table),
             lens=_cuda(lens), ql=_cuda(ql), ql_max=int(ql.max()), len_max=int(lens.max()))
    s["k_pages"], s["k_scale"] = _pool(c, gen, pages)
    s["v_pages"], s["v_scale"] = _pool(c, gen, pages)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, c["hq"], device="cuda", dtype=torch.float32)
    s["ws"] = None  # the call's scratch space, from the first pass on
    return s


def _prepare_append(c, rng, gen):
    ql, lens = _append_lengths(c)
    table, pages = _tables(lens, c["page"], rng)
    T, hq, hkv, d = int(ql.sum()), c["hq"], c["hkv"], c["d"]
    qkv = _normal(gen, T, hq + 2 * hkv, d).to(torch.bfloat16)
    s = dict(case=c, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cos_sin=None,
             bt=_cuda(table), lens=_cuda(lens), ql=_cuda(ql), wq=None, wk=None,
             q_out=torch.empty(T, hq, d, device="cuda", dtype=torch.bfloat16))
    if c["rot"]:
        ang = np.arange(int(lens.max()) + 1)[:, None] * THETA ** (-np.arange(0, c["rot"], 2) / c["rot"])[None, :]
        s["cos_sin"] = _cuda(np.concatenate([np.cos(ang), np.sin(ang)], 1), torch.float32)
    if c["norm"]:
        s["wq"] = (1 + 0.2 * _normal(gen, d)).to(torch.bfloat16)
        s["wk"] = (1 + 0.2 * _normal(gen, d)).to(torch.bfloat16)
    s["k_pages"], s["k_scale"] = _pool(c, gen, pages)
    s["v_pages"], s["v_scale"] = _pool(c, gen, pages)
    return s


def _prepare_read(c, rng, gen):
    starts, lens = _read_lengths(c)
    table, pages = _tables(starts + lens, c["page"], rng)
    s = dict(case=c, bt=_cuda(table), starts=_cuda(starts), lens=_cuda(lens))
    pool = _pool if c["kv"] in _QMAX else _token_pool
    s["k_pages"], s["k_scale"] = pool(c, gen, pages)
    s["v_pages"], s["v_scale"] = pool(c, gen, pages)
    T, out = int(lens.sum()), torch.bfloat16 if c["out"] == "bf16" else torch.float32
    s["k_out"] = torch.empty(T, c["hkv"], c["d"], device="cuda", dtype=out)
    s["v_out"] = torch.empty_like(s["k_out"])
    return s


def _prepare_logits(c, rng, gen):
    B, n, V = c["seqs"], c["n"], c["vocab"]
    f32 = torch.float32
    type_ = torch.bfloat16 if c["type"] == "bf16" else f32
    # A model's logits: a few likely tokens above a broad floor.
    x = 3.0 * _normal(gen, B, n + 1, V + c["pad"])
    s = dict(case=c, logits=x.to(type_)[..., :V], out=torch.empty(B, n + 1, V, device="cuda", dtype=f32))
    del x
    likely = torch.topk(s["logits"][:, 0].float(), 50, dim=-1).indices.cpu().numpy()
    pick = lambda m: likely[np.arange(B)[:, None], rng.integers(0, 50, (B, m))]  # noqa: E731
    s["drafts"] = _cuda(pick(n)) if n else None
    s["parents"] = _cuda(np.floor(rng.random((B, n)) * np.arange(1, n + 1))) if c["tree"] else None
    for name in ("tokens", "token_lens", "prompt_lens", "repetition", "frequency", "presence",
                 "bias_tokens", "bias", "mask"):
        s[name] = None
    if c["hist"]:  # text: frequent tokens over and over, and the likely ones among them
        sizes = _sizes(c)
        H = c["hist"]
        zipf = np.minimum((V * rng.random((B, H)) ** 4).astype(np.int64), V - 1)
        s["tokens"] = _cuda(np.where(rng.random((B, H)) < 0.1, pick(H), zipf))
        lens = sizes.integers((H + 1) // 2, H + 1, B)
        s["token_lens"], s["prompt_lens"] = _cuda(lens), _cuda(lens - lens // 3)
        s["repetition"] = _cuda(rng.uniform(1.0, 1.3, B), f32)
        s["frequency"] = _cuda(rng.uniform(0.0, 0.5, B), f32)
        s["presence"] = _cuda(rng.uniform(-0.2, 0.6, B), f32)
    if c["bias"]:
        t = rng.integers(0, V, (B, c["bias"]))
        t[:, ::3] = pick(t[:, ::3].shape[1])
        t[rng.random(t.shape) < 0.1] = -1
        s["bias_tokens"], s["bias"] = _cuda(t), _cuda(rng.uniform(-5, 5, t.shape), f32)
    if c["mask"]:  # a grammar: about a third of the words allow nothing, a third anything
        w = rng.integers(-2**31, 2**31, (B, n + 1, -(-V // 32)))
        w = np.where(rng.random(w.shape) < 0.33, 0, np.where(rng.random(w.shape) < 0.5, -1, w))
        s["mask"] = _cuda(w)
    t = rng.uniform(0.5, 1.5, B)
    t[1::4] = 0.0  # one sequence in four decodes greedily
    s["temperature"] = _cuda(t, f32) if c["kind"] == "probs" else None
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "read": _prepare_read,
            "logits": _prepare_logits}[case["op"]](case, rng, gen)


# ---- the package's entry points ---------------------------------------------------------
_QUANT = {"fp8": "fp8_block", "int8": "int8_block", "fp8_token": "fp8", "int8_token": "int8", "bf16": None}


def _own(s):
    from verify_attention_spec_gb300 import binding as vas

    c = s["case"]
    if c["op"] == "logits":
        vas.spec_logits(s["logits"], s["out"], tokens=s["tokens"], token_lens=s["token_lens"],
                        prompt_lens=s["prompt_lens"], draft_tokens=s["drafts"], parents=s["parents"],
                        repetition_penalty=s["repetition"], frequency_penalty=s["frequency"],
                        presence_penalty=s["presence"], bias_tokens=s["bias_tokens"], bias=s["bias"],
                        mask=s["mask"], temperature=s["temperature"], probs=c["kind"] == "probs")
        return
    quant, scales = _QUANT[c["kv"]], dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "append":
        vas.paged_kv_append(s["q"], s["k"], s["v"], s["bt"], s["lens"], s["ql"], s["q_out"], s["k_pages"],
                            s["v_pages"], cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"],
                            interleaved=c["inter"], eps=EPS, quant=quant, **scales)
    elif c["op"] == "read":
        vas.paged_kv_read(s["k_pages"], s["v_pages"], s["bt"], s["lens"], s["k_out"], s["v_out"],
                          starts=s["starts"], quant=quant, **scales)
    else:
        dims = vas.attn_dims(s["q"], s["k_pages"], s["bt"], s["lens"], quant=quant)
        if s["ws"] is None:
            s["ws"] = vas.alloc_workspace(dims)
        vas.paged_attn_fwd_quant(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["bt"],
                                 s["lens"], s["ql"], s["out"], s["lse"], s["ws"], quant=quant, dims=dims)


# ---- the plain form -----------------------------------------------------------------------
def _token_places(s, T):
    """Sequence, cache position, page and slot of every new token."""
    seq = torch.repeat_interleave(torch.arange(s["ql"].numel(), device="cuda"), s["ql"], output_size=T)
    row0 = torch.cumsum(s["ql"], 0) - s["ql"]
    pos = (s["lens"] - s["ql"])[seq] + torch.arange(T, device="cuda") - row0[seq]
    page = s["bt"][seq, pos // s["case"]["page"]].long()
    return seq, pos, page, pos % s["case"]["page"]


def _decoded(codes, kv):
    return codes.view(torch.float8_e4m3fn if kv == "fp8" else torch.int8).float()


def _plain_attend(s):
    c = s["case"]
    B, T, hkv, d = s["ql"].numel(), s["q"].shape[0], c["hkv"], c["d"]
    g, L, Q = c["hq"] // hkv, s["len_max"], s["ql_max"]
    seq, pos, _, _ = _token_places(s, T)
    j = pos - (s["lens"] - s["ql"])[seq]
    t = torch.arange(L, device="cuda")
    page = s["bt"][:, t // c["page"]].clamp(min=0).long()
    slot = (t % c["page"])[None, :]

    def rows(pages, scales):  # [B, L, Hkv, D] in 32 bits
        return _decoded(pages[page, slot], c["kv"]).mul_(scales[page][..., None])

    q = torch.zeros(B, Q, c["hq"], d, device="cuda")
    q[seq, j] = s["q"].float()
    q = q.view(B, Q, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * Q, d)
    z = torch.matmul(q, rows(s["k_pages"], s["k_scale"]).permute(0, 2, 3, 1)) / math.sqrt(d)
    last = (s["lens"] - s["ql"])[:, None] + torch.arange(Q, device="cuda")[None, :]
    hidden = (t[None, None, :] > last[:, :, None]) | (t[None, None, :] >= s["lens"][:, None, None])
    z = z.view(B, hkv, g, Q, L).masked_fill(hidden[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    n = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, hkv, g * Q, L), rows(s["v_pages"], s["v_scale"]).permute(0, 2, 1, 3))
    o = (o.view(B, hkv, g, Q, d) / n).permute(0, 3, 1, 2, 4).reshape(B, Q, c["hq"], d)
    lse = (m + torch.log(n))[..., 0].permute(0, 3, 1, 2).reshape(B, Q, c["hq"])
    s["out"].copy_(o[seq, j])
    s["lse"].copy_(lse[seq, j])


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    a, b = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :r // 2], y[..., r // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    c = s["case"]
    kv, P = c["kv"], c["page"]
    _, pos, page, slot = _token_places(s, s["q"].shape[0])

    def head(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        if c["rot"]:
            row = s["cos_sin"][pos.long()][:, None, :]
            x = _rotate(x, row[..., :c["rot"] // 2], row[..., c["rot"] // 2:], c["inter"])
        return x

    pages = s["k_pages"].shape[0]
    first = torch.full((pages,), P, device="cuda").scatter_reduce(0, page, slot.long(), "amin")
    fresh, touched = first == 0, first < P

    def store(x, codes, scales):
        m = torch.zeros(pages, c["hkv"], device="cuda")
        m.scatter_reduce_(0, page[:, None].expand(-1, c["hkv"]), x.abs().amax(-1), "amax")
        start = m / torch.full_like(m, _QMAX[kv])
        if kv == "fp8":
            start = _power(start)
        # A page that holds tokens keeps its scale, times the power of two that the new ones need.
        need = _power(torch.maximum(m / (_GROW[kv] * scales), torch.ones_like(m)))
        grown = scales * need
        new = torch.where(fresh[:, None], start, torch.where(touched[:, None], grown, scales))
        ratio = (scales / new)[page][:, None, :, None]
        old = codes[page]  # the pages of the new tokens, once a token
        live = torch.arange(P, device="cuda")[None, :] < first[page][:, None]
        kept = _codes(_decoded(old, kv) * ratio, kv)
        codes[page] = torch.where(live[:, :, None, None], kept, old)
        codes[page, slot] = _codes(x / new[page][..., None], kv)
        scales.copy_(new)

    s["q_out"].copy_(head(s["q"], s["wq"]))
    store(head(s["k"], s["wk"]), s["k_pages"], s["k_scale"])
    store(s["v"].float(), s["v_pages"], s["v_scale"])


def _plain_read(s):
    c = s["case"]
    T = s["k_out"].shape[0]
    seq = torch.repeat_interleave(torch.arange(s["lens"].numel(), device="cuda"), s["lens"], output_size=T)
    pos = s["starts"][seq] + torch.arange(T, device="cuda") - (torch.cumsum(s["lens"], 0) - s["lens"])[seq]
    page, slot = s["bt"][seq, pos // c["page"]].long(), pos % c["page"]
    for name in ("k", "v"):
        x, sc = s[name + "_pages"][page, slot], s[name + "_scale"]
        if sc is None:
            x = x.float()
        elif sc.dim() == 2:
            x = _decoded(x, c["kv"]) * sc[page][..., None]
        else:
            x = _decoded(x, c["kv"].split("_")[0]) * sc.transpose(-1, -2)[page, slot][..., None]
        s[name + "_out"].copy_(x)


def _plain_logits(s):
    c = s["case"]
    B, n, V = c["seqs"], c["n"], c["vocab"]
    z = s["logits"].float()
    per = lambda x: x[:, None, None]  # noqa: E731
    if s["tokens"] is not None:
        at = torch.arange(s["tokens"].shape[1], device="cuda")[None, :]
        t = s["tokens"].long()
        prompt = at < s["prompt_lens"][:, None]
        given = (at < s["token_lens"][:, None]) & ~prompt
        in_prompt = torch.zeros(B, V, device="cuda").scatter_add_(1, t, prompt.float())
        count = torch.zeros(B, V, device="cuda").scatter_add_(1, t, given.float())
        count = count[:, None].repeat(1, n + 1, 1)
        if n:  # the drafts on the way to each row
            if s["parents"] is None:
                way = torch.ones(n + 1, n, device="cuda").tril(-1).expand(B, -1, -1)
            else:
                up = torch.zeros(B, n + 1, n + 1, device="cuda")
                up[:, 1:].scatter_(2, s["parents"].long()[..., None], 1.0)
                way = torch.linalg.matrix_power(up + torch.eye(n + 1, device="cuda"), n)[:, :, 1:].clamp(max=1)
            count.scatter_add_(2, s["drafts"].long()[:, None].expand(-1, n + 1, -1), way.contiguous())
        seen = (count > 0) | (in_prompt > 0)[:, None]
        r = per(s["repetition"])
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - per(s["frequency"]) * count - per(s["presence"]) * (count > 0)
    if s["bias"] is not None:
        some = s["bias_tokens"] >= 0
        add = torch.zeros(B, V, device="cuda")
        add.scatter_add_(1, s["bias_tokens"].clamp(min=0).long(), s["bias"] * some)
        z = z + add[:, None]
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        z = z.masked_fill(bits.flatten(-2)[..., :V] == 0, -math.inf)
    if c["kind"] == "probs":
        temp = per(s["temperature"])
        m = z.amax(-1, keepdim=True)
        e = torch.exp((z - m.clamp(min=-3e38)) / torch.where(temp > 0, temp, torch.ones_like(temp)))
        p = e / e.sum(-1, keepdim=True)
        best = torch.where(z == m, torch.arange(V, device="cuda"), V).amin(-1, keepdim=True)
        hot = torch.zeros_like(p).scatter_(-1, best, 1.0)
        z = torch.where(m == -math.inf, torch.zeros_like(p), torch.where(temp > 0, p, hot))
    s["out"].copy_(z)


def _outputs(s):
    op, kv = s["case"]["op"], s["case"].get("kv")
    if op == "attend":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "logits":
        return s["out"]
    type_ = torch.float8_e4m3fn if kv == "fp8" else torch.int8
    return {"q": s["q_out"], "k": s["k_pages"].view(type_), "k_scale": s["k_scale"],
            "v": s["v_pages"].view(type_), "v_scale": s["v_scale"]}


def run(state):
    if own:
        _own(state)
    else:
        {"attend": _plain_attend, "append": _plain_append, "read": _plain_read,
         "logits": _plain_logits}[state["case"]["op"]](state)
    return _outputs(state)


# ---- what a pass cannot do without ----------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "logits":
        rows = c["seqs"] * (c["n"] + 1)
        size = 2 if c["type"] == "bf16" else 4
        return {"bytes": rows * (c["vocab"] * (size + 4) + (c["vocab"] / 8 if c["mask"] else 0))
                + c["seqs"] * (4 * c["hist"] + 8 * c["bias"]),
                "flops": rows * c["vocab"] * 8}
    if c["op"] == "read":
        T = int(_read_lengths(c)[1].sum())
        of = {"bf16": 2 * c["d"], "fp8_token": c["d"] + 4, "int8_token": c["d"] + 4}
        stored = of.get(c["kv"], c["d"] + 4 / c["page"])
        return {"bytes": 2 * T * c["hkv"] * (stored + c["d"] * (2 if c["out"] == "bf16" else 4)),
                "flops": 2 * T * c["hkv"] * c["d"]}
    token = 2 * c["hkv"] * (c["d"] + 4 / c["page"])  # K and V of one cached token
    if c["op"] == "append":
        T = int(_append_lengths(c)[0].sum())
        return {"bytes": T * ((2 * c["hq"] + 2 * c["hkv"]) * c["d"] * 2 + token),
                "flops": T * (c["hq"] + c["hkv"]) * c["d"] * 7}
    ql, lens = _attend_lengths(c)
    attended = float((ql * lens - ql * (ql - 1) / 2).sum())
    return {"bytes": int(lens.sum()) * token + int(ql.sum()) * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * attended * c["hq"] * c["d"]}


# ---- the operators in 64 bits ------------------------------------------------------------------
def _exact_attend(c, s):
    """One sequence at a time, softmax in 64 bits."""
    ql, lens, table = s["ql"].tolist(), s["lens"].tolist(), s["bt"].long()
    type_ = torch.float8_e4m3fn if c["kv"] == "fp8" else torch.int8
    g, out, lse = c["hq"] // c["hkv"], [], []
    q, row = s["q"].double(), 0
    for n, L, ids in zip(ql, lens, table):
        ids = ids[:-(-L // c["page"])]

        def rows(pages, scales):
            x = pages[ids].view(type_).double() * scales[ids].double()[:, None, :, None]
            return x.reshape(-1, c["hkv"], c["d"])[:L]

        k, v = rows(s["k_pages"], s["k_scale"]), rows(s["v_pages"], s["v_scale"])
        x = q[row:row + n].view(n, c["hkv"], g, c["d"])
        z = torch.einsum("nhgd,lhd->hgnl", x, k) * c["d"] ** -0.5
        late = torch.arange(L, device="cuda")[None, :] > (L - n + torch.arange(n, device="cuda"))[:, None]
        z = z.masked_fill(late, -math.inf)
        m = torch.logsumexp(z, -1)
        o = torch.einsum("hgnl,lhd->nhgd", torch.exp(z - m[..., None]), v)
        out.append(o.reshape(n, c["hq"], c["d"]))
        lse.append(m.permute(2, 0, 1).reshape(n, c["hq"]))
        row += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_append(c, s):
    """Page by page of each sequence, in 64 bits on the host."""
    ql, lens, table = (s[x].cpu().numpy() for x in ("ql", "lens", "bt"))
    P, fp8, top = c["page"], c["kv"] == "fp8", _QMAX[c["kv"]]
    type_ = torch.float8_e4m3fn if fp8 else torch.int8
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    at = np.concatenate([np.arange(n - q, n) for n, q in zip(lens, ql)])

    def head(x, w):
        x = f64(x)
        if w is not None:
            x = x / np.sqrt(np.mean(x ** 2, -1, keepdims=True) + EPS) * f64(w)
        if not c["rot"]:
            return x
        cs, r, y = f64(s["cos_sin"])[at], c["rot"], x.copy()
        even, odd = (slice(0, r, 2), slice(1, r, 2)) if c["inter"] else (slice(0, r // 2), slice(r // 2, r))
        turned = (x[..., even] + 1j * x[..., odd]) * (cs[:, :r // 2] + 1j * cs[:, r // 2:])[:, None, :]
        y[..., even], y[..., odd] = turned.real, turned.imag
        return y

    def code(x):
        if fp8:
            return torch.from_numpy(x).float().to(type_).double().numpy()
        return np.rint(x)

    out = {"q": head(s["q"], s["wq"])}
    for name, x in (("k", head(s["k"], s["wk"])), ("v", f64(s["v"]))):
        codes, scale = f64(s[name + "_pages"].view(type_)), f64(s[name + "_scale"])
        row = 0
        for i, (n, q) in enumerate(zip(lens, ql)):
            for p in range((n - q) // P, -(-n // P)):
                lo, hi = max(n - q, p * P), min(n, (p + 1) * P)
                new, id_ = x[row + lo - (n - q):row + hi - (n - q)], table[i, p]
                m = np.abs(new).max((0, 2))
                if lo == p * P:
                    sc = 2.0 ** np.ceil(np.log2(m / top)) if fp8 else m / top
                else:
                    sc = scale[id_] * 2.0 ** np.maximum(0, np.ceil(np.log2(m / (_GROW[c["kv"]] * scale[id_]))))
                    codes[id_, :lo - p * P] = code(codes[id_, :lo - p * P] * (scale[id_] / sc)[:, None])
                codes[id_, lo - p * P:hi - p * P] = code(new / sc[:, None])
                scale[id_] = sc
            row += q
        # Whole codes next to a half have no value in 64 bits: their scales are in 32.
        out[name], out[name + "_scale"] = (codes if fp8 else None), scale
    return out


def _exact_read(c, s):
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = {"k": [], "v": []}
    for i, (a, n) in enumerate(zip(starts, lens)):
        ids = s["bt"][i, a // c["page"]:-(-(a + n) // c["page"])].long()
        off = a % c["page"]
        for name in out:
            x, sc = s[name + "_pages"][ids], s[name + "_scale"]
            if sc is not None:
                x = x.view(torch.float8_e4m3fn if c["kv"].startswith("fp8") else torch.int8)
                sc = sc[ids].double()
                sc = sc[:, None, :] if sc.dim() == 2 else sc.transpose(1, 2)
                x = x.double() * sc[..., None]
            out[name].append(x.double().reshape(-1, c["hkv"], c["d"])[off:off + n])
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_logits(c, s):
    """Row by row: the few tokens that are counted or biased, one after another, in 64 bits."""
    n, V = c["n"], c["vocab"]
    all_rows = []
    f = lambda name, b: float(s[name][b])  # noqa: E731
    for b in range(c["seqs"]):
        for j in range(n + 1):
            z = s["logits"][b, j].double().cpu().numpy()
            if s["tokens"] is not None:
                text = s["tokens"][b, :int(s["token_lens"][b])].cpu().numpy()
                before, after = text[:int(s["prompt_lens"][b])], text[int(s["prompt_lens"][b]):]
                way, u = [], j
                while u > 0:
                    way.append(int(s["drafts"][b, u - 1]))
                    u = u - 1 if s["parents"] is None else int(s["parents"][b, u - 1])
                count = np.bincount(np.concatenate([after, np.asarray(way, after.dtype)]), minlength=V)
                for x in np.union1d(before, np.flatnonzero(count)):
                    z[x] = z[x] / f("repetition", b) if z[x] > 0 else z[x] * f("repetition", b)
                    z[x] -= f("frequency", b) * count[x] + f("presence", b) * (count[x] > 0)
            if s["bias"] is not None:
                for x, y in zip(s["bias_tokens"][b].tolist(), s["bias"][b].tolist()):
                    if x >= 0:
                        z[x] += y
            if s["mask"] is not None:
                words = s["mask"][b, j].cpu().numpy().view(np.uint8)
                z[np.unpackbits(words, bitorder="little")[:V] == 0] = -np.inf
            if c["kind"] == "probs":
                if not np.isfinite(z.max()):
                    z = np.zeros(V)
                elif f("temperature", b) == 0.0:
                    z = (np.arange(V) == int(np.argmax(z))).astype(np.float64)
                else:
                    z = np.exp((z - z.max()) / f("temperature", b))
                    z /= z.sum()
            all_rows.append(z)
    return np.stack(all_rows).reshape(c["seqs"], n + 1, V)


def exact(case, seed):
    if case["op"] == "logits" and case["seqs"] * (case["n"] + 1) * (1500 + case["hist"]) > 4000000:
        return None
    return {"attend": _exact_attend, "append": _exact_append, "read": _exact_read,
            "logits": _exact_logits}[case["op"]](case, prepare(case, seed))
