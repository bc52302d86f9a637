"""The operators around a latent (MLA) KV cache: their plain forms, and the calls a user makes of the library.

Four operators, in the order in which a step of a latent-attention model runs them:

``rope``      rotary positions of query heads: pairs in the half or the interleaved layout, a part of each
              head, frequencies scaled for long contexts; backward is the rotation by the negative angle.
``append``    new rows into a cache: normalise the leading dimensions (RMS or layer norm), rotate the rotary
              part, round to BF16 or to FP8 with one scale per row, store at the token's row, through a page
              table or not.
``latent``    attention of each sequence's newest tokens over its cached latent rows (absorbed form: all heads
              read one 576-wide row per key, its first 512 dimensions being the value), causal, paged or not.
``expanded``  attention of whole prompts or chunks in the expanded form: 128 + 64 wide keys (the 64 rotary
              dimensions shared by the heads), 128 wide values, ragged sequences packed one after another.
"""
import math

import torch

own = False

LATENT, ROT, DV, NOPE = 512, 64, 512, 128
KV_DIM = LATENT + ROT
INDEX_DIM = 128
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step of 32 sequences far into a long context: the rotary part of 128 absorbed query heads.
        dict(name="rope_decode", op="rope", T=32, H=128, D=576, off=512, rd=64, inter=True, scaling="yarn",
             pos=131072, back=False, dtype="bf16"),
        # A prompt chunk's indexer queries: 64 heads, the first half of each head rotated, the rest copied.
        dict(name="rope_prompt", op="rope", T=8192, H=64, D=128, off=0, rd=64, inter=False, scaling="none",
             pos=32768, back=False, dtype="bf16"),
        # The gradient of a rotation, in FP32, odd token count and head count.
        dict(name="rope_gradient", op="rope", T=1021, H=37, D=192, off=128, rd=64, inter=True, scaling="linear",
             pos=1048576, back=True, dtype="f32"),
        # One decode step: 32 new latent rows, normalised and rotated, into an FP8 paged cache.
        dict(name="append_decode_fp8", op="append", kind="kv", B=32, G=1, ctx=1024, page=64, fp8=True),
        # The prompts of four sequences: their latent rows into a BF16 paged cache.
        dict(name="append_prompt_bf16", op="append", kind="kv", B=4, G=8191, ctx=8192, page=64, fp8=False),
        # The same prompts' indexer keys (layer norm, half-layout rotation) into a contiguous FP8 cache.
        dict(name="append_index_keys", op="append", kind="index", B=4, G=8191, ctx=8192, page=0, fp8=True),
        # A single request's decode step over a short context: latency counts.
        dict(name="latent_single", op="latent", B=1, G=1, H=128, ctx=1000, page=64, fp8=False),
        # Batched decode at 32K-64K per sequence, paged BF16 cache.
        dict(name="latent_decode_bf16", op="latent", B=32, G=1, H=128, ctx=65536, page=64, fp8=False),
        # Four verify tokens of eight sequences at up to 64K, 16 heads on this device, FP8 cache.
        dict(name="latent_verify_fp8", op="latent", B=8, G=4, H=16, ctx=65536, page=32, fp8=True),
        # A 500-token chunk of one prompt behind 15K cached rows (chunked prompt processing over pages).
        dict(name="latent_chunk_bf16", op="latent", B=1, G=500, H=128, ctx=16000, page=16, fp8=False),
        # Short prompts of odd lengths packed together, a few heads each.
        dict(name="expanded_ragged", op="expanded", B=7, Lq=301, prefix=0, H=16, causal=True),
        # A chunk of 2048 queries behind as many earlier keys, 128 heads.
        dict(name="expanded_chunk", op="expanded", B=1, Lq=2048, prefix=2048, H=128, causal=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "latent", "latent", "expanded", "expanded"])
    if op == "rope":
        rd = rng.choice([32, 64, 64, 96, 128])
        off = rng.choice([0, 64, 128, 512])
        D = off + rd + rng.choice([0, 0, 64])
        H = _log(rng, 1, 128)
        T = _log(rng, 1, max(1, min(16384, 8192 * 64 * 128 // (H * D))))
        return dict(op=op, T=T, H=H, D=D, off=off, rd=rd, inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), pos=_log(rng, T, 1048576),
                    back=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        B = _log(rng, 1, 64)
        G = _log(rng, 1, 32764 // B)
        return dict(op=op, kind=rng.choice(["kv", "kv", "index"]), B=B, G=G, ctx=G + _log(rng, 1, 4096),
                    page=rng.choice([0, 16, 32, 64, 128]), fp8=rng.random() < 0.5)
    if op == "latent":
        H = rng.choice([8, 16, 20, 32, 64, 128])
        G = rng.choice([1, 1, 1, 2, 4, 5, _log(rng, 8, 512)])
        B = _log(rng, 1, 48 if G <= 5 else 4)
        top = 500 * 16000 * 128 // (B * G * H)
        ctx = _log(rng, G, max(G, min(131072, top, 2097152 // B)))
        return dict(op=op, B=B, G=G, H=H, ctx=ctx, page=rng.choice([0, 16, 32, 64, 64, 128]), fp8=rng.random() < 0.5)
    H = _log(rng, 1, 128)
    B = _log(rng, 1, 8)
    Lq = _log(rng, 1, 2048 // B)
    prefix = rng.choice([0, 0, _log(rng, 1, 2048 // B)])
    return dict(op=op, B=B, Lq=Lq, prefix=prefix, H=H, causal=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs

ROPE_KINDS = {
    "none": dict(theta=10000.0, scaling="none"),
    "linear": dict(theta=10000.0, scaling="linear", factor=8.0),
    "ntk": dict(theta=10000.0, scaling="ntk", factor=4.0),
    "yarn": dict(theta=10000.0, scaling="yarn", factor=32.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0,
                 mscale=0.1 * math.log(32.0) + 1.0),
}


def _lib():
    from long_context_sparse_indexer_b200 import lsa
    return lsa


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"rope": _prepare_rope, "append": _prepare_append, "latent": _prepare_latent,
            "expanded": _prepare_expanded}[case["op"]](case, g)


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, scale, generator=g)


def _integers(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _prepare_rope(c, g):
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    x = _normal(g, c["T"], c["H"], c["D"], dtype=dt)
    start = _integers(g, 0, max(1, c["pos"] - c["T"] + 1), 1)
    # A prompt's positions follow one another; a decode batch's are all over the context.
    pos = start + torch.arange(c["T"], device="cuda", dtype=torch.int32) if c["T"] > 64 else \
        _integers(g, 0, c["pos"], c["T"])
    s = dict(case=c, x=x, pos=pos, y=torch.empty_like(x))
    if own:
        s["rope"] = _lib().Rope(c["rd"], interleaved=c["inter"], **ROPE_KINDS[c["scaling"]])
    return s


def _pages(c, g, B, rows):
    """A page table of every sequence's pages in a random order ([B, pages per sequence], or None), and the
    cache's leading shape (pages or sequences, rows in each)."""
    if not c["page"]:
        return None, (B, rows)
    n = (rows + c["page"] - 1) // c["page"]
    order = torch.randperm(B * n + 3, generator=g, device="cuda")[:B * n]
    return order.to(torch.int32).view(B, n), (B * n + 3, c["page"])


def _batch(c, seq_len, q_pos, rows):
    B, G = c["B"], c["G"]
    q_seq = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(G)
    s = dict(seq_len=seq_len, q_seq=q_seq, q_pos=q_pos.reshape(-1).contiguous())
    if own:
        s["batch"] = _lib().Batch(s["seq_len"], s["q_seq"], s["q_pos"], rows, q_group=G)
    return s


def _prepare_append(c, g):
    B, G, ctx = c["B"], c["G"], c["ctx"]
    kv = c["kind"] == "kv"
    dim = KV_DIM if kv else INDEX_DIM
    table, lead = _pages(c, g, B, ctx)
    start = _integers(g, 0, ctx - G + 1, B)
    q_pos = start[:, None] + torch.arange(G, device="cuda", dtype=torch.int32)
    s = dict(case=c, table=table, dim=dim, norm_dim=LATENT if kv else INDEX_DIM, off=LATENT if kv else 0, inter=kv)
    s["x"] = _normal(g, B * G, dim, scale=1.5)
    s["gamma"] = 1.0 + 0.1 * _normal(g, s["norm_dim"], dtype=torch.float32)
    s["beta"] = None if kv else 0.1 * _normal(g, s["norm_dim"], dtype=torch.float32)
    if c["fp8"]:
        s["data"] = torch.zeros(*lead, dim, device="cuda", dtype=torch.uint8)
        s["scale"] = torch.ones(*lead, device="cuda")
    else:
        s["data"], s["scale"] = torch.zeros(*lead, dim, device="cuda", dtype=torch.bfloat16), None
    s.update(_batch(c, start + G, q_pos, ctx))
    if own:
        lsa = _lib()
        s["rope"] = lsa.Rope(ROT, interleaved=s["inter"], **ROPE_KINDS["yarn"])
        s["cache"] = lsa.Cache(s["data"], s["scale"])
        s["pages"] = None if table is None else lsa.PageTable(table)
    return s


def _prepare_latent(c, g):
    B, G, H, ctx = c["B"], c["G"], c["H"], c["ctx"]
    table, lead = _pages(c, g, B, ctx)
    # Contexts between half and the whole of `ctx`, the last G positions being the new tokens'.
    seq_len = _integers(g, max(G, ctx // 2), ctx + 1, B)
    q_pos = seq_len[:, None] - G + torch.arange(G, device="cuda", dtype=torch.int32)
    rows = _normal(g, *lead, KV_DIM)
    s = dict(case=c, table=table, scale=None)
    if c["fp8"]:
        amax = rows.abs().amax(-1).float().clamp_min(1e-6)
        s["scale"] = amax / E4M3_MAX
        s["data"] = (rows.float() * (E4M3_MAX / amax)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["data"] = rows
    s["q"] = _normal(g, B * G, H, KV_DIM, scale=2.0)
    s["sm"] = 1.0 / math.sqrt(KV_DIM)
    s["o"] = torch.empty(B * G, H, DV, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty(B * G, H, device="cuda")
    s.update(_batch(c, seq_len, q_pos, ctx))
    if own:
        lsa = _lib()
        s["cache"] = lsa.Cache(s["data"], s["scale"])
        s["pages"] = None if table is None else lsa.PageTable(table)
        s["ws"] = torch.empty(lsa.latent_attn_workspace_size(B * G, G, H), dtype=torch.uint8, device="cuda")
    return s


def _prepare_expanded(c, g):
    B, Lq, H = c["B"], c["Lq"], c["H"]
    # Queries per sequence between a half and the whole of Lq, and as many keys more as the prefix has.
    nq = [Lq - (i * 37) % (Lq // 2 + 1) for i in range(B)]
    nk = [n + c["prefix"] for n in nq]
    starts = lambda n: torch.tensor([sum(n[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    T, S = sum(nq), sum(nk)
    # Keys and values come side by side from one projection of the latent rows.
    kv = _normal(g, S, H, NOPE + NOPE)
    return dict(case=c, nq=nq, nk=nk, q_start=starts(nq), k_start=starts(nk), q=_normal(g, T, H, NOPE + ROT, scale=2.0),
                k_nope=kv[..., :NOPE], v=kv[..., NOPE:], k_rope=_normal(g, S, ROT), sm=1.0 / math.sqrt(NOPE + ROT),
                o=torch.empty(T, H, NOPE, device="cuda", dtype=torch.bfloat16), lse=torch.empty(T, H, device="cuda"))


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "latent": _own_latent,
                "expanded": _own_expanded}[c["op"]](state)
    return {"rope": _plain_rope, "append": _plain_append, "latent": _plain_latent,
            "expanded": _plain_expanded}[c["op"]](state)


def _own_rope(s):
    c = s["case"]
    _lib().rope(s["rope"], s["pos"], s["x"], s["y"], offset=c["off"], backward=c["back"])
    return s["y"]


def _own_append(s):
    _lib().cache_append(s["batch"], s["x"], s["cache"], pages=s["pages"], norm="rms" if s["beta"] is None else "layer",
                        norm_dim=s["norm_dim"], gamma=s["gamma"], beta=s["beta"], eps=EPS, rope=s["rope"],
                        rope_offset=s["off"])
    return _cache_values(s)


def _cache_values(s):
    if s["scale"] is None:
        return s["data"]
    return {"codes": s["data"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _own_latent(s):
    _lib().latent_attn(s["batch"], s["q"], s["cache"], s["sm"], s["o"], s["lse"], pages=s["pages"], ws=s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_expanded(s):
    _lib().latent_attn_expanded(s["q"], s["k_nope"], s["k_rope"], s["v"], s["q_start"], s["k_start"], max(s["nq"]),
                                s["sm"], s["o"], s["lse"], causal=s["case"]["causal"])
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms

def _frequencies(rd, kind):
    """Angle per position of each pair, in 64 bits, and the factor on the rotated values."""
    k = ROPE_KINDS[kind]
    theta, i = k["theta"], torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    if kind == "ntk":
        theta = theta * k["factor"] ** (rd / (rd - 2.0))
    f = theta ** (-2.0 * i / rd)
    if kind == "linear":
        f = f / k["factor"]
    if kind == "yarn":
        # Pairs that turn more than beta_fast times over the original length keep their frequency, those that
        # turn fewer than beta_slow times are slowed by the factor, with a linear ramp over the pairs between.
        pair = lambda turns: rd * math.log(k["orig_len"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(pair(k["beta_fast"]))), min(rd - 1, math.ceil(pair(k["beta_slow"])))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f / k["factor"] * ramp + f * (1.0 - ramp)
    return f, k.get("mscale", 1.0)


def _rotate(x, pos, rd, off, inter, kind, back=False):
    """x [T, ..., D] in 32 bits with dimensions [off, off + rd) rotated by each row's position."""
    f, m = _frequencies(rd, kind)
    a = pos.double()[:, None] * f
    cos, sin = (a.cos() * m).float(), (a.sin() * m).float()
    if back:
        sin = -sin
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (rd // 2,)
    cos, sin = cos.view(shape), sin.view(shape)
    r = x[..., off:off + rd]
    if inter:
        u, w = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([x[..., :off], r, x[..., off + rd:]], -1)


def _plain_rope(s):
    c = s["case"]
    return _rotate(s["x"].float(), s["pos"], c["rd"], c["off"], c["inter"], c["scaling"], c["back"]).to(s["x"].dtype)


def _rows_of(s, seq, row):
    """(page or sequence, row in it) of each sequence's row."""
    if s["table"] is None:
        return seq.long(), row.long()
    p = s["case"]["page"]
    return s["table"][seq.long(), (row // p).long()].long(), (row % p).long()


def _plain_append(s):
    x, n = s["x"].float(), s["norm_dim"]
    h = x[:, :n]
    if s["beta"] is None:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"]
    else:
        h = h - h.mean(-1, keepdim=True)
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"] + s["beta"]
    y = _rotate(torch.cat([h, x[:, n:]], -1), s["q_pos"], ROT, s["off"], s["inter"], "yarn")
    at = _rows_of(s, s["q_seq"], s["q_pos"])
    if s["scale"] is None:
        s["data"][at] = y.to(torch.bfloat16)
    else:
        amax = y.abs().amax(-1)
        s["scale"][at] = amax / E4M3_MAX
        s["data"][at] = (y * (E4M3_MAX / amax)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return _cache_values(s)


def _cached_rows(s, n):
    """Rows 0..n-1 of every sequence's cache, in 32 bits: [B, n, 576]."""
    B = s["case"]["B"]
    seq = torch.arange(B, device="cuda")[:, None].expand(B, n)
    at = _rows_of(s, seq, torch.arange(n, device="cuda")[None, :].expand(B, n))
    if s["scale"] is None:
        return s["data"][at].float()
    return s["data"].view(torch.float8_e4m3fn)[at].float() * s["scale"][at][..., None]


def _softmax_of(z):
    """Unnormalised weights, their sums and the log-sum-exp of scores whose masked entries are -inf."""
    m = z.amax(-1, keepdim=True)
    e = (z - m.clamp_min(-3e38)).exp()
    l = e.sum(-1, keepdim=True)
    return e, l, (m + l.log()).squeeze(-1)


def _plain_latent(s):
    c = s["case"]
    B, G, H, n = c["B"], c["G"], c["H"], c["ctx"]
    k = _cached_rows(s, n)
    z = (s["q"].float().view(B, G * H, KV_DIM) @ k.transpose(1, 2)).view(B, G, H, n) * s["sm"]
    seen = torch.arange(n, device="cuda") <= s["q_pos"].view(B, G, 1, 1)
    e, l, lse = _softmax_of(z.masked_fill_(~seen, -math.inf))
    o = (e.view(B, G * H, n) @ k[..., :DV]).view(B * G, H, DV) / l.view(B * G, H, 1)
    return {"o": o.to(torch.bfloat16), "lse": lse.view(B * G, H)}


def _plain_expanded(s):
    c = s["case"]
    seq_of = lambda n: torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))  # noqa: E731
    q, seq_q, seq_k = s["q"].float(), seq_of(s["nq"]), seq_of(s["nk"])
    z = q[..., :NOPE].transpose(0, 1) @ s["k_nope"].float().permute(1, 2, 0)
    z = (z + q[..., NOPE:].transpose(0, 1) @ s["k_rope"].float().t()) * s["sm"]
    seen = seq_q[:, None] == seq_k[None, :]
    if c["causal"]:
        # The last query of a sequence sees its last key.
        iq = torch.arange(len(seq_q), device="cuda") - s["q_start"][seq_q] + c["prefix"]
        seen &= (torch.arange(len(seq_k), device="cuda") - s["k_start"][seq_k])[None, :] <= iq[:, None]
    e, l, lse = _softmax_of(z.masked_fill_(~seen, -math.inf))
    o = (e @ s["v"].float().transpose(0, 1)) / l
    return {"o": o.transpose(0, 1).contiguous().to(torch.bfloat16), "lse": lse.t().contiguous()}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * c["D"] * (2 if c["dtype"] == "bf16" else 4) + 4 * c["T"], "flops": 3 * n * c["rd"]}
    if c["op"] == "append":
        n, d = c["B"] * c["G"], KV_DIM if c["kind"] == "kv" else INDEX_DIM
        return {"bytes": n * (2 * d + (d + 4 if c["fp8"] else 2 * d) + 12), "flops": 8 * n * d}
    if c["op"] == "latent":
        # Contexts average three quarters of ctx; each of the G tokens sees all but the ones after it.
        keys, T = c["B"] * 0.75 * c["ctx"], c["B"] * c["G"]
        pairs = T * c["H"] * max(0.75 * c["ctx"] - (c["G"] - 1) / 2.0, 1.0)
        return {"bytes": keys * (KV_DIM + 4 if c["fp8"] else 2 * KV_DIM) + T * c["H"] * (2 * KV_DIM + 2 * DV + 4),
                "flops": pairs * 2 * (KV_DIM + DV)}
    nq = [c["Lq"] - (i * 37) % (c["Lq"] // 2 + 1) for i in range(c["B"])]
    pairs = sum(n * (n + c["prefix"]) - (n * (n - 1) / 2.0 if c["causal"] else 0) for n in nq) * c["H"]
    T, S = sum(nq), sum(nq) + c["B"] * c["prefix"]
    return {"bytes": T * c["H"] * (2 * (NOPE + ROT) + 2 * NOPE + 4) + S * (c["H"] * 4 * NOPE + 2 * ROT),
            "flops": pairs * 2 * (2 * NOPE + ROT)}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "latent": _exact_latent,
            "expanded": _exact_expanded}[case["op"]](case, prepare(case, seed))


def _angles(pos, rd, kind):
    """[T, rd / 2] complex factors mscale * exp(i * angle), pair by pair."""
    k = ROPE_KINDS[kind]
    freq = []
    for j in range(rd // 2):
        base = k["theta"] * (k["factor"] ** (rd / (rd - 2.0)) if kind == "ntk" else 1.0)
        w = math.exp(-2.0 * j / rd * math.log(base))
        if kind == "linear":
            w /= k["factor"]
        if kind == "yarn":
            at = [rd / 2.0 * math.log(k["orig_len"] / (2.0 * math.pi * b), base) for b in (k["beta_fast"], k["beta_slow"])]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
            t = min(1.0, max(0.0, (j - lo) / max(hi - lo, 1e-3)))
            w = w * (1.0 - t + t / k["factor"])
        freq.append(w)
    a = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    return torch.polar(torch.full_like(a, k.get("mscale", 1.0)), a)


def _turned(x, turn, off, inter):
    """x [T, n, D] in 64 bits with the rotary dimensions multiplied, as complex pairs, by turn [T, rd / 2]."""
    half = turn.shape[1]
    r = x[:, :, off:off + 2 * half]
    r = r.reshape(*r.shape[:2], half, 2) if inter else r.reshape(*r.shape[:2], 2, half).transpose(2, 3)
    z = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn[:, None, :])
    y = x.clone()
    y[:, :, off:off + 2 * half] = (z if inter else z.transpose(2, 3)).reshape(*z.shape[:2], 2 * half)
    return y


def _exact_rope(c, s):
    turn = _angles(s["pos"], c["rd"], c["scaling"])
    return _turned(s["x"].double(), turn.conj().resolve_conj() if c["back"] else turn, c["off"], c["inter"])


def _exact_append(c, s):
    x = s["x"].double()
    n = s["norm_dim"]
    centre = 0.0 if s["beta"] is None else x[:, :n].mean(1, keepdim=True)
    power = ((x[:, :n] - centre) ** 2).sum(1, keepdim=True) / n
    x[:, :n] = (x[:, :n] - centre) / (power + EPS).sqrt() * s["gamma"].double()
    if s["beta"] is not None:
        x[:, :n] += s["beta"].double()
    y = _turned(x[:, None, :], _angles(s["q_pos"], ROT, "yarn"), s["off"], s["inter"])[:, 0]
    b, r = s["q_seq"].long(), s["q_pos"].long()
    if s["table"] is not None:
        b, r = s["table"].long()[b, r // c["page"]], r % c["page"]
    data = torch.zeros(s["data"].shape, dtype=torch.float64, device="cuda")
    if s["scale"] is None:
        data[b, r] = y
        return data
    scale = s["scale"].double()
    scale[b, r] = y.abs().amax(1) / E4M3_MAX
    data[b, r] = y / scale[b, r][:, None]
    return {"codes": data, "scale": scale}


def _exact_latent(c, s):
    G, H = c["G"], c["H"]
    o = torch.zeros(c["B"] * G, H, DV, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["B"] * G, H, dtype=torch.float64, device="cuda")
    lens = s["seq_len"].tolist()
    for b in range(c["B"]):
        rows = torch.arange(lens[b], device="cuda")
        at = (torch.full_like(rows, b), rows) if s["table"] is None else \
            (s["table"][b].long()[rows // c["page"]], rows % c["page"])
        k = s["data"][at].double() if s["scale"] is None else \
            s["data"].view(torch.float8_e4m3fn)[at].double() * s["scale"].double()[at][:, None]
        for t0 in range(b * G, (b + 1) * G, 32):
            t1 = min(t0 + 32, (b + 1) * G)
            z = torch.einsum("thd,ld->thl", s["q"][t0:t1].double(), k) * s["sm"]
            z.masked_fill_(rows[None, None, :] > s["q_pos"][t0:t1, None, None], -math.inf)
            lse[t0:t1] = torch.logsumexp(z, -1)
            o[t0:t1] = torch.einsum("thl,ld->thd", torch.exp(z - lse[t0:t1, :, None]), k[:, :DV])
    return {"o": o, "lse": lse}


def _exact_expanded(c, s):
    T, H = s["q"].shape[:2]
    o = torch.zeros(T, H, NOPE, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    t0 = s0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        kr = s["k_rope"][s0:s0 + nk].double()
        hidden = torch.arange(nk, device="cuda")[None, :] > torch.arange(nq, device="cuda")[:, None] + nk - nq
        for h in range(H):
            q = s["q"][t0:t0 + nq, h].double()
            z = torch.cat([s["k_nope"][s0:s0 + nk, h].double(), kr], 1)
            z = q @ z.t() * s["sm"]
            if c["causal"]:
                z.masked_fill_(hidden, -math.inf)
            lse[t0:t0 + nq, h] = torch.logsumexp(z, 1)
            o[t0:t0 + nq, h] = torch.softmax(z, 1) @ s["v"][s0:s0 + nk, h].double()
        t0, s0 = t0 + nq, s0 + nk
    return {"o": o, "lse": lse}
