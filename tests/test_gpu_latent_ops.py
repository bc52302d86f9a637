"""Rotary positions, cache append and latent attention against their definitions in 64 bits."""
import math

import pytest
import torch

from long_context_sparse_indexer_b200 import lsa

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}      # half a step, relative
E4M3 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(0, scale, generator=g)


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ rotary positions

def _turn(x, pos, r, off, backward=False):
    """(rotated x, |u| + |w| of each element's pair) in 64 bits; x [T, H, D]."""
    rd, m = r.c.rot_dim, r.c.mscale
    a = pos.double()[:, None, None] * torch.tensor(r.inv_freq, dtype=torch.float64, device=DEV)
    c, s = a.cos() * m, a.sin() * m * (-1 if backward else 1)
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    ev = torch.arange(rd // 2, device=DEV)
    i, j = (off + 2 * ev, off + 2 * ev + 1) if r.c.interleaved else (off + ev, off + rd // 2 + ev)
    u, w = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    size[..., i] = size[..., j] = (u.abs() + w.abs()) * abs(m)
    return y, size


def _rope_close(got, x, pos, r, off, backward=False):
    # One rounding to the type; in 32 bits the products, their sum, sine and cosine and the angle's reduction
    # are together within 2^-21 of |u| + |w|.
    y, size = _turn(x, pos, r, off, backward)
    assert ((got.double() - y).abs() <= HALF[x.dtype] * y.abs() + 2.0 ** -21 * size).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,off,rd", [(1, 1, 2, 0, 2), (1, 1, 64, 0, 64), (3, 5, 576, 512, 64), (70, 128, 576, 512, 64),
                                          (517, 3, 128, 0, 64), (33, 1, 100, 10, 38), (2, 64, 192, 128, 64),
                                          (5, 7, 320, 64, 256), (9, 2, 136, 8, 128), (300, 128, 128, 0, 128)])
def test_rope(cuda, dtype, inter, T, H, D, off, rd):
    g = _gen(T * 7 + D)
    x = _normal(g, T, H, D, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    r = lsa.Rope(rd, interleaved=inter, scaling="yarn", factor=32.0, mscale=1.25)
    y = torch.full_like(x, float("nan"))
    assert lsa.rope(r, pos, x, y, offset=off) is y
    _rope_close(y, x, pos, r, off)
    keep = torch.ones(D, dtype=torch.bool, device=DEV)
    keep[off:off + rd] = False
    assert torch.equal(y[..., keep], x[..., keep])
    # In place gives the same bits, and the rest of the row stays.
    z = x.clone()
    lsa.rope(r, pos, z, offset=off)
    assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_strided_views(cuda, dtype, inter):
    """The rotary slice of a wider tensor, other token and head orders, unaligned rows, a broadcast input."""
    g = _gen(5)
    r = lsa.Rope(64, interleaved=inter, scaling="linear", factor=4.0)
    pos = torch.randint(0, 4096, (6,), generator=g, device=DEV, dtype=torch.int32)
    q = _normal(g, 6, 10, 576, dtype=dtype)
    y = torch.empty(6, 10, 64, dtype=dtype, device=DEV)
    lsa.rope(r, pos, q[..., 512:], y)
    _rope_close(y, q[..., 512:], pos, r, 0)
    before = q.clone()
    lsa.rope(r, pos, q[..., 512:])                                   # in place inside the wider rows
    assert torch.equal(q[..., 512:], y) and torch.equal(q[..., :512], before[..., :512])
    hm = _normal(g, 10, 6, 64, dtype=dtype).transpose(0, 1)          # heads outermost in memory
    out = torch.empty(10, 6, 64, dtype=dtype, device=DEV).transpose(0, 1)
    lsa.rope(r, pos, hm, out)
    _rope_close(out, hm, pos, r, 0)
    odd = _normal(g, 6 * 10 * 67 + 1, dtype=dtype)[1:].view(6, 10, 67)[..., 2:66]
    out = torch.empty(6, 10, 65, dtype=dtype, device=DEV)[..., 1:]
    lsa.rope(r, pos, odd, out)
    _rope_close(out, odd, pos, r, 0)
    one = _normal(g, 1, 1, 64, dtype=dtype).expand(6, 10, 64)
    lsa.rope(r, pos, one, y)
    _rope_close(y, one, pos, r, 0)


def test_rope_far_rows(cuda):
    """Tokens 2^31 + 64 elements apart."""
    x, pos, r = _normal(_gen(8), 3, 2, 128), _ints(5, 900, 77), lsa.Rope(64)
    far = torch.empty(2 ** 32 + 4096, dtype=torch.bfloat16, device=DEV).as_strided((3, 2, 128), (2 ** 31 + 64, 128, 1))
    far.copy_(x)
    lsa.rope(r, pos, far, offset=64)
    assert torch.equal(far, lsa.rope(r, pos, x, torch.empty_like(x), offset=64))


def test_rope_far_and_negative_positions(cuda):
    """Angles at the ends of int32 keep their fraction of a turn (64 bits: 2^31 rad within 2^-21)."""
    r = lsa.Rope(64, interleaved=True)
    pos = _ints(0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789)
    x = _normal(_gen(3), 6, 4, 64, dtype=torch.float32)
    y = lsa.rope(r, pos, x, torch.empty_like(x))
    _rope_close(y, x, pos, r, 0)
    assert torch.equal(y[0], x[0])
    huge = lsa.Rope(64, theta=1e6, scaling="ntk", factor=8.0)
    y = lsa.rope(huge, pos, x, torch.empty_like(x))
    _rope_close(y, x, pos, huge, 0)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(cuda, inter):
    """backward is the adjoint: against the formula, and <y(x), g> = <x, backward(g)> by differences."""
    g = _gen(11)
    r = lsa.Rope(96, interleaved=inter, scaling="yarn", factor=8.0, mscale=1.2)
    pos = torch.randint(0, 100000, (37,), generator=g, device=DEV, dtype=torch.int32)
    x, dy, step = (_normal(g, 37, 9, 128, dtype=torch.float32) for _ in range(3))
    dx = lsa.rope(r, pos, dy, torch.empty_like(dy), offset=16, backward=True)
    _rope_close(dx, dy, pos, r, 16, backward=True)
    f = lambda v: lsa.rope(r, pos, v, torch.empty_like(v), offset=16).double()  # noqa: E731
    # The map is linear, so the difference is exact up to the roundings of f (2^-21 of |u| + |w|, random sign).
    diff = ((f(x + step) - f(x)) * dy.double()).sum()
    want = ((x + step).double() - x.double()).mul(dx.double()).sum()
    bound = 2.0 ** -20 * ((x.abs() + step.abs()) * 2).double().mul(dy.abs().double() * 2).sum() * 1.2
    assert (diff - want).abs() <= bound


# ------------------------------------------------------------------ cache append

def _append_reference(x, pos, norm, nd, gamma, beta, eps, r, off):
    """(row, error bound of its 32-bit arithmetic) in 64 bits."""
    h = x.double().clone()
    n = h[:, :nd]
    if norm == "layer":
        n = n - n.mean(1, keepdim=True)
    size = x.double().abs()
    if norm != "none":
        rs = 1 / (n.square().mean(1, keepdim=True) + eps).sqrt()
        h[:, :nd] = n * rs * (gamma.double() if gamma is not None else 1)
        top = x[:, :nd].double().abs().amax(1, keepdim=True) * rs * (gamma.abs().max().double() if gamma is not None else 1)
        if beta is not None:
            h[:, :nd] += beta.double()
            top = top + beta.abs().max().double()
        size[:, :nd] = top
    # Sums of up to 1024 terms in 32 bits (lanes, then a tree: fewer than 32 + 5 roundings each) and a handful of
    # products: within 2^-18 of the largest term.  The rotation adds 2^-21 of its pair.
    if r is not None:
        y, pair = _turn(h[:, None], pos, r, off)
        rot = size[:, off:off + r.c.rot_dim].amax(1, keepdim=True) * 2 * abs(r.c.mscale)
        size[:, off:off + r.c.rot_dim] = rot
        h = y[:, 0]
    return h, 2.0 ** -18 * size


def _check_append(data, scale, at, y, err):
    got = data[at]
    if scale is None:
        assert ((got.double() - y).abs() <= HALF[torch.bfloat16] * y.abs() + err * (1 + 2.0 ** -7)).all()
        return
    amax = y.abs().amax(1)
    s = scale[at].double()
    e = err.amax(1)
    zero = amax == 0
    assert ((s - amax / 448).abs() <= e / 448 + 2.0 ** -23 * amax / 448)[~zero].all() and (s[zero] == 1).all()
    v = got.view(E4M3).double() * s[:, None]
    # Half a step of e4m3: 2^-4 relative, 2^-10 of the scale among the subnormals.
    assert ((v - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s[:, None] + 2 * e[:, None] + err).all()


KV = dict(dim=576, norm="rms", nd=512, off=512, inter=True)
INDEX = dict(dim=128, norm="layer", nd=128, off=0, inter=False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [0, 8, 24, 64])
@pytest.mark.parametrize("kind", ["kv", "index", "plain", "wide", "small"])
@pytest.mark.parametrize("B,G", [(1, 1), (5, 3), (3, 301)])
def test_append(cuda, fp8, page, kind, B, G):
    k = {"kv": KV, "index": INDEX, "plain": dict(dim=576, norm="none", nd=576, off=0, inter=False),
         "wide": dict(dim=1024, norm="layer", nd=1016, off=740, inter=False),
         "small": dict(dim=16, norm="rms", nd=8, off=6, inter=True)}[kind]
    g = _gen(B * 1000 + G + page)
    dim, L = k["dim"], G + 37
    T = B * G
    rd = {"plain": 0, "wide": 256, "small": 8}.get(kind, 64)
    r = lsa.Rope(rd, interleaved=k["inter"], scaling="yarn", factor=8.0, mscale=1.1) if rd else None
    x = _normal(g, T, dim + 8, scale=3.0)[:, :dim]                   # rows further apart than they are wide
    gamma = 1 + 0.2 * _normal(g, k["nd"], dtype=torch.float32) if kind != "small" else None
    beta = 0.3 * _normal(g, k["nd"], dtype=torch.float32) if kind == "index" else None
    start = torch.randint(0, L - G + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    q_pos = (start[:, None] + torch.arange(G, device=DEV, dtype=torch.int32)).reshape(-1)
    q_seq = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(G)
    lead, rows, pages, at = B, L, None, (q_seq.long(), q_pos.long())
    if page:
        n = -(-L // page)
        table = torch.full((B, n + 1), -1, dtype=torch.int32, device=DEV)
        table[:, :n] = torch.randperm(B * n + 2, generator=g, device=DEV)[:B * n].view(B, n)
        pages, lead, rows = lsa.PageTable(table), B * n + 2, page
        at = (table[q_seq.long(), (q_pos // page).long()].long(), (q_pos % page).long())
    pool = torch.randint(0, 100, (lead, rows, dim + 16), generator=g, device=DEV).to(torch.uint8)
    data = pool[..., :dim] if fp8 else pool.to(torch.bfloat16)[..., :dim]
    scale = torch.full((lead, rows), 7.0, device=DEV) if fp8 else None
    before, st = data.clone(), _status()
    if kind == "plain":
        x[T // 2] = 0                                                # a row of zeros
    batch = lsa.Batch(start + G, q_seq, q_pos, L, q_group=G)
    lsa.cache_append(batch, x, lsa.Cache(data, scale), pages=pages, norm=k["norm"], norm_dim=k["nd"], gamma=gamma,
                     beta=beta, eps=1e-5, rope=r, rope_offset=k["off"], dev_status=st)
    assert lsa.read_device_status(st) == lsa.OK
    y, err = _append_reference(x, q_pos, k["norm"], k["nd"], gamma, beta, 1e-5, r, k["off"])
    _check_append(data, scale, at, y, err)
    other = torch.ones(lead, rows, dtype=torch.bool, device=DEV)
    other[at] = False
    assert torch.equal(data[other], before[other])                   # rows not named stay
    if fp8:
        assert (scale[other] == 7).all()


def test_append_padding_bad_tokens_and_bad_values(cuda):
    """Padding stores nothing; a position, sequence or page outside the batch is reported and skipped; a NaN or
    an infinity is reported and stored as NaN codes (FP8) or as it is (BF16)."""
    g = _gen(1)
    x = _normal(g, 6, 128)
    r = lsa.Rope(64)
    table = _ints(3, 1, 2, 9, 0, -1).view(2, 3)                      # a bad entry in each sequence

    def run(q_seq, q_pos, xx=x, fp8=True, pages=None, lens=(20, 20)):
        data = torch.zeros(4 if pages else 2, 8 if pages else 24, 128, device=DEV,
                           dtype=torch.uint8 if fp8 else torch.bfloat16)
        scale = torch.zeros(data.shape[:2], device=DEV) if fp8 else None
        st = _status()
        n = len(q_seq)
        lsa.cache_append(lsa.Batch(_ints(*lens), _ints(*q_seq), _ints(*q_pos), 24), xx[:n], lsa.Cache(data, scale),
                         pages=pages, rope=r, dev_status=st)
        return data, scale, lsa.read_device_status(st)
    data, scale, st = run([0, 1, 77], [3, -1, -5])
    assert st == lsa.OK and (scale != 0).sum() == 1 and scale[0, 3] > 0          # padding, its sequence not read
    for seq, pos in ((2, 0), (-1, 0), (0, 20), (1, 24), (0, 2 ** 31 - 1)):
        data, scale, st = run([0, seq], [1, pos])
        assert st == lsa.ERR_DEVICE_DATA and (scale != 0).sum() == 1
    pg = lsa.PageTable(table)
    data, scale, st = run([0, 1], [9, 15], pages=pg)
    assert st == lsa.OK and scale[1, 1] > 0 and scale[0, 7] > 0 and (scale != 0).sum() == 2
    data, scale, st = run([1, 1], [0, 8], pages=pg)                  # page 9 of 4, then page 0
    assert st == lsa.ERR_DEVICE_DATA and (scale != 0).sum() == 1 and scale[0, 0] > 0
    bad = x.clone()
    bad[0, 70], bad[1, 5] = float("nan"), float("inf")
    data, scale, st = run([0, 0, 1], [0, 1, 2], bad)
    assert st == lsa.ERR_DEVICE_DATA and (data[0, :2] == 0x7f).all() and (scale[0, :2] == 1).all()
    assert (data[1, 2] != 0x7f).all()
    data, _, st = run([0, 1], [0, 1], bad, fp8=False)
    assert st == lsa.ERR_DEVICE_DATA and data[0, 0].isnan().sum() == 1
    assert torch.equal(data[0, 0, 100:], bad[0, 100:])


def test_append_tiny_rows(cuda):
    """Rows down to the smallest BF16 subnormal, where 448 / max|row| overflows: codes as for any other row, the scale
    rounded to a 32-bit subnormal (half a step of 2^-149, times codes of at most 448)."""
    x = _normal(_gen(9), 8, 128)
    x = (x.double() * torch.tensor([2.0 ** -e for e in (30, 59, 61, 64, 100, 124, 127, 130)], device=DEV)[:, None]).to(torch.bfloat16)
    x[:, 3] = 0
    st, data = _status(), torch.zeros(1, 8, 128, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(1, 8, device=DEV)
    lsa.cache_append(lsa.Batch(_ints(8), _ints(*[0] * 8), _ints(*range(8)), 8), x, lsa.Cache(data, scale), dev_status=st)
    assert lsa.read_device_status(st) == lsa.OK
    v, y = data.view(E4M3).double()[0] * scale.double()[0, :, None], x.double()
    step = 2.0 ** -4 * y.abs() * (1 + 2.0 ** -20) + 2.0 ** -10 * scale.double()[0, :, None] + 448 * 2.0 ** -150 * (1 + 2.0 ** -4)
    assert v.isfinite().all() and ((v - y).abs() <= step).all()


def test_append_far_rows(cuda):
    """Rows more than 2^32 bytes into a pool, and sequences as far apart."""
    x, r = _normal(_gen(3), 6, 576), lsa.Rope(64, interleaved=True)
    q_seq, q_pos = _ints(0, 0, 0, 1, 1, 1), _ints(5, 6, 70, 0, 64, 99)
    for fp8 in (False, True):
        dt, n = (torch.uint8, 120000) if fp8 else (torch.bfloat16, 60000)
        run = lambda cache, pages: lsa.cache_append(lsa.Batch(_ints(100, 100), q_seq, q_pos, 100), x, cache, pages=pages,  # noqa: E731
                                                    norm="rms", norm_dim=512, rope=r, rope_offset=512)
        small = torch.zeros(2, 100, 576, dtype=dt, device=DEV)
        ss = torch.zeros(2, 100, device=DEV) if fp8 else None
        run(lsa.Cache(small, ss), None)
        want = small[q_seq.long(), q_pos.long()]
        pool = torch.empty(n, 64, 576, dtype=dt, device=DEV)
        ps = torch.zeros(n, 64, device=DEV) if fp8 else None
        table = _ints(n - 1, n - 3, n - 2, n - 9).view(2, 2)
        run(lsa.Cache(pool, ps), lsa.PageTable(table))
        at = (table[q_seq.long(), (q_pos // 64).long()].long(), (q_pos % 64).long())
        assert torch.equal(pool[at], want) and (ps is None or torch.equal(ps[at], ss[q_seq.long(), q_pos.long()]))
        far = pool.view(-1).as_strided((2, 100, 576), (pool.numel() - 100 * 576, 576, 1))
        fs = torch.zeros(2, 100, device=DEV) if fp8 else None
        run(lsa.Cache(far, fs), None)
        assert torch.equal(far[q_seq.long(), q_pos.long()], want)
        del pool, far


# ------------------------------------------------------------------ latent attention, absorbed form

def _latent_reference(q, rows, lim, sm):
    """o, lse, sum of p |v| and the largest sum of |q k| sm, in 64 bits: q [H, 576], rows [L, 576], keys < lim."""
    if lim <= 0:
        return q.new_zeros(q.shape[0], 512).double(), q.new_full((q.shape[0],), -math.inf).double(), None, 0.0
    k = rows[:lim].double()
    z = q.double() @ k.t() * sm
    p = z.softmax(-1)
    return p @ k[:, :512], z.logsumexp(-1), p @ k[:, :512].abs(), float((q.double().abs() @ k.abs().t()).max()) * sm


def _close(o, lse, ref, terms, what):
    """Scores: `terms` products summed in 32 bits, within terms * 2^-24 of sum |q k| (dz, natural-log units).  o: its
    own rounding, the BF16 rounding of each weight (2^-8 relative) and e^dz on weights and their sum."""
    ro, rl, size, qk = ref
    if size is None:
        assert (o == 0).all() and (lse is None or (lse == -math.inf).all()), what
        return
    dz = terms * 2.0 ** -24 * qk + 2.0 ** -20
    bound = HALF[o.dtype] * ro.abs() + (2.0 ** -8 * (1 + 2.0 ** -7) + 2.5 * dz) * size
    assert ((o.double() - ro).abs() <= bound).all(), (what, ((o.double() - ro).abs() / bound).max())
    if lse is not None:
        assert ((lse.double() - rl).abs() <= dz + 2.0 ** -22 * (1 + rl.abs())).all(), what


class Latent:
    """A cache of `lens` rows per sequence, paged (page > 0) or not, NaN in every row that no position names, and
    the query tokens `q_pos` (list per sequence, equal lengths)."""

    def __init__(self, seed, H, lens, q_pos, page=64, fp8=False, L=None, f32=False, scale=2.0, wide=False, bad_pages=True):
        g = _gen(seed)
        self.B, self.G, self.H, self.page, self.fp8 = len(lens), len(q_pos[0]), H, page, fp8
        self.L = L or max(max(lens), 1)
        self.lens, self.q_pos = lens, q_pos
        T, B = self.B * self.G, self.B
        n = -(-self.L // page) if page else 0
        lead, rows = (B * n + 2, page) if page else (B, self.L)
        dim = 576 + (32 if wide else 0)
        raw = _normal(g, lead, rows, 576)
        seq = torch.arange(B, device=DEV)[:, None].expand(B, self.L)
        r = torch.arange(self.L, device=DEV)[None, :].expand(B, self.L)
        self.pages, at = None, (seq, r)
        if page:
            table = torch.randperm(B * n + 2, generator=g, device=DEV)[:B * n].view(B, n).to(torch.int32)
            at = (table.long()[seq, r // page], r % page)
            if bad_pages:                                            # entries behind the last row are never read
                used = torch.tensor([-(-x // page) for x in lens], device=DEV)[:, None]
                table = torch.where(torch.arange(n, device=DEV)[None, :] < used, table, torch.full_like(table, -7))
            self.pages = lsa.PageTable(table.contiguous())
        live = torch.zeros(lead, rows, dtype=torch.bool, device=DEV)
        inside = r < torch.tensor([max(max(p) + 1, 0) for p in q_pos], device=DEV)[:, None]
        live[at[0][inside], at[1][inside]] = True
        if fp8:
            amax = raw.abs().amax(-1).float()
            sc = (amax / 448) * torch.exp2(torch.randint(-3, 4, amax.shape, generator=g, device=DEV).float())
            codes = (raw.float() * (448 / amax)[..., None]).to(E4M3).view(torch.uint8)
            codes[~live] = 0x7f
            sc[~live] = float("nan")
            self.values = codes.view(E4M3).double() * sc.double()[..., None]
            data = torch.zeros(lead, rows, dim, dtype=torch.uint8, device=DEV)
            data[..., :576] = codes
            self.cache = lsa.Cache(data[..., :576], sc)
        else:
            raw[~live] = float("nan")
            self.values = raw.double()
            data = torch.full((lead, rows, dim), float("nan"), dtype=torch.bfloat16, device=DEV)
            data[..., :576] = raw
            self.cache = lsa.Cache(data[..., :576])
        self.rows = self.values[at]                                  # [B, L, 576]
        self.q = _normal(g, T, H, 576, scale=scale)
        self.sm = 1 / 24.0
        pos = torch.tensor(q_pos, dtype=torch.int32, device=DEV).reshape(-1)
        self.batch = lsa.Batch(_ints(*lens), torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(self.G),
                               pos, self.L, q_group=self.G)
        self.o = torch.full((T, H, 512), float("nan"), device=DEV, dtype=torch.float32 if f32 else torch.bfloat16)
        self.lse = torch.full((T, H), float("nan"), device=DEV)
        self.ws = torch.full((lsa.latent_attn_workspace_size(T, self.G, H),), 0xff, dtype=torch.uint8, device=DEV)
        self.st = _status()

    def run(self, stream=None):
        lsa.latent_attn(self.batch, self.q, self.cache, self.sm, self.o, self.lse, pages=self.pages, ws=self.ws,
                        dev_status=self.st, stream=stream)

    def check(self, what="", tokens=None):
        assert lsa.read_device_status(self.st) == lsa.OK, what
        for t in tokens if tokens is not None else range(self.B * self.G):
            b = t // self.G
            ref = _latent_reference(self.q[t], self.rows[b], self.q_pos[b][t % self.G] + 1, self.sm)
            _close(self.o[t], self.lse[t], ref, 576, (what, t))


def _tail(lens, G):
    return [[n - G + i for i in range(G)] for n in lens]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [0, 8, 24, 64, 128])
@pytest.mark.parametrize("H,lens,G", [(128, [1], 1), (128, [64, 65, 1, 63], 1), (16, [300, 5, 1000], 4), (1, [129], 2),
                                      (20, [700, 33], 5), (130, [200], 3), (64, [2049, 1500], 1), (128, [515], 70),
                                      (7, [31, 97], 31)])
def test_latent(cuda, fp8, page, H, lens, G):
    s = Latent(H + len(lens) + G, H, lens, _tail(lens, G), page=page, fp8=fp8)
    s.run()
    s.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_latent_long_ragged_contexts(cuda, fp8):
    """Work cut inside sequences of very different lengths, every part joined; padding tokens and a padding
    group among them; 32-bit results."""
    lens = [40001, 3, 9000, 1, 17777, 64]
    pos = _tail(lens, 2)
    pos[1] = [-1, 2]
    pos[2] = [8999, -1]
    pos[3] = [-1, -1]
    s = Latent(9, 128, lens, pos, page=32, fp8=fp8, f32=True)
    s.run()
    s.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,H,top", [(300, 128, 60), (400, 128, 200), (150, 300, 130), (250, 128, 700)])
def test_latent_many_short_contexts(cuda, fp8, B, H, top):
    """Many units per cluster, most of them of one to a few key tiles, padding among them."""
    lens = [1 + (i * 7919) % top for i in range(B)]
    pos = [[-1] if i % 13 == 5 else [n - 1] for i, n in enumerate(lens)]
    s = Latent(B + top, H, lens, pos, page=16 if fp8 else 8 * (1 + B % 4), fp8=fp8)
    s.run()
    s.check()
    o = s.o.clone()
    s.run()
    assert torch.equal(o, s.o)


def test_latent_positions_inside_the_context(cuda):
    """Tokens in any order and not at the end; rows behind the group's last position are never used."""
    s = Latent(4, 48, [900, 400], [[700, 12, 0, 311, 699], [5, 4, 3, 2, 1]], page=40)
    s.run()
    s.check()


def test_latent_wide_rows_and_lse_optional(cuda):
    for fp8 in (False, True):
        for page in (0, 16):
            s = Latent(8, 128, [333, 77], _tail([333, 77], 2), page=page, fp8=fp8, wide=True, L=401)
            lse, s.lse = s.lse, None
            s.run()
            s.lse = lse.fill_(0)
            assert lsa.read_device_status(s.st) == lsa.OK
            o = s.o.clone()
            s.run()
            s.check()
            assert torch.equal(o, s.o)


def test_latent_peaked_and_extreme_scores(cuda):
    """Scores in the hundreds, rising along the row (the running maximum moves at every tile) and falling."""
    for sign in (1.0, -1.0):
        s = Latent(21, 128, [3000], [[2999]], page=64, scale=0.0)
        s.q[..., 0] = 24.0
        r = s.cache.data.view(-1, 576)
        ramp = torch.linspace(-400, 400, 3000, device=DEV) * sign
        table = s.pages.table[0].long()
        at = (table[torch.arange(3000, device=DEV) // 64], torch.arange(3000, device=DEV) % 64)
        s.cache.data[at[0], at[1], 0] = ramp.to(torch.bfloat16)
        s.rows = s.cache.data.double()[at][None]
        assert r.shape[1] == 576
        s.run()
        s.check()


def test_latent_every_fp8_code_and_far_scales(cuda):
    """Rows of all 254 finite codes (subnormal ones alone in some), scales from 2^-40 to 2^20, one row far above the others."""
    finite = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8, device=DEV)
    tiny = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 129, 130, 131, 132, 133, 134, 135], dtype=torch.uint8, device=DEV)
    for top, kind in ((-40, finite), (20, finite), (0, tiny), (12, tiny)):
        s = Latent(40 + top, 20, [200], [[199]], page=32, fp8=True, scale=1.0 if kind is tiny else 0.02)
        g = _gen(top + 99)
        at = (s.pages.table[0].long()[torch.arange(200, device=DEV) // 32], torch.arange(200, device=DEV) % 32)
        s.cache.data[at] = kind[torch.randint(0, len(kind), (200, 576), generator=g, device=DEV)]
        s.cache.scale[at] = torch.exp2(top - torch.rand(200, generator=g, device=DEV) * 3)
        s.sm = 2.0 ** -max(top, 0) / 24
        s.rows = (s.cache.data.view(E4M3)[at].double() * s.cache.scale[at].double()[:, None])[None]
        s.run()
        s.check(top)


def test_latent_bad_batch_is_reported(cuda):
    def run(q_seq, q_pos, lens=(30, 30), page=None):
        s = Latent(2, 16, [30, 30], [[29, 29], [29, 29]], page=16, bad_pages=False)
        if page is not None:
            s.pages.table[0, 1] = page
        s.batch = lsa.Batch(_ints(*lens), _ints(*q_seq), _ints(*q_pos), 30, q_group=2)
        s.run()
        return s, lsa.read_device_status(s.st)
    s, st = run([0, 0, 1, 1], [29, 30, 3, 3])
    assert st == lsa.ERR_DEVICE_DATA and (s.o[1] == 0).all() and (s.lse[1] == -math.inf).all() and s.o[0].isfinite().all()
    s, st = run([0, 1, 1, 1], [29, 29, 3, 3])                        # a group of two sequences
    assert st == lsa.ERR_DEVICE_DATA and (s.o[1] == 0).all() and s.o[2].abs().sum() > 0
    s, st = run([5, 5, 1, 1], [29, 29, 3, 3])
    assert st == lsa.ERR_DEVICE_DATA and (s.o[:2] == 0).all() and s.o[2].abs().sum() > 0
    s, st = run([0, 0, 1, 1], [29, 29, 3, 3], lens=(40, 30))         # longer than the cache
    assert st == lsa.ERR_DEVICE_DATA and (s.o[:2] == 0).all() and s.o[2].abs().sum() > 0
    s, st = run([0, 0, 1, 1], [29, 29, 3, 3], page=99)                 # a page outside the pool
    assert st == lsa.ERR_DEVICE_DATA and s.o.isfinite().all() and s.o[2:].abs().sum() > 0
    s, st = run([0, 0, 1, 1], [-1, -1, -1, -1])
    assert st == lsa.OK and (s.o == 0).all() and (s.lse == -math.inf).all()


def test_latent_twice_the_same_and_on_other_streams(cuda):
    """Same bits again; two calls at once on two streams with their own workspaces; captured and replayed with
    other contents and lengths."""
    s = Latent(31, 128, [5000, 700], _tail([5000, 700], 1))
    z = Latent(32, 128, [3000, 4100], _tail([3000, 4100], 1), fp8=True)
    s.run()
    z.run()
    torch.cuda.synchronize()
    so, zo = s.o.clone(), z.o.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        s.o.fill_(float("nan")), z.o.fill_(float("nan"))
        torch.cuda.synchronize()
        s.run(a)
        z.run(b)
        torch.cuda.synchronize()
        assert torch.equal(s.o, so) and torch.equal(z.o, zo)
    s.check("stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    n = Latent(33, 128, [2000, 4999], _tail([2000, 4999], 1), L=5000)
    for k in ("data",):
        s.cache.data.copy_(n.cache.data)
    s.pages.table.copy_(n.pages.table)
    s.q.copy_(n.q)
    s.batch.q_pos.copy_(n.batch.q_pos)
    s.batch.seq_len.copy_(n.batch.seq_len)
    s.rows, s.q_pos = n.rows, n.q_pos
    graph.replay()
    torch.cuda.synchronize()
    s.check("replay")


@pytest.mark.parametrize("fp8", [False, True])
def test_latent_far_rows(cuda, fp8):
    """Pages more than 2^32 bytes into their pool, and sequences as far apart."""
    s = Latent(51, 16, [300, 131], _tail([300, 131], 2), page=64, fp8=fp8)
    n = 120000 if fp8 else 60000
    pool = torch.empty(n, 64, 576, dtype=s.cache.data.dtype, device=DEV)
    lead = s.cache.data.shape[0]
    pool[n - lead:] = s.cache.data
    scale = None
    if fp8:
        scale = torch.empty(n, 64, device=DEV)
        scale[n - lead:] = s.cache.scale
    s.cache = lsa.Cache(pool, scale)
    s.pages.table[s.pages.table >= 0] += n - lead
    s.run()
    s.check("pages")
    z = Latent(52, 16, [300, 131], _tail([300, 131], 2), page=0, fp8=fp8)
    far = pool.view(-1).as_strided((2, 300, 576), (pool.numel() - 300 * 576, 576, 1))
    far.copy_(z.cache.data)
    z.cache = lsa.Cache(far, z.cache.scale)
    z.run()
    z.check("sequences")


@pytest.mark.parametrize("fp8", [False, True])
def test_latent_sequences_side_by_side_and_shared(cuda, fp8):
    """Sequences as columns of one [rows, sequences, 576] tensor, all sequences on the same rows (stride 0), and two
    sequences whose tables name the same pages."""
    s = Latent(61, 20, [200, 333], _tail([200, 333], 2), page=0, fp8=fp8)
    s.cache = lsa.Cache(s.cache.data.transpose(0, 1).contiguous().transpose(0, 1), s.cache.scale)
    s.run()
    s.check("columns")
    s = Latent(62, 20, [300, 300], [[299, 298], [70, 299]], page=0, fp8=fp8)
    s.cache = lsa.Cache(s.cache.data[1:].expand(2, -1, -1), s.cache.scale[1:].expand(2, -1) if fp8 else None)
    s.rows = s.rows[[1, 1]]
    s.run()
    s.check("shared rows")
    s = Latent(63, 20, [300, 300], [[299, 298], [70, 299]], page=64, fp8=fp8)
    s.pages.table[0, :4] = s.pages.table[1, :4]
    s.rows[0, :256] = s.rows[1, :256]
    s.run()
    s.check("shared pages")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,lens", [(20, [30000]), (128, [30000]), (200, [9000]), (128, [20000] + [50] * 40)])
def test_latent_units_of_many_parts(cuda, fp8, H, lens):
    """One context cut over the whole GPU and joined, alone and among short ones, in both output types."""
    for f32 in (False, True):
        s = Latent(70 + H, H, lens, _tail(lens, 1), fp8=fp8, f32=f32, scale=0.5)
        s.run()
        s.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,lens,G", [(128, [700, 64, 1, 2000], 1), (128, [4000], 4), (64, [65, 129, 1500, 30, 700, 64, 128, 1], 2),
                                      (128, [300 + 17 * i for i in range(33)], 1), (16, [40] * 70, 1), (128, [100, 5000] * 20, 1)])
def test_latent_units_cut_apart(cuda, fp8, H, lens, G):
    """Up to as many units as clusters, of even and uneven lengths, one token of padding among them."""
    pos = [list(p) for p in _tail([max(n, G) for n in lens], G)]
    if len(lens) > 3:
        pos[2] = [-1] * G
    s = Latent(len(lens) + H + G, H, [max(n, G) for n in lens], pos, fp8=fp8)
    s.run()
    s.check()


def test_first_calls_of_a_process_are_captured(cuda):
    """A process whose first calls are captured replays them."""
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import test_gpu_latent_ops as t
s, z, e = t.Latent(1, 128, [700], [[699]]), t.Latent(2, 16, [700], [[699]], fp8=True), t.Expanded(3, 4, [300], [400])
x, y = t._normal(t._gen(4), 5, 3, 64), torch.zeros(5, 3, 64, dtype=torch.bfloat16, device="cuda")
pos, r, starts = t._ints(0, 1, 2, 3, 4), t.lsa.Rope(64), (t._ints(0, 300), t._ints(0, 400))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    s.run(), z.run(), e.run(starts=starts)
    t.lsa.rope(r, pos, x, y)
    t.lsa.cache_append(z.batch, z.q[:1, 0], z.cache, pages=z.pages)
graph.replay()
torch.cuda.synchronize()
s.check(), e.check()
assert t.lsa.read_device_status(z.st) == t.lsa.OK and z.o.isfinite().all() and torch.equal(x[0], y[0])
"""
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_latent_matches_sparse_attention_over_every_row(cuda):
    """The sparse path given every visible row computes the same attention (contiguous BF16 cache)."""
    lens = [700, 64]
    s = Latent(6, 128, lens, _tail(lens, 1), page=0)
    s.run()
    idx = torch.full((2, 700), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens):
        idx[b, :n] = torch.arange(n, device=DEV, dtype=torch.int32)
    o, lse = torch.empty_like(s.o), torch.empty_like(s.lse)
    lsa.sparse_attn(s.batch, s.q, s.cache, idx, _ints(*lens), s.sm, o, lse, Dv=512)
    s.o, s.lse = s.o, s.lse
    s.check()
    s.o, s.lse = o, lse
    s.check("sparse")


# ------------------------------------------------------------------ latent attention, expanded form

class Expanded:
    def __init__(self, seed, H, nq, nk, causal=True, f32=False, split=False, gap=0, scale=2.0):
        g = _gen(seed)
        self.H, self.nq, self.nk, self.causal, self.sm = H, nq, nk, causal, 1 / math.sqrt(192)
        starts = lambda n, g0: [g0 + sum(n[:i]) for i in range(len(n) + 1)]  # noqa: E731
        self.qs, self.ks = starts(nq, gap), starts(nk, gap)
        T, S = sum(nq) + 2 * gap, sum(nk) + 2 * gap
        self.q = _normal(g, T, H, 192, scale=scale)
        if split:
            self.kn, self.v = _normal(g, H, S, 128).transpose(0, 1), _normal(g, S, H, 136)[..., :128]
            self.kr = _normal(g, S, 576)[:, 512:]
        else:
            kv = _normal(g, S, H, 256)
            self.kn, self.v, self.kr = kv[..., :128], kv[..., 128:], _normal(g, S, 64)
        if gap:                                                      # rows of no sequence
            for x in (self.kn, self.v, self.kr):
                x[:gap] = float("nan")
                x[S - gap:] = float("nan")
        self.o = torch.full((T, H, 128), 7.0, device=DEV, dtype=torch.float32 if f32 else torch.bfloat16)
        self.lse = torch.full((T, H), 7.0, device=DEV)
        self.st = _status()

    def run(self, max_q=None, stream=None, lse=True, starts=None):
        qs, ks = starts or (_ints(*self.qs), _ints(*self.ks))
        lsa.latent_attn_expanded(self.q, self.kn, self.kr, self.v, qs, ks,
                                 max(self.nq) if max_q is None else max_q, self.sm, self.o, self.lse if lse else None,
                                 causal=self.causal, dev_status=self.st, stream=stream)

    def check(self, what=""):
        assert lsa.read_device_status(self.st) == lsa.OK
        done = torch.zeros(self.q.shape[0], dtype=torch.bool, device=DEV)
        for b, (n, m) in enumerate(zip(self.nq, self.nk)):
            q0, k0 = self.qs[b], self.ks[b]
            done[q0:q0 + n] = True
            if n == 0:
                continue
            q = self.q[q0:q0 + n].double().transpose(0, 1)
            k = torch.cat([self.kn[k0:k0 + m], self.kr[k0:k0 + m, None].expand(m, self.H, 64)], -1).double().permute(1, 2, 0)
            v = self.v[k0:k0 + m].double().transpose(0, 1)
            z = q @ k * self.sm
            if self.causal:
                z.masked_fill_(torch.arange(m, device=DEV)[None, :] > torch.arange(n, device=DEV)[:, None] + m - n, -math.inf)
            lse = z.logsumexp(-1)
            p = (z - lse.clamp_min(-1e30)[..., None]).exp()
            qk = float((q.abs() @ k.abs()).max()) * self.sm if m else 0.0
            o, l = self.o[q0:q0 + n].transpose(0, 1), self.lse[q0:q0 + n].t()
            empty = lse == -math.inf
            assert (o[empty] == 0).all() and (l[empty] == -math.inf).all(), what
            if (~empty).any():
                ref = ((p @ v)[~empty], lse[~empty], (p @ v.abs())[~empty], qk)
                _close(o[~empty], l[~empty], ref, 192, (what, b))
        assert (self.o[~done] == 7).all() and (self.lse[~done] == 7).all(), what     # rows of no sequence


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,nk", [(1, [1], [1]), (3, [1, 1], [5, 129]), (16, [127, 128, 129, 1], [127, 128, 129, 1]),
                                     (2, [300], [300]), (4, [5, 64, 33], [700, 64, 1000]), (5, [257], [256]),
                                     (2, [40, 3], [7, 0]), (1, [513, 0, 255], [640, 9, 255]), (128, [70], [70])])
def test_expanded(cuda, causal, H, nq, nk):
    s = Expanded(H + sum(nq), H, nq, nk, causal=causal)
    s.run()
    s.check()


def test_expanded_strides_gaps_and_32_bit_results(cuda):
    """Keys with the heads outermost, values in padded rows, the rotary part a slice of a latent cache; rows of
    no sequence (NaN around the keys) left as they were; a larger max_q than needed."""
    for f32 in (False, True):
        s = Expanded(5, 6, [200, 77, 1], [333, 77, 130], split=True, gap=9, f32=f32)
        s.run(max_q=5000)
        s.check()
    s = Expanded(5, 6, [200, 77, 1], [333, 77, 130], split=True, gap=9)
    s.run(lse=False)
    s.lse.fill_(7.0)
    o = s.o.clone()
    s.run()
    s.check()
    assert torch.equal(o, s.o)


def test_expanded_far_rows(cuda):
    """Tokens 2^28 elements apart: the last ones lie more than 2^32 elements into the tensors."""
    s = Expanded(14, 2, [20], [20])
    buf = torch.empty(19 * 2 ** 28 + 8192, dtype=torch.bfloat16, device=DEV)

    def spread(t, off):
        f = buf[off:].as_strided(t.shape, (2 ** 28, *t.stride()[1:]))
        return f.copy_(t)
    s.q, s.kn, s.v, s.kr = spread(s.q, 0), spread(s.kn, 1024), spread(s.v, 2048), spread(s.kr, 4096)
    s.run()
    s.check()
    del buf


def test_expanded_extreme_scores(cuda):
    for sign in (1.0, -1.0):
        s = Expanded(2, 2, [400], [1000], scale=0.0)
        s.q[..., 190] = 24.0
        s.kr[:, 62] = (torch.linspace(-200, 200, 1000, device=DEV) * sign).to(torch.bfloat16)
        s.run()
        s.check()


def test_expanded_bad_starts_are_reported(cuda):
    for qs, ks in (([0, 5, 31], [0, 5, 30]), ([0, 5, 30], [0, 5, 31]), ([-1, 5, 30], [0, 5, 30]), ([0, 5, 30], [0, 35, 30])):
        s = Expanded(1, 2, [5, 25], [5, 25])
        s.qs, s.ks = qs, ks
        s.run()
        assert lsa.read_device_status(s.st) == lsa.ERR_DEVICE_DATA
    s = Expanded(1, 2, [5, 25], [5, 25])
    s.run(max_q=20)                                                  # shorter than the longest sequence
    assert lsa.read_device_status(s.st) == lsa.ERR_DEVICE_DATA
    assert (s.o[25:] == 7).all()


def test_expanded_merges_over_key_chunks(cuda):
    """Chunks of the keys attended apart (the newest causal, the older whole) and merged give the whole."""
    s = Expanded(12, 8, [150], [500])
    old, new = Expanded(12, 8, [150], [350], causal=False, f32=True), Expanded(12, 8, [150], [150], f32=True)
    for part, lo, hi in ((old, 0, 350), (new, 350, 500)):
        part.q, part.kn, part.v, part.kr = s.q, s.kn[lo:hi], s.v[lo:hi], s.kr[lo:hi]
        part.run()
    lsa.merge_partials(torch.stack([old.o, new.o]), torch.stack([old.lse, new.lse]), s.o, s.lse)
    s.check()


def test_expanded_streams_and_replay(cuda):
    s, z = Expanded(3, 16, [700, 5], [700, 90]), Expanded(4, 16, [333], [900])
    s.run()
    z.run()
    torch.cuda.synchronize()
    so, zo = s.o.clone(), z.o.clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    s.o.fill_(7.0), z.o.fill_(7.0)
    sst, zst = [(_ints(*x.qs), _ints(*x.ks)) for x in (s, z)]        # made before the other streams read them
    torch.cuda.synchronize()
    s.run(stream=a, starts=sst)
    z.run(stream=b, starts=zst)
    torch.cuda.synchronize()
    assert torch.equal(s.o, so) and torch.equal(z.o, zo)
    qs, ks = _ints(*s.qs), _ints(*s.ks)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsa.latent_attn_expanded(s.q, s.kn, s.kr, s.v, qs, ks, 700, s.sm, s.o, s.lse)
    s.nq, s.nk = [100, 605], [201, 589]
    s.qs, s.ks = [0, 100, 705], [0, 201, 790]
    qs.copy_(_ints(*s.qs)), ks.copy_(_ints(*s.ks))
    s.q.normal_(), s.kr.normal_()
    graph.replay()
    torch.cuda.synchronize()
    s.check("replay")


# ------------------------------------------------------------------ together

def test_prompt_then_decode_through_the_cache(cuda):
    """A prompt's rows appended and attended in both forms: with k_nope = W_k c and v = W_v c, the expanded
    attention equals the absorbed one over the cached rows with q W_k in front and W_v behind; then decode steps
    append one row each and attend to all of them."""
    g = _gen(77)
    H, L, page = 8, 150, 16
    r = lsa.Rope(64, interleaved=True, scaling="yarn", factor=8.0)
    x = _normal(g, L, 576)
    gamma = 1 + 0.1 * _normal(g, 512, dtype=torch.float32)
    n = -(-L // page)
    pool = torch.zeros(n + 2, page, 576, dtype=torch.bfloat16, device=DEV)
    pages = lsa.PageTable(torch.randperm(n + 2, generator=g, device=DEV)[:n].view(1, n).to(torch.int32))
    cache, st = lsa.Cache(pool), _status()
    wk, wv = (_normal(g, H, 128, 512, dtype=torch.float32, scale=512 ** -0.5).double() for _ in range(2))
    q = _normal(g, L, H, 192)
    pos = torch.arange(L, device=DEV, dtype=torch.int32)
    lsa.rope(r, pos, q[..., 128:])
    zero = torch.zeros(L, dtype=torch.int32, device=DEV)
    P = 140                                                          # prompt, then decode steps
    lsa.cache_append(lsa.Batch(_ints(P), zero[:P], pos[:P], L, q_group=P), x[:P], cache, pages=pages, norm="rms",
                     norm_dim=512, gamma=gamma, rope=r, rope_offset=512, dev_status=st)
    at = (pages.table[0].long()[pos.long() // page], pos.long() % page)
    rows = pool[at][:P]
    kn = torch.einsum("hdc,lc->lhd", wk, rows[:, :512].double()).bfloat16()
    v = torch.einsum("hdc,lc->lhd", wv, rows[:, :512].double()).bfloat16()
    o1 = torch.empty(P, H, 128, dtype=torch.bfloat16, device=DEV)
    lsa.latent_attn_expanded(q[:P], kn, rows[:, 512:], v, _ints(0, P), _ints(0, P), P, 192 ** -0.5, o1, dev_status=st)
    qa = torch.cat([torch.einsum("lhd,hdc->lhc", q[..., :128].double(), wk).bfloat16(), q[..., 128:]], -1).contiguous()

    def absorbed(lo, hi):
        T = hi - lo
        o = torch.empty(T, H, 512, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(lsa.latent_attn_workspace_size(T, T, H), dtype=torch.uint8, device=DEV)
        lsa.latent_attn(lsa.Batch(_ints(hi), zero[:T], pos[lo:hi].contiguous(), L, q_group=T), qa[lo:hi], cache,
                        192 ** -0.5, o, pages=pages, ws=ws, dev_status=st)
        return torch.einsum("lhc,hdc->lhd", o.double(), wv)
    o2 = absorbed(0, P)
    # BF16 roundings of q W_k, k_nope, v, the weights and the outputs, each 2^-8 relative: a few per cent at most.
    assert (o1.double() - o2).norm() <= 0.03 * o2.norm()
    for t in range(P, L):
        lsa.cache_append(lsa.Batch(_ints(t + 1), zero[:1], pos[t:t + 1], L), x[t:t + 1], cache, pages=pages, norm="rms",
                         norm_dim=512, gamma=gamma, rope=r, rope_offset=512, dev_status=st)
        o3 = absorbed(t, t + 1)
        k = pool[at][:t + 1].double()
        z = torch.einsum("hc,lc->hl", qa[t].double(), k) * 192 ** -0.5
        want = torch.einsum("hl,lc,hdc->hd", z.softmax(-1), k[:, :512], wv)
        assert (o3[0] - want).norm() <= 0.01 * want.norm()           # two BF16 roundings
    assert lsa.read_device_status(st) == lsa.OK


def test_appended_keys_feed_the_indexer_and_the_sparse_attention(cuda):
    """Appended FP8 indexer keys and latent rows drive the library's own decode: scores, top-k, sparse attention
    (every row selected) and the latent attention agree with 64-bit references over the stored values."""
    g = _gen(50)
    B, L, H, HI = 2, 300, 128, 32
    pos = torch.arange(L, device=DEV, dtype=torch.int32).repeat(B)
    seq = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(L)
    whole = lsa.Batch(_ints(L, L), seq, pos, L, q_group=L)
    ki = lsa.Cache(torch.zeros(B, L, 128, dtype=torch.uint8, device=DEV), torch.zeros(B, L, device=DEV))
    kv = lsa.Cache(torch.zeros(B, L, 576, dtype=torch.bfloat16, device=DEV))
    r, st = lsa.Rope(64), _status()
    lsa.cache_append(whole, _normal(g, B * L, 128), ki, norm="layer", rope=r, dev_status=st)
    lsa.cache_append(whole, _normal(g, B * L, 576), kv, norm="rms", norm_dim=512, rope=r, rope_offset=512, dev_status=st)
    step = lsa.Batch(_ints(L, L), _ints(0, 1), _ints(L - 1, L - 1), L)
    qi, w = _normal(g, B, HI, 128), torch.rand(B, HI, generator=g, device=DEV)
    lsa.rope(r, step.q_pos, qi)
    sc = torch.empty(B, L, device=DEV)
    lsa.index_score(step, qi, w, ki, sc, n_cols=L, dev_status=st)
    keys = ki.data.view(E4M3).double() * ki.scale.double()[..., None]
    want = (torch.einsum("bhd,bld->bhl", qi.double(), keys).relu() * w.double()[..., None]).sum(1)
    assert ((sc.double() - want).abs() <= 1e-3 * want.abs() + 1e-5 * want.abs().max()).all()
    idx, cnt = torch.empty(B, L, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    lsa.topk(step, sc, L, L, 0, 0, idx, cnt, dev_status=st)
    q = _normal(g, B, H, 576)
    o = [torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lsa.sparse_attn(step, q, kv, idx, cnt, 1 / 24, o[0], Dv=512, dev_status=st)
    ws = torch.empty(lsa.latent_attn_workspace_size(B, 1, H), dtype=torch.uint8, device=DEV)
    lsa.latent_attn(step, q, kv, 1 / 24, o[1], ws=ws, dev_status=st)
    assert lsa.read_device_status(st) == lsa.OK
    for b in range(B):
        ref = _latent_reference(q[b], kv.data[b], L, 1 / 24)
        for x in o:
            _close(x[b], None, ref, 576, b)
