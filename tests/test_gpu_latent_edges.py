"""Rotation, cache append and latent attention where a call's meaning has an edge: values that are not finite, rows marked
bad, pages that share their rows, joined results, prompts of very different lengths, waits that run out."""
import math
import time

import pytest
import torch

from long_context_sparse_indexer_b200 import lsa

from .test_gpu_latent_ops import DEV, Expanded, Latent, _close, _gen, _ints, _latent_reference, _normal, _status, _tail

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


# ------------------------------------------------------------------ queries that are not finite

# What a query row holds: one NaN; one infinity (scores of both signs); an infinity against a key dimension of one
# sign, so that every score is -inf or every score +inf.  The softmax is NaN for each.
QUERIES = ["nan", "inf", "all_minus", "all_plus"]


def _spoil(row, kind):
    if kind in ("nan", "inf"):
        row[5] = NAN if kind == "nan" else INF
    else:
        row[-1] = INF if kind == "all_minus" else -INF


@pytest.mark.parametrize("kind", QUERIES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,lens,G,f32", [(128, [700, 64, 1], 1, False), (16, [300, 40], 4, True), (128, [30000], 1, False),
                                          (64, [20000], 2, True), (128, [4000 + 7 * i for i in range(12)], 1, True)])
def test_latent_query_that_is_not_finite(cuda, kind, fp8, H, lens, G, f32):
    """o and lse of its row are NaN, in one run or joined from many; every other row keeps its bits; padding stays zero."""
    pos = _tail(lens, G)
    if G > 1:
        pos[0][0] = -1                                               # padding, spoiled too
    s = Latent(H + len(lens), H, lens, pos, fp8=fp8, f32=f32, scale=0.5)
    s.cache.data[..., 575] = 0xb8 if fp8 else -1.0                   # e4m3 -1
    s.run()
    o, lse = s.o.clone(), s.lse.clone()
    assert o.isfinite().all()
    T = len(lens) * G
    rows = sorted({(0, 0), (0, H - 1), (T - 1, H // 2), (T // 2, H // 3)})
    for t, h in rows:
        _spoil(s.q[t, h], kind)
    s.run()
    assert lsa.read_device_status(s.st) == lsa.OK
    for t, h in rows:
        if pos[t // G][t % G] < 0:
            continue
        assert s.o[t, h].isnan().all() and s.lse[t, h].isnan(), (t, h)
        s.o[t, h], s.lse[t, h] = o[t, h], lse[t, h]
    assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("kind", QUERIES)
@pytest.mark.parametrize("causal,f32", [(True, False), (False, True)])
def test_expanded_query_that_is_not_finite(cuda, kind, causal, f32):
    """As above; a query that sees no key gives zero and -inf whatever it holds."""
    s = Expanded(8, 3, [300, 40], [500, 7], causal=causal, f32=f32)
    s.kr[:, 63] = -1.0
    s.run()
    o, lse = s.o.clone(), s.lse.clone()
    rows = [(0, 0), (130, 2), (299, 1), (300, 0), (339, 2)]          # 300: 33 keys short of its first, when causal
    for t, h in rows:
        _spoil(s.q[t, h], kind)
    s.run()
    assert lsa.read_device_status(s.st) == lsa.OK
    for t, h in rows:
        if causal and t == 300:
            assert (s.o[t, h] == 0).all() and s.lse[t, h] == -INF
            continue
        assert s.o[t, h].isnan().all() and s.lse[t, h].isnan(), (t, h)
        s.o[t, h], s.lse[t, h] = o[t, h], lse[t, h]
    assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


# ------------------------------------------------------------------ joined results

@pytest.mark.parametrize("R", [1, 3, 30, 40])
def test_merge_of_parts_that_are_not_finite(cuda, R):
    """A part whose lse is NaN makes the joined o and lse NaN, alone or among others; the other rows keep their bits."""
    g = _gen(R)
    o_parts, l_parts = _normal(g, R, 2, 5, 512, dtype=torch.float32), _normal(g, R, 2, 5, dtype=torch.float32)
    o, lse = torch.empty(2, 5, 512, dtype=torch.bfloat16, device=DEV), torch.empty(2, 5, device=DEV)
    lsa.merge_partials(o_parts, l_parts, o, lse)
    want, wl = o.clone(), lse.clone()
    for p, t, h in ((R - 1, 0, 1), (0, 1, 4)):
        o_parts[p, t, h], l_parts[p, t, h] = NAN, NAN
    o_parts[:, 1, 2], l_parts[:, 1, 2] = NAN, NAN                    # every part
    lsa.merge_partials(o_parts, l_parts, o, lse)
    for t, h in ((0, 1), (1, 4), (1, 2)):
        assert o[t, h].isnan().all() and lse[t, h].isnan(), (t, h)
        o[t, h], lse[t, h] = want[t, h], wl[t, h]
    assert torch.equal(o, want) and torch.equal(lse, wl)


# ------------------------------------------------------------------ rows marked bad

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("G", [1, 3])
def test_tokens_that_see_a_bad_row(cuda, fp8, bad, G):
    """A row that the append reports (a NaN or an infinity in it) makes the attention of every token that sees it NaN;
    tokens of groups that end before it are not touched."""
    g = _gen(17)
    L, H, at = 300, 20, 130
    data = torch.zeros(1, L, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    cache, st = lsa.Cache(data, torch.zeros(1, L, device=DEV) if fp8 else None), _status()
    x = _normal(g, L, 576)
    x[at, 7] = bad
    pos = torch.arange(L, device=DEV, dtype=torch.int32)
    zero = torch.zeros(L, dtype=torch.int32, device=DEV)
    lsa.cache_append(lsa.Batch(_ints(L), zero, pos, L), x, cache, dev_status=st)
    assert lsa.read_device_status(st) == lsa.ERR_DEVICE_DATA
    T = 8 * G
    p = torch.tensor([4, 77, 120, at - 1, at, at + 1, 200, L - 1], device=DEV, dtype=torch.int32)
    p = (p[:, None] - torch.arange(G, device=DEV, dtype=torch.int32).flip(0)).reshape(-1).contiguous()
    q = _normal(g, T, H, 576)
    q[..., 7] = q[..., 7].abs() + 0.5                                # the infinity's score is +inf
    o, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, device=DEV)
    ws, st = torch.empty(lsa.latent_attn_workspace_size(T, G, H), dtype=torch.uint8, device=DEV), _status()
    lsa.latent_attn(lsa.Batch(_ints(L), zero[:T], p, L, q_group=G), q, cache, 1 / 24, o, lse, ws=ws, dev_status=st)
    assert lsa.read_device_status(st) == lsa.OK
    rows = data[0].view(torch.float8_e4m3fn).double() * cache.scale[0].double()[:, None] if fp8 else data[0].double()
    for t in range(T):
        if int(p[t]) >= at:
            assert o[t].isnan().all() and lse[t].isnan().all(), t
        elif fp8 or int(p[t // G * G + G - 1]) < at:
            _close(o[t], lse[t], _latent_reference(q[t], rows, int(p[t]) + 1, 1 / 24), 576, t)


# ------------------------------------------------------------------ pages that share their rows

@pytest.mark.parametrize("fp8", [False, True])
def test_latent_pages_on_the_same_rows(cuda, fp8):
    """A pool whose pages all lie on one page's rows (stride 0): every page holds those rows."""
    s = Latent(64, 20, [300, 131], _tail([300, 131], 2), page=64, fp8=fp8, bad_pages=False)
    lead = s.cache.data.shape[0]
    one = _normal(_gen(65), 1, 64, 576)
    scale = None
    if fp8:
        one = (one.float() * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.full((1, 64), 1 / 64, device=DEV).expand(lead, -1)
    s.cache = lsa.Cache(one.expand(lead, -1, -1), scale)
    rows = one[0].view(torch.float8_e4m3fn).double() / 64 if fp8 else one[0].double()
    s.rows = rows.repeat(5, 1)[None, :300].expand(2, -1, -1)
    s.run()
    s.check()


# ------------------------------------------------------------------ sequences without keys, and of very different lengths

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("f32", [False, True])
def test_expanded_without_any_key(cuda, causal, f32):
    """No key in the call at all (S = 0): zero and -inf for every query, rows of no sequence left as they were."""
    s = Expanded(9, 5, [3, 0, 300], [0, 0, 0], causal=causal, f32=f32)
    s.run()
    s.check()
    assert (s.o == 0).all() and (s.lse == -INF).all()
    s = Expanded(9, 1, [1], [0], causal=causal, f32=f32)
    s.run()
    s.check()
    assert (s.o == 0).all() and (s.lse == -INF).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,nk", [(2, [2500] + [1 + 37 * i % 100 for i in range(40)], [2500] + [1 + 37 * i % 100 for i in range(40)]),
                                     (20, [1, 900, 3, 1, 64], [3000, 900, 3, 1, 2000])])
def test_expanded_prompts_of_very_different_lengths(cuda, causal, H, nq, nk):
    """One long prompt among many short ones: most places of the longest have no counterpart in the others."""
    s = Expanded(H + len(nq), H, nq, nk, causal=causal)
    s.run()
    s.check()


# ------------------------------------------------------------------ a wait that runs out

@pytest.mark.parametrize("H,nq,nk", [(16, [700, 300, 1, 130], [1900, 350, 1, 130]),      # many key tiles, the last of each partial
                                     (128, [100, 40, 129], [100, 90, 257]),              # one to three, several items a CTA
                                     (64, [256, 512], [256, 512])])                      # no partial tile
def test_expanded_gives_up_and_the_context_stays_usable(cuda, H, nq, nk):
    """With a limit of 1 ns the loading warps give up: the status says so, the launch ends at once (nothing is waited for
    that cannot come: such a wait would sit out its 2 s), and the next one gives the same bits as before."""
    s = Expanded(H, H, nq, nk)
    s.run()
    s.check()
    o, lse = s.o.clone(), s.lse.clone()
    gave_up = 0
    prev = lsa.set_wait_limit_ns(1)
    try:
        for _ in range(5):
            s.st.zero_()
            torch.cuda.synchronize()
            t0 = time.monotonic()
            s.run()
            torch.cuda.synchronize()
            assert time.monotonic() - t0 < 1.0
            status = lsa.read_device_status(s.st)
            assert status in (lsa.OK, lsa.ERR_TIMEOUT), lsa.status_string(status)
            gave_up += status == lsa.ERR_TIMEOUT
    finally:
        lsa.set_wait_limit_ns(prev)
    assert gave_up
    for _ in range(2):
        s.st.zero_()
        s.o.fill_(7.0), s.lse.fill_(7.0)
        s.run()
        s.check()
        assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


# ------------------------------------------------------------------ positions behind a sequence's length

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("entry", [3, -9, 99])
def test_append_behind_the_length_stores_nothing(cuda, fp8, entry):
    """A position behind its sequence's length, whatever the page table holds there (a page of the pool or not): reported,
    no row stored; the tokens beside it are."""
    table = _ints(0, 1, entry, entry).view(1, 4)
    data = torch.zeros(5, 8, 128, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    scale = torch.zeros(5, 8, device=DEV) if fp8 else None
    st = _status()
    x = _normal(_gen(5), 4, 128)
    lsa.cache_append(lsa.Batch(_ints(12), _ints(0, 0, 0, 0), _ints(11, 12, 16, 31), 32), x, lsa.Cache(data, scale),
                     pages=lsa.PageTable(table), dev_status=st)
    assert lsa.read_device_status(st) == lsa.ERR_DEVICE_DATA
    assert data[1, 3].any() and data.flatten(2).any(-1).sum() == 1
    assert scale is None or (scale != 0).sum() == 1


# ------------------------------------------------------------------ one context over shards

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,L,cuts,G", [(128, 5000, [0, 1700, 1701, 5000], 1), (16, 700, [0, 64, 690, 700], 4), (40, 900, [0, 900], 2)])
def test_latent_merges_over_shards(cuda, fp8, H, L, cuts, G):
    """Rows of one context in several caches: 32-bit results over each, merged, are the attention over all of them.  A token
    that lies before a shard is padding there."""
    s = Latent(H + L, H, [L], _tail([L], G), page=0, fp8=fp8)
    n = len(cuts) - 1
    o, lse = torch.empty(n, G, H, 512, device=DEV), torch.empty(n, G, H, device=DEV)
    st = _status()
    for i, (a, e) in enumerate(zip(cuts, cuts[1:])):
        cache = lsa.Cache(s.cache.data[:, a:e], s.cache.scale[:, a:e] if fp8 else None)
        pos = torch.where(s.batch.q_pos < a, -1, s.batch.q_pos.clamp(max=e - 1) - a).to(torch.int32)
        lsa.latent_attn(lsa.Batch(_ints(e - a), s.batch.q_seq, pos, e - a, q_group=G), s.q, cache, s.sm, o[i], lse[i], ws=s.ws,
                        dev_status=st)
    assert lsa.read_device_status(st) == lsa.OK
    lsa.merge_partials(o, lse, s.o, s.lse)
    s.check()


# ------------------------------------------------------------------ many short segments

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,B,top", [(96, 86, 12000), (128, 300, 100), (16, 90, 700)])
def test_latent_segments_of_one_to_a_few_tiles_again_and_again(cuda, fp8, H, B, top):
    """Contexts from one row up, several a CTA: every wait comes to its end whatever the warps' pace (status OK), the same
    bits each time."""
    g = torch.Generator().manual_seed(B)
    lens = [max(1, int(math.exp(float(torch.rand(1, generator=g)) * math.log(top)))) for _ in range(B)]
    pos = [[-1] if i % 11 == 3 else [n - 1] for i, n in enumerate(lens)]
    s = Latent(B, H, lens, pos, page=8, fp8=fp8)
    s.run()
    s.check()
    o, lse = s.o.clone(), s.lse.clone()
    for _ in range(200):
        s.run()
    assert lsa.read_device_status(s.st) == lsa.OK
    assert torch.equal(s.o, o) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("f32", [False, True])
def test_latent_segments_of_one_then_two_tiles(cuda, f32):
    """FP8, runs of segments of 3, 9, 1, 1, 2, 1, 1, 1, 2 key tiles and the like, at which the scales once ran ahead of the
    products and the call timed out."""
    tiles = [90, 1, 1, 13, 1, 2, 2, 86, 14, 1, 36, 12, 1, 1, 1, 1, 17, 17, 142, 10, 3, 1, 7, 10, 1, 2, 1, 1, 1, 1, 1, 2, 2, 68, 1,
             14, 1, 45, 1, 2, 12, 3, 1, 37, 1, 80, 1, 2, 1, 1, 18, 2, 12, 1, 140, 9, 1, 1, 2, 1, 1, 1, 140, 181, 2, 1, 1, 33, 1, 1, 2,
             1, 5, 1, 2, 3, 1, 31, 2, 132, 99, 1, 1, 6]
    lens = [64 * n - (i * 13) % 64 for i, n in enumerate(tiles)]
    s = Latent(7, 96, lens, _tail(lens, 1), page=8, fp8=True, f32=f32, wide=True)
    for _ in range(100):
        s.run()
    s.check()
