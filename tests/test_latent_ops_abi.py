"""Rotary positions, cache append and latent attention without a GPU: frequencies and refused calls."""
import ctypes
import math

import pytest
import torch

from long_context_sparse_indexer_b200 import lsa


def test_frequencies_follow_their_formulas():
    r = lsa.Rope(64, theta=10000.0)
    assert r.inv_freq == pytest.approx([10000.0 ** (-2 * i / 64) for i in range(32)], rel=1e-14)
    r = lsa.Rope(8, theta=500.0, scaling="linear", factor=4.0)
    assert r.inv_freq == pytest.approx([500.0 ** (-i / 4) / 4 for i in range(4)], rel=1e-14)
    r = lsa.Rope(8, theta=500.0, scaling="ntk", factor=4.0)
    assert r.inv_freq == pytest.approx([(500.0 * 4 ** (8 / 6)) ** (-i / 4) for i in range(4)], rel=1e-14)


def test_yarn_keeps_fast_pairs_and_slows_slow_ones():
    """theta 10000, 64 dims, 4096 positions: pair(32 turns) = 10.47, pair(1 turn) = 22.5, so pairs 0..10 are
    kept, pairs 23..31 divided by the factor, and pair 15 takes (15 - 10) / 13 of the slowed frequency."""
    assert math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(10000))) == 10
    assert math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(10000))) == 23
    r = lsa.Rope(64, theta=10000.0, scaling="yarn", factor=16.0, orig_len=4096)
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert r.inv_freq[:11] == pytest.approx(plain[:11], rel=1e-14)
    assert r.inv_freq[23:] == pytest.approx([f / 16 for f in plain[23:]], rel=1e-14)
    assert r.inv_freq[15] == pytest.approx(plain[15] * (8 / 13 + 5 / 13 / 16), rel=1e-12)


def test_rope_refusals():
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=258), dict(rot_dim=64, theta=1.0),
               dict(rot_dim=64, theta=float("nan")), dict(rot_dim=64, scaling="linear", factor=0.0),
               dict(rot_dim=2, scaling="ntk", factor=2.0), dict(rot_dim=64, scaling="yarn", factor=2.0, orig_len=0),
               dict(rot_dim=64, scaling="yarn", factor=2.0, beta_fast=0.0), dict(rot_dim=64, mscale=float("inf"))):
        with pytest.raises(lsa.LsaError):
            lsa.Rope(**kw)
    with pytest.raises(ValueError):
        lsa.Rope(64, scaling="other")
    lib, r = lsa.library(), lsa.Rope(64).c

    def call(T=2, H=3, D=64, off=0, pos=16, dt=lsa.BF16, x=4096, xt=192, xh=64, y=8192, yt=192, yh=64, rr=r):
        return lib.lsa_rope_apply(ctypes.byref(rr), T, H, D, off, pos, dt, x, xt, xh, y, yt, yh, 0, None)
    assert call(T=0) == lsa.OK and call(H=0) == lsa.OK                # nothing to do, nothing launched
    assert call(off=1) == lsa.ERR_INVALID_ARG                         # rotary part beyond the row
    assert call(D=32) == lsa.ERR_INVALID_ARG
    assert call(off=-1, D=128) == lsa.ERR_INVALID_ARG
    assert call(dt=lsa.FP8_E4M3) == lsa.ERR_UNSUPPORTED
    assert call(D=8200) == lsa.ERR_UNSUPPORTED
    assert call(H=65536) == lsa.ERR_UNSUPPORTED
    assert call(T=1 << 20, H=4096) == lsa.ERR_INVALID_ARG             # rows past 31 bits
    assert call(pos=None) == lsa.ERR_INVALID_ARG
    assert call(x=None) == lsa.ERR_INVALID_ARG and call(y=None) == lsa.ERR_INVALID_ARG
    assert call(x=4097) == lsa.ERR_INVALID_ARG and call(y=8193) == lsa.ERR_INVALID_ARG
    assert call(y=4096, yt=256) == lsa.ERR_INVALID_ARG                # in place with other strides
    assert call(yh=0) == lsa.ERR_INVALID_ARG                          # rows written over one another
    bad = lsa.CRope(63, 0, 1.0, 0)
    assert call(rr=bad) == lsa.ERR_INVALID_ARG


def _batch(T=2, B=2, q_group=1, L=100):
    return lsa.CBatch(B, T, q_group, L, 16, 16, 16)        # fake device pointers: never dereferenced


def _cache(dtype=lsa.BF16, dim=576, scale=16, data=4096, rows=100, seq_stride=None):
    return lsa.CCache(data, scale if dtype == lsa.FP8_E4M3 else None, dtype, dim,
                      rows * dim if seq_stride is None else seq_stride, dim, rows)


def _pages(table=16, ld=7, n=7, page=16, n_pages=20):
    return lsa.CPages(table, ld, n, page, n_pages, 0)


BAD_PAGES = [(dict(page=0), lsa.ERR_INVALID_ARG), (dict(n_pages=0), lsa.ERR_INVALID_ARG),
             (dict(ld=6), lsa.ERR_INVALID_ARG), (dict(n=6, ld=7), lsa.ERR_INVALID_ARG),      # 96 rows < L_alloc
             (dict(table=None), lsa.ERR_INVALID_ARG), (dict(page=20), lsa.ERR_UNSUPPORTED)]


def test_append_refusals():
    lib, r = lsa.library(), lsa.Rope(64).c

    def call(b=None, c=None, x=4096, ld=576, norm=1, nd=512, g=16, be=None, eps=1e-6, rope=r, off=512, pages=None):
        b, c = b or _batch(), c or _cache()
        return lib.lsa_cache_append(ctypes.byref(b), x, ld, norm, nd, g, be, eps,
                                    ctypes.byref(rope) if rope else None, off, ctypes.byref(c),
                                    ctypes.byref(pages) if pages else None, None, None)
    assert call(b=_batch(T=0)) == lsa.OK
    assert call(c=_cache(dim=1032)) == lsa.ERR_UNSUPPORTED
    assert call(c=_cache(dim=580)) == lsa.ERR_INVALID_ARG             # rows of no whole 16 bytes
    assert call(c=_cache(dtype=lsa.FP8_E4M3, scale=None)) == lsa.ERR_INVALID_ARG
    assert call(c=_cache(data=4104)) == lsa.ERR_INVALID_ARG
    assert call(c=_cache(seq_stride=0)) == lsa.ERR_INVALID_ARG        # both sequences in the same rows
    assert call(norm=3) == lsa.ERR_UNSUPPORTED
    assert call(nd=4) == lsa.ERR_INVALID_ARG and call(nd=584) == lsa.ERR_INVALID_ARG
    assert call(nd=12) == lsa.ERR_UNSUPPORTED
    assert call(eps=-1.0) == lsa.ERR_INVALID_ARG and call(eps=float("nan")) == lsa.ERR_INVALID_ARG
    assert call(be=16) == lsa.ERR_INVALID_ARG                         # RMS norm has no beta
    assert call(off=520) == lsa.ERR_INVALID_ARG
    assert call(ld=568) == lsa.ERR_INVALID_ARG and call(ld=580) == lsa.ERR_INVALID_ARG
    assert call(x=None) == lsa.ERR_INVALID_ARG and call(x=4104) == lsa.ERR_INVALID_ARG
    assert call(b=_batch(T=65536)) == lsa.ERR_UNSUPPORTED
    for kw, want in BAD_PAGES:
        assert call(pages=_pages(**kw)) == want, kw


def test_latent_attn_refusals():
    lib = lsa.library()
    need = lsa.latent_attn_workspace_size(2, 1, 128)
    assert need > 0 and lsa.latent_attn_workspace_size(0, 1, 128) == 0

    def call(b=None, c=None, q=4096, H=128, sm=0.1, o=8192, dt=lsa.BF16, lse=None, ws=1 << 20, wsb=need, pages=None):
        b, c = b or _batch(), c or _cache()
        return lib.lsa_latent_attn(ctypes.byref(b), q, H, ctypes.byref(c), ctypes.byref(pages) if pages else None,
                                   sm, o, dt, lse, ws, wsb, None, None)
    assert call(b=_batch(T=0), ws=None, wsb=0) == lsa.OK
    assert call(b=_batch(T=3, q_group=2)) == lsa.ERR_INVALID_ARG
    assert call(c=_cache(dim=512)) == lsa.ERR_INVALID_ARG
    assert call(c=_cache(dtype=7)) == lsa.ERR_UNSUPPORTED
    assert call(H=0) == lsa.ERR_INVALID_ARG and call(H=1025) == lsa.ERR_UNSUPPORTED
    for sm in (0.0, -1.0, float("nan"), float("inf")):
        assert call(sm=sm) == lsa.ERR_INVALID_ARG
    assert call(dt=lsa.FP8_E4M3) == lsa.ERR_UNSUPPORTED
    assert call(q=None) == lsa.ERR_INVALID_ARG and call(q=4104) == lsa.ERR_INVALID_ARG
    assert call(o=None) == lsa.ERR_INVALID_ARG and call(o=8200) == lsa.ERR_INVALID_ARG
    assert call(lse=18) == lsa.ERR_INVALID_ARG
    assert call(ws=None) == lsa.ERR_WORKSPACE and call(wsb=need - 1) == lsa.ERR_WORKSPACE
    assert call(ws=(1 << 20) + 16) == lsa.ERR_WORKSPACE
    for kw, want in BAD_PAGES:
        assert call(pages=_pages(**kw)) == want, kw


def test_expanded_refusals():
    lib = lsa.library()

    def call(B=2, T=10, S=20, H=4, max_q=8, qs=16, ks=16, q=4096, qt=768, qh=192, k=4096, kt=1024, kh=256, r=4096, rt=64,
             v=4352, vt=1024, vh=256, sm=0.1, o=8192, dt=lsa.BF16, lse=None):
        return lib.lsa_latent_attn_expanded(B, T, S, H, max_q, qs, ks, q, qt, qh, k, kt, kh, r, rt, v, vt, vh, sm, 1,
                                            o, dt, lse, None, None)
    assert call(B=0) == lsa.OK and call(T=0) == lsa.OK and call(max_q=0) == lsa.OK
    for kw in (dict(B=-1), dict(T=-1), dict(S=-1), dict(H=0), dict(max_q=-1), dict(qs=None), dict(ks=None),
               dict(q=None), dict(o=None), dict(k=None), dict(r=None), dict(v=None), dict(q=4104), dict(k=4104),
               dict(r=4104), dict(v=4104), dict(o=8200), dict(lse=18), dict(qt=769), dict(kh=-256), dict(vt=1028),
               dict(sm=0.0), dict(sm=float("nan"))):
        assert call(**kw) == lsa.ERR_INVALID_ARG, kw
    for kw in (dict(B=65536), dict(H=1025), dict(dt=lsa.FP8_E4M3)):
        assert call(**kw) == lsa.ERR_UNSUPPORTED, kw


def test_binding_refuses_wrong_tensors():
    """Shapes, types and devices are refused before a pointer reaches the library (CPU tensors here)."""
    r = lsa.Rope(64)
    pos = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    for bad in (lambda: lsa.rope(r, pos, x.float().double()), lambda: lsa.rope(r, pos, x[0]),
                lambda: lsa.rope(r, pos, x, x.float()), lambda: lsa.rope(r, pos.long(), x),
                lambda: lsa.rope(r, pos[:1], x), lambda: lsa.rope(r, pos, x.transpose(1, 2)),
                lambda: lsa.rope(r, pos, x)):                            # a CPU tensor
        with pytest.raises(ValueError):
            bad()
    b = lsa.Batch(torch.ones(1, dtype=torch.int32), pos, pos, 8)
    cache = lsa.Cache(torch.zeros(1, 8, 576, dtype=torch.bfloat16))
    q, o = torch.zeros(2, 4, 576, dtype=torch.bfloat16), torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    for bad in (lambda: lsa.latent_attn(b, q[..., :512], cache, 0.1, o), lambda: lsa.latent_attn(b, q, cache, 0.1, q),
                lambda: lsa.latent_attn(b, q, cache, 0.1, o),
                lambda: lsa.latent_attn(b, q, lsa.Cache(cache.data[:, :4]), 0.1, o),
                lambda: lsa.cache_append(b, q[:, 0, :512], cache), lambda: lsa.cache_append(b, q[:, 0], cache, norm="x"),
                lambda: lsa.cache_append(b, q[:, 0], cache, norm="rms", norm_dim=512, gamma=torch.ones(576)),
                lambda: lsa.cache_append(b, q[:, 0], cache, pages=lsa.PageTable(torch.zeros(1, 1)))):
        with pytest.raises(ValueError):
            bad()
    k, v, kr = torch.zeros(5, 4, 128).bfloat16(), torch.zeros(5, 4, 128).bfloat16(), torch.zeros(5, 64).bfloat16()
    qe, st = torch.zeros(2, 4, 192).bfloat16(), torch.zeros(2, dtype=torch.int32)
    oe = torch.zeros(2, 4, 128).bfloat16()
    for bad in (lambda: lsa.latent_attn_expanded(qe, k[:4], kr, v, st, st, 2, 0.1, oe),
                lambda: lsa.latent_attn_expanded(qe.float(), k, kr, v, st, st, 2, 0.1, oe),
                lambda: lsa.latent_attn_expanded(qe, k, kr, v, st, st.long(), 2, 0.1, oe),
                lambda: lsa.latent_attn_expanded(qe, k, kr, v, st, st, 2, 0.1, oe)):
        with pytest.raises(ValueError):
            bad()
