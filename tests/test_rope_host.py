"""Refusals of fa_rope, fa_rope_bwd, fa_kv_append_rope, fa_kv_plan_positions and fa_fwd_paged_chunk, which are made on
the host before anything touches a GPU, and the phases, which are computed there.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import rope_util as ru

A = [1 << (20 + 2 * i) for i in range(16)]  # harmless fake device addresses, far apart
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where nothing is launched")


# ------------------------------------------------------------------ phases
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, span=4096), dict(scaling="yarn", factor=2.0, span=50, fast=8.0, slow=2.0)])
def test_phases(rot, kw):
    """Phases are the frequencies in turns: the angles at far positions agree with the definition's.  A double's
    frequency is off by a few steps of 2^-53 of itself, and so is its angle."""
    phases, amplitude = fa.fa_rope_phases(rot, device="cpu", **kw)
    f, a = ru.frequencies(rot, **kw)
    assert phases.dtype == torch.int64 and phases.shape == (rot // 2,)
    assert amplitude == np.float32(a)
    for pos in (0, 1, 77, 100_003, 2 ** 31 - 1, -5):
        turns = [(int(p) % 2 ** 64) * pos % 2 ** 64 / 2.0 ** 64 for p in phases.tolist()]
        want = [pos * x / (2 * math.pi) for x in f]
        off = [(t - w + 0.5) % 1.0 - 0.5 for t, w in zip(turns, want)]
        assert all(abs(o) <= 2.0 ** -48 * abs(pos) * x + 2.0 ** -50 * abs(w) + abs(pos) * 2.0 ** -63 for o, x, w in zip(off, f, want)), (pos, off)


def test_phases_of_given_frequencies():
    f = [0.0, 1.0, -0.25, 2 * math.pi, 7.0] + [0.01 * i for i in range(3)]
    phases, amplitude = fa.fa_rope_phases(16, frequencies=f, device="cpu")
    turns = [int(p) % 2 ** 64 / 2.0 ** 64 for p in phases.tolist()]
    assert amplitude == 1.0
    assert all(abs((t - x / (2 * math.pi) + 0.5) % 1.0 - 0.5) < 1e-15 for t, x in zip(turns, f))
    half, _ = fa.fa_rope_phases(16, frequencies=f, scaling="linear", factor=2.0, device="cpu")
    assert abs(int(half[1]) - int(phases[1]) // 2) <= 1024


def test_phases_refusals():
    for kw in (dict(rot_dim=15), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=32, scaling="ntk", factor=2.0, frequencies=[1.0] * 16),
               dict(rot_dim=32, base=1.0), dict(rot_dim=32, base=math.nan), dict(rot_dim=32, scaling="linear", factor=0.5),
               dict(rot_dim=32, scaling="yarn", factor=2.0), dict(rot_dim=32, scaling="yarn", factor=2.0, span=100, fast=1.0, slow=2.0),
               dict(rot_dim=32, frequencies=[math.inf] * 16)):
        with pytest.raises(fa.FAError):
            fa.fa_rope_phases(device="cpu", **kw)
    with pytest.raises(ValueError):
        fa.fa_rope_phases(32, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        fa.fa_rope_phases(32, frequencies=[1.0], device="cpu")
    out, amp = (ctypes.c_ulonglong * 8)(), ctypes.c_float()
    call = fa.lib().fa_rope_phases
    assert call(None, ctypes.byref(amp), 16, 1e4, 0, 1, 0, 0, 0, None) == fa.FA_ERR_NULLPTR
    assert call(out, None, 16, 1e4, 0, 1, 0, 0, 0, None) == fa.FA_ERR_NULLPTR
    assert call(out, ctypes.byref(amp), 16, 1e4, 4, 1, 0, 0, 0, None) == fa.FA_ERR_BAD_SHAPE


# -------------------------------------------------------------------- rope
def rope(ptrs=None, B=2, S=10, Hq=4, Hk=2, D=64, rot=32, strides="packed", pos_stride=0, inter=0, amplitude=1.0, bwd=False):
    p = list(A[:6]) if ptrs is None else ptrs  # q, k, q_out, k_out, positions, phases
    if strides == "packed":
        strides = [x for H in (Hq, Hk, Hq, Hk) for x in (H * S * D, H * D, D)]
    return (fa.fa_rope_bwd_raw if bwd else fa.fa_rope_raw)(*p, B, S, Hq, Hk, D, rot, strides, pos_stride, inter, amplitude, 0)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_pointers(bwd):
    for i in range(6):
        p = list(A[:6])
        if i != 4:  # positions may be NULL
            p[i] = 0
            assert rope(p, bwd=bwd) == fa.FA_ERR_NULLPTR, i
        p[i] = A[i] + 2
        assert rope(p, bwd=bwd) == fa.FA_ERR_MISALIGNED, i
        if i not in (4,):
            p[i] = A[i] + 4
            assert rope(p, bwd=bwd) == fa.FA_ERR_MISALIGNED, i
    assert rope(strides=None, bwd=bwd) == fa.FA_ERR_NULLPTR


@pytest.mark.parametrize("kw", [dict(B=0), dict(S=0), dict(Hq=0), dict(Hk=-1), dict(Hq=65536), dict(B=1 << 16, S=1 << 15), dict(rot=0), dict(rot=8),
                                dict(rot=40), dict(rot=80), dict(rot=-16), dict(inter=2), dict(inter=-1), dict(pos_stride=-1), dict(pos_stride=9)])
def test_rope_shapes(kw):
    assert rope(**kw) == fa.FA_ERR_BAD_SHAPE


def test_rope_other_refusals():
    for D in (0, 32, 96, 256):
        assert rope(D=D, rot=16) == fa.FA_ERR_UNSUPPORTED_D
    for a in (0.0, -1.0, math.nan, math.inf):
        assert rope(amplitude=a) == fa.FA_ERR_BAD_SCALE
    ok = [2560, 256, 64, 1280, 128, 64] * 2
    for i, x in ((0, 2561), (4, -8), (2, 1 << 40), (7, 252)):
        s = list(ok)
        s[i] = x
        assert rope(strides=s) == fa.FA_ERR_BAD_SHAPE, (i, x)
    for i, x in ((7, 64), (8, 32), (6, 256), (6, 0), (8, 0)):  # outputs whose elements meet
        s = list(ok)
        s[i] = x
        assert rope(strides=s) == fa.FA_ERR_BAD_SHAPE, (i, x)


def test_rope_aliases():
    def at(**kw):
        names = ("q", "k", "q_out", "k_out", "positions", "phases")
        p = list(A[:6])
        for n, x in kw.items():
            p[names.index(n)] = x
        return p

    assert rope(at(q_out=A[0] + 16)) == fa.FA_ERR_ALIAS          # not quite in place
    assert rope(at(q_out=A[1])) == fa.FA_ERR_ALIAS               # over k
    assert rope(at(k_out=A[2] + 128)) == fa.FA_ERR_ALIAS         # over the other output
    assert rope(at(q_out=A[4] - 64)) == fa.FA_ERR_ALIAS          # over positions
    assert rope(at(k_out=A[5] - 64)) == fa.FA_ERR_ALIAS          # over phases
    # in place with other strides
    s = [2560, 256, 64, 1280, 128, 64, 2560, 64, 640, 1280, 128, 64]
    assert rope(at(q_out=A[0]), strides=s) == fa.FA_ERR_ALIAS
    # columns of one fused tensor, but overlapping ones
    fused = [6400, 640, 64] * 4
    assert rope(at(q=A[0], k=A[0] + 2 * 256, q_out=A[2], k_out=A[2] + 2 * 192), strides=fused) == fa.FA_ERR_ALIAS
    assert rope(at(q=A[0], k=A[0] + 2 * 256, q_out=A[2], k_out=A[2] + 2 * 576), strides=fused) == fa.FA_ERR_ALIAS  # into the next row


@no_gpu
def test_rope_valid_calls_without_gpu_report_cuda_error():
    assert rope() == fa.FA_ERR_CUDA and rope(bwd=True) == fa.FA_ERR_CUDA
    p = list(A[:6])
    p[1] = p[3] = p[4] = 0
    assert rope(p, Hk=0) == fa.FA_ERR_CUDA
    p = [A[0], A[1], A[0], A[1], 0, A[5]]
    assert rope(p) == fa.FA_ERR_CUDA                              # in place
    fused = [6400, 640, 64] * 4
    for S, B in ((10, 2), (1, 2), (10, 1), (1, 1)):
        p = [A[0], A[0] + 2 * 256, A[2], A[2] + 2 * 256, 0, A[5]]
        assert rope(p, strides=fused, S=S, B=B) == fa.FA_ERR_CUDA, (S, B)
        p = [A[0], A[0] + 2 * 256, A[0], A[0] + 2 * 256, 0, A[5]]
        assert rope(p, strides=fused, S=S, B=B) == fa.FA_ERR_CUDA, (S, B)
    p = [A[0], A[1], A[2], A[2] + 128 * 3, 0, A[5]]               # heads of one row, k's behind q's
    assert rope(p, Hq=3, Hk=1, B=1, S=1, strides=[0, 0, 64] * 4) == fa.FA_ERR_CUDA


# --------------------------------------------- append with rotation, positions, chunks
def append(ptrs=None, T=16, Hkv=2, Hq=4, D=64, rot=32, inter=0, amplitude=1.0, strides=(128, 128, 256, 256), num_pages=4, page=16):
    p = list(A[:13]) if ptrs is None else ptrs
    return fa.fa_kv_append_rope_raw(*p, T, Hkv, Hq, D, rot, inter, amplitude, *strides, num_pages, page, 0)


def plan(ptrs=None, B=4, T=16, max_pages=8, num_free=8, num_pages=32, page=64):
    p = list(A[:10]) if ptrs is None else ptrs
    return fa.fa_kv_plan_positions_raw(*p, B, T, max_pages, num_free, num_pages, page, 0)


def chunk(ptrs=None, B=2, T=2, Hq=4, Hkv=2, D=64, scale=0.125, qs=256, max_pages=8, num_pages=4, page=16, ws=1 << 50, ws_bytes=1 << 40):
    p = list(A[:10]) if ptrs is None else ptrs
    return fa.fa_fwd_paged_chunk_raw(*p, B, T, Hq, Hkv, D, scale, qs, max_pages, num_pages, page, ws, ws_bytes, 0)


@pytest.mark.parametrize("call,n,wide", [(plan, 10, ()), (append, 13, (0, 1, 3, 5, 6, 9, 11, 12)), (chunk, 10, (0, 4, 5, 8))])
def test_null_and_misaligned_pointers(call, n, wide):
    for i in range(n):
        p = list(A[:n])
        p[i] = 0
        assert call(p) == fa.FA_ERR_NULLPTR, i  # of an optional pair, one without the other
        p[i] = A[i] + 2
        assert call(p) == fa.FA_ERR_MISALIGNED, i
    for i in wide:
        p = list(A[:n])
        p[i] = A[i] + 4
        assert call(p) == fa.FA_ERR_MISALIGNED, i


@pytest.mark.parametrize("call", [plan, append, chunk])
@pytest.mark.parametrize("page", [0, 8, 24, 256, -16])
def test_page_sizes(call, page):
    assert call(page=page) == fa.FA_ERR_BAD_PAGE


@pytest.mark.parametrize("call,kw", [
    (plan, dict(B=0)), (plan, dict(B=8193)), (plan, dict(T=0)), (plan, dict(num_free=0)), (plan, dict(T=2 ** 30 + 1)),
    (append, dict(T=0)), (append, dict(T=2 ** 30 + 1)), (append, dict(Hkv=0)), (append, dict(Hkv=1025)), (append, dict(Hq=3)), (append, dict(Hq=0)),
    (append, dict(Hq=65536)), (append, dict(rot=0)), (append, dict(rot=20)), (append, dict(rot=80)), (append, dict(inter=3)),
    (append, dict(strides=(120, 128, 256, 256))), (append, dict(strides=(128, 132, 256, 256))), (append, dict(strides=(128, 128, 248, 256))),
    (append, dict(strides=(128, 128, 256, 255))), (append, dict(num_pages=1 << 27)),
    (chunk, dict(Hq=3)), (chunk, dict(B=0)), (chunk, dict(T=0)), (chunk, dict(qs=255)), (chunk, dict(Hkv=0)), (chunk, dict(max_pages=0)),
    (chunk, dict(T=2 ** 30 + 1, Hq=1, Hkv=1)), (chunk, dict(T=1 << 25, Hq=64, Hkv=1, qs=4096)), (chunk, dict(B=8193)),
    (chunk, dict(max_pages=(2 ** 31 - 1) // 16 - 63))])
def test_bad_shapes(call, kw):
    assert call(**kw) == fa.FA_ERR_BAD_SHAPE


def test_head_dims_scales_and_amplitudes():
    for D in (0, 32, 96, 256):
        assert append(D=D, rot=16) == fa.FA_ERR_UNSUPPORTED_D and chunk(D=D) == fa.FA_ERR_UNSUPPORTED_D
    for x in (math.nan, math.inf, 0.0, -0.5):
        assert append(amplitude=x) == fa.FA_ERR_BAD_SCALE and chunk(scale=x) == fa.FA_ERR_BAD_SCALE
    assert chunk(scale=3e38) == fa.FA_ERR_BAD_SCALE


def test_chunk_workspace():
    need = fa.fa_fwd_paged_chunk_workspace_bytes(2, 2, 4, 2, 64)
    assert need > 0
    assert chunk(ws=0) == fa.FA_ERR_WORKSPACE and chunk(ws=(1 << 50) + 8) == fa.FA_ERR_WORKSPACE and chunk(ws_bytes=need - 1) == fa.FA_ERR_WORKSPACE
    for bad in ((0, 2, 4, 2, 64), (2, 2, 3, 2, 64), (2, 2, 4, 2, 96), (2, 0, 4, 2, 64), (2, 2 ** 30 + 1, 1, 1, 64), (2, 1 << 30, 2, 1, 64)):
        assert fa.fa_fwd_paged_chunk_workspace_bytes(*bad) == 0


def test_aliases():
    p = list(A[:10])
    p[8] = p[0]  # positions over cached_lens
    assert plan(p) == fa.FA_ERR_ALIAS
    p = list(A[:10])
    p[8] = p[7]  # and over the slots
    assert plan(p) == fa.FA_ERR_ALIAS
    for i, x in ((5, A[6]), (0, A[5] + 16), (2, A[5] + 16), (11, A[5] + 16), (12, A[6] + 16), (12, A[0]), (12, A[11] + 16), (12, A[2] - 32)):
        p = list(A[:13])
        p[i] = x
        assert append(p) == fa.FA_ERR_ALIAS, (i, x)
    p = list(A[:10])
    p[8] = p[0]
    assert chunk(p) == fa.FA_ERR_ALIAS and chunk(ws=A[4]) == fa.FA_ERR_ALIAS


@no_gpu
def test_valid_calls_without_gpu_report_cuda_error():
    assert plan() == append() == chunk() == fa.FA_ERR_CUDA
    p = list(A[:13])
    p[9] = p[10] = p[11] = p[12] = None  # no means, no queries
    assert append(p, Hq=0, strides=(128, 128, 0, 0)) == fa.FA_ERR_CUDA
    p = list(A[:13])
    p[11], p[0], p[1] = A[0], A[0] + 2 * 256, A[0] + 2 * 384  # columns of one fused tensor; queries in place
    p[12] = p[11]
    assert append(p, strides=(512, 512, 512, 512)) == fa.FA_ERR_CUDA
    p[12] = A[0] + 2 * 128
    assert append(p, strides=(512, 512, 512, 512)) == fa.FA_ERR_ALIAS


def test_wrappers_reject_what_does_not_fit():
    i = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2)
    ph = torch.zeros(16, dtype=torch.int64)
    with pytest.raises(ValueError):
        fa.fa_rope(q, q.clone(), ph)
    with pytest.raises(ValueError):
        fa.fa_rope_bwd(q, None, ph)
    with pytest.raises(ValueError):
        fa.fa_kv_append_rope(q, q, i, ph, i, c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        fa.fa_fwd_paged_chunk(q, i, i[:3], torch.zeros(3, 2, dtype=torch.int32), c, c.clone(), s, s.clone())
