"""The paged cache's entry points reject bad arguments on the host before they touch
the GPU, the plain implementations that the GPU tests compare with hold their own
pins, and the Python wrappers check what they are given.  No GPU needed."""
import math

import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import paged_util as pu

A = [1 << (20 + 2 * i) for i in range(14)]  # harmless fake device addresses, far apart


def plan(ptrs=None, B=4, T=16, max_pages=8, num_free=8, num_pages=32, page=64):
    p = list(A[:9]) if ptrs is None else ptrs
    return fa.fa_kv_plan_raw(*p, B, T, max_pages, num_free, num_pages, page, 0)


def append(ptrs=None, T=16, Hkv=2, D=64, ks=128, vs=128, num_pages=4, page=16):
    p = list(A[:9]) if ptrs is None else ptrs
    return fa.fa_kv_append_raw(*p, T, Hkv, D, ks, vs, num_pages, page, 0)


def select(ptrs=None, B=2, T=2, Hq=4, Hkv=2, D=64, qs=256, max_pages=8, num_pages=4, page=16, top=4, first=1, last=1):
    p = list(A[:8]) if ptrs is None else ptrs
    return fa.fa_page_select_raw(*p, B, T, Hq, Hkv, D, qs, max_pages, num_pages, page, top, first, last, 0)


def attend(ptrs=None, B=2, T=2, Hq=4, Hkv=2, D=64, scale=0.125, qs=256, max_pages=8, num_pages=4, page=16, width=4,
           ws=1 << 50, ws_bytes=1 << 40):
    p = list(A[:12]) if ptrs is None else ptrs
    return fa.fa_fwd_paged_raw(*p, B, T, Hq, Hkv, D, scale, qs, max_pages, num_pages, page, width, ws, ws_bytes, 0)


CALLS = [(plan, 9, ()), (append, 9, (7, 8)), (select, 8, ()), (attend, 12, (8, 9))]


@pytest.mark.parametrize("call,n,optional", CALLS)
def test_null_and_misaligned_pointers(call, n, optional):
    for i in range(n):
        p = list(A[:n])
        p[i] = 0
        assert call(p) == fa.FA_ERR_NULLPTR, i  # of an optional pair, one without the other
        p[i] = A[i] + 2
        assert call(p) == fa.FA_ERR_MISALIGNED, i
    # codes and bf16 need 16 bytes, int32 and fp32 arrays 4
    wide = {plan: (), append: (0, 1, 3, 4, 7), select: (0, 4), attend: (0, 4, 5, 10)}[call]
    for i in wide:
        p = list(A[:n])
        p[i] = A[i] + 4
        assert call(p) == fa.FA_ERR_MISALIGNED, i


@pytest.mark.parametrize("call", [plan, append, select, attend])
@pytest.mark.parametrize("page", [0, 1, 8, 24, 48, 256, -16])
def test_page_sizes(call, page):
    assert call(page=page) == fa.FA_ERR_BAD_PAGE
    assert "page" in fa.fa_strerror(fa.FA_ERR_BAD_PAGE)


@pytest.mark.parametrize("call", [append, select, attend])
@pytest.mark.parametrize("D", [0, 32, 96, 256])
def test_head_dims(call, D):
    assert call(D=D) == fa.FA_ERR_UNSUPPORTED_D


@pytest.mark.parametrize("call,kw", [
    (plan, dict(B=0)), (plan, dict(B=8193)), (plan, dict(T=0)), (plan, dict(max_pages=0)), (plan, dict(num_free=0)),
    (plan, dict(num_pages=0)), (plan, dict(num_pages=1 << 25, page=64)), (plan, dict(max_pages=1 << 27, page=16)),
    (append, dict(T=0)), (append, dict(Hkv=0)), (append, dict(Hkv=1025)), (append, dict(ks=120)), (append, dict(vs=132)),
    (append, dict(num_pages=1 << 27)), (append, dict(ks=-128)),
    (select, dict(Hq=5)), (select, dict(Hq=0)), (select, dict(top=0)), (select, dict(first=-1)), (select, dict(last=-1)),
    (select, dict(first=3, last=2)), (select, dict(max_pages=49153)), (select, dict(qs=248)), (select, dict(B=0)),
    (attend, dict(Hq=3)), (attend, dict(B=0)), (attend, dict(T=0)), (attend, dict(width=0)), (attend, dict(qs=255)),
    (attend, dict(Hkv=0)), (attend, dict(max_pages=0))])
def test_bad_shapes(call, kw):
    assert call(**kw) == fa.FA_ERR_BAD_SHAPE


@pytest.mark.parametrize("call,name", [(plan, "T"), (plan, "num_free"), (append, "T"), (select, "T"), (select, "top"),
                                       (attend, "T")])
def test_counts_that_an_int_cannot_step_past(call, name):
    """A loop that steps past the end of 2^31 - 1 items would go on at negative indexes."""
    kw = dict(Hq=1, Hkv=1) if call in (select, attend) else {}
    for n in (2 ** 31 - 1, 2 ** 31 - 2 ** 17, 2 ** 30 + 1):
        assert call(**{**kw, name: n}) == fa.FA_ERR_BAD_SHAPE


@pytest.mark.parametrize("call", [select, attend])
@pytest.mark.parametrize("T,Hq", [(1 << 30, 2), (1 << 20, 1 << 15), (1 << 25, 64)])
def test_query_rows_that_an_int_does_not_count(call, T, Hq):
    assert call(T=T, Hq=Hq, Hkv=1, qs=64 * Hq) == fa.FA_ERR_BAD_SHAPE


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 0.0, -0.5, 3e38])
def test_attend_scale(scale):
    assert attend(scale=scale) == fa.FA_ERR_BAD_SCALE


def test_attend_workspace():
    need = fa.fa_fwd_paged_workspace_bytes(2, 2, 4, 2, 64)
    assert need > 0
    assert attend(ws=0) == fa.FA_ERR_WORKSPACE
    assert attend(ws=(1 << 50) + 8) == fa.FA_ERR_WORKSPACE
    assert attend(ws_bytes=need - 1) == fa.FA_ERR_WORKSPACE
    for bad in ((0, 2, 4, 2, 64), (2, 2, 3, 2, 64), (2, 2, 4, 2, 96), (2, 0, 4, 2, 64)):
        assert fa.fa_fwd_paged_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(2, 2 ** 30 + 1, 1, 1, 64), (2, 2 ** 31 - 1, 1, 1, 128), (2, 1 << 30, 2, 1, 64),
                                          (2, 1 << 16, 1 << 15, 1, 64)])
def test_no_workspace_for_sizes_that_are_refused(B, T, Hq, Hkv, D):
    assert attend(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, qs=Hq * D) == fa.FA_ERR_BAD_SHAPE
    assert fa.fa_fwd_paged_workspace_bytes(B, T, Hq, Hkv, D) == 0


def test_aliases():
    p = list(A[:9])
    p[8] = p[3]  # free_left over free_count
    assert plan(p) == fa.FA_ERR_ALIAS
    p = list(A[:9])
    p[6] = p[0] + 8  # seq_lens over cached_lens
    assert plan(p) == fa.FA_ERR_ALIAS
    p = list(A[:9])
    p[4] = p[3]  # the two caches are one
    assert append(p) == fa.FA_ERR_ALIAS
    p = list(A[:9])
    p[0] = p[3] + 16  # keys inside the cache
    assert append(p) == fa.FA_ERR_ALIAS
    p = list(A[:8])
    p[6] = p[3]  # sel over the block table
    assert select(p) == fa.FA_ERR_ALIAS
    p = list(A[:12])
    p[10] = p[0]  # o over q
    assert attend(p) == fa.FA_ERR_ALIAS
    assert attend(ws=A[4]) == fa.FA_ERR_ALIAS
    # keys and values in one fused tensor do not alias
    if not torch.cuda.is_available():
        p = list(A[:9])
        p[1] = p[0] + 2 * 128
        assert append(p, ks=256, vs=256) == fa.FA_ERR_CUDA


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path only")
@pytest.mark.parametrize("call,n,optional", CALLS)
def test_valid_calls_without_gpu_report_cuda_error(call, n, optional):
    assert call() == fa.FA_ERR_CUDA
    if optional:
        p = list(A[:n])
        for i in optional:
            p[i] = None
        assert call(p) == fa.FA_ERR_CUDA


def test_wrappers_reject_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2)
    with pytest.raises(ValueError):
        fa.fa_kv_plan(i, i.clone(), i.clone(), i[:1], torch.zeros(4, 2, dtype=torch.int32), 4, 16, num_tokens=4)
    with pytest.raises(ValueError):
        fa.fa_kv_append(q, q, i, c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        fa.fa_page_select(q, i, i[:3], torch.zeros(3, 2, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.int8), s, 16, 4)
    with pytest.raises(ValueError):
        fa.fa_fwd_paged(q, i, i[:3], torch.zeros(3, 2, dtype=torch.int32), c, c.clone(), s, s.clone())


# ------------------------------------------- pins of the plain implementations
def test_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    v = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(pu.E4M3)) and np.array_equal(v[~np.isnan(v)], pu.E4M3[~np.isnan(v)])
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * s for s in (1e-3, 1.0, 100.0)] +
                       [(pu._POS[:-1] + pu._POS[1:]) / 2, pu._POS, -pu._POS]).astype(np.float32).clip(-448, 448)
    assert np.array_equal(pu.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(pu.to_e4m3([np.inf, -np.inf, np.nan, 1e9])) == [0x7E, 0xFE, 0x7F, 0x7E]


def test_scale_is_the_smallest_power_of_two():
    for a in (448.0, 448.0000001, 447.0, 1.75, 1.7500001, 3e-20, 0.4375, 5.0):
        s = pu.pow2_scale(a)
        assert a <= 448 * s and a > 224 * s and math.log2(s) == int(math.log2(s))
    assert pu.pow2_scale(0.0) == 1.0 and pu.pow2_scale(1e-40) == 2.0 ** -100


def test_plan_by_hand():
    table = np.full((3, 4), -1)
    table[0, 0] = 5
    cu, lens, slots, left, table = pu.plan([10, 0, 0], [10, 20, 3], [7, 8, 9], 3, table, 40, 16, 16)
    assert cu == [0, 10, 30, 33] and lens == [20, 20, 0] and left == 0
    assert list(table[0, :2]) == [5, 9] and list(table[1, :2]) == [8, 7] and list(table[2]) == [-1] * 4
    assert slots[:6] == [90, 91, 92, 93, 94, 95] and slots[6] == 144 and slots[10] == 128 and slots[26] == 112
    assert slots[30:] == [-1] * 10


def test_attend_matches_dense_softmax():
    c = pu.Cache([37, 0, 16], 2, 16, 64, seed=1, device="cpu")
    q, cu, _ = pu.queries([2, 0, 1], 4, 64, 2, pad=1, device="cpu")
    qn = pu.f64(q)
    o, lse, _, _ = pu.attend(qn, cu, c.lens, c.table, c.kc, c.vc, c.ks, c.vs, 0.125, 16)
    K = np.concatenate([pu.E4M3[c.kc[p, 1]] * c.ks[p, 1] for p in c.table[0, :3]])[:36]
    V = np.concatenate([pu.E4M3[c.vc[p, 1]] * c.vs[p, 1] for p in c.table[0, :3]])[:36]
    s = torch.from_numpy(K @ qn[0, 3]) * 0.125
    assert np.allclose(o[0, 3], (torch.softmax(s, 0).numpy() @ V), rtol=1e-12, atol=1e-14)
    assert abs(lse[0, 3] - float(torch.logsumexp(s, 0))) < 1e-12
