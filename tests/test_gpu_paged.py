"""GPU parity of the paged 8-bit cache's operators (fa_kv_plan, fa_kv_append,
fa_page_select, fa_fwd_paged) against plain 64-bit implementations of their
definitions, at the sizes and contents where they can go wrong, and a run of them
together as a serving loop uses them."""
import threading

import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert fa.fa_device_status() == fa.FA_OK


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- plan
def run_plan(cached, new, free, count, table, T, num_pages, page):
    d_table = i32(table.tolist())
    cu, lens, slots, left = fa.fa_kv_plan(i32(cached), i32(new), i32(free), i32([count]), d_table, num_pages, page, num_tokens=T)
    ref = pu.plan(cached, new, free, count, table, T, num_pages, page)
    for name, a, r in zip(("cu_q", "seq_lens", "slot_map", "left", "table"), (cu, lens, slots, left, d_table), ref):
        assert np.array_equal(a.cpu().numpy().reshape(np.shape(r)), np.array(r)), name


@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("B,short", [(1, 1.0), (7, 1.0), (64, 0.6), (300, 1.0), (1025, 0.9), (8192, 0.5)])
def test_plan(page, B, short):
    rng = np.random.default_rng(B * 1000 + page)
    cached = rng.integers(0, 300, size=B)
    new = np.where(rng.random(B) < 0.5, 1, rng.integers(0, 90 if B > 1000 else 400, size=B))
    held, need = -(-cached // page), -(-(cached + new) // page)
    width = int(need.max()) + 1
    num_pages = int(need.sum()) + 5
    ids = rng.permutation(num_pages)
    table = np.full((B, width), -1)
    for b in range(B):
        table[b, :held[b]], ids = ids[:held[b]], ids[held[b]:]
    count = int(short * (need - held).sum())
    run_plan(cached.tolist(), new.tolist(), ids.tolist(), count, table, int(new.sum()) + 17, num_pages, page)


def test_plan_invalid_requests():
    """Negative lengths, a request longer than its table row, pages outside the cache, too few token slots,
    and more free pages claimed than the list holds."""
    table = np.array([[3, -1, -1], [-1] * 3, [40, -1, -1], [2, 6, -1], [-9, -1, -1], [-1] * 3, [-1] * 3])
    cached, new = [5, -4, 9, 30, 3, 0, 0], [20, 9, 12, 40, 2, 0, 30]
    for count in (0, 1, 2, 3, 6, 99, -5):
        run_plan(cached, new, [10, 11, 70, -3, 12, 13], count, table, 118, 30, 16)
    run_plan(cached, new, [10, 11, 9, 8, 12, 13], 6, table, 20, 30, 16)  # tokens behind T are dropped
    run_plan([0] * 4, [0] * 4, [1], 1, np.full((4, 1), -1), 3, 4, 128)  # nothing to do
    big = 2 ** 31 - 1
    run_plan([big, 0, 1], [big, big, 5], [1, 2], 2, np.full((3, 2), 0), 12, 4, 64)  # sums past 32 bits


def test_plan_in_two_threads():
    """Batches of different sizes, all of which need more shared memory than a kernel has without asking."""
    calls, checks = [], []
    for B in (8192, 6200):
        one = torch.ones(B, dtype=torch.int32, device="cuda")
        table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, B, 1)]
        args = (one, one.clone(), i32([0]), i32([0]), table, B, 16, *out)
        calls.append(lambda args=args: fa.fa_kv_plan(*args))
        checks.append(out)
    two_threads(*calls)
    for cu, lens, slots, left in checks:
        assert torch.equal(cu, torch.arange(cu.numel(), device="cuda", dtype=torch.int32)) and int(left) == 0
        assert bool((lens == 2).all()) and bool((slots == 1).all())


# ------------------------------------------------------------------ append
def run_append(lens, new, Hkv, page, D, seed, pad=0, means=True, change=None, gap=False):
    """Appends `new` tokens behind `lens` cached ones and compares every page and scale."""
    c = pu.Cache([a + b for a, b in zip(lens, new)], Hkv, page, D, seed)
    rng = np.random.default_rng(seed)
    T = sum(new) + pad
    slots = []
    for b, (a, n) in enumerate(zip(lens, new)):
        slots += [int(c.table[b, t // page]) * page + t % page for t in range(a, a + n)]
    slots = np.array(slots + [-1] * pad, np.int32)
    if gap:
        slots[rng.integers(0, T, size=max(1, T // 9))] = -1
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn((T, 2 * Hkv, D), generator=g) * torch.exp(torch.randn((T, 2 * Hkv, 1), generator=g))).to(torch.bfloat16)
    if change:
        change(wide)
    k, v = wide[:, :Hkv], wide[:, Hkv:]
    dw = wide.cuda()
    fa.fa_kv_append(dw[:, :Hkv], dw[:, Hkv:], torch.from_numpy(slots).cuda(), *c.pages, k_mean=c.d_mean if means else None,
                    k_mean_scale=c.d_ms if means else None)
    mean, ms = c.mean.copy(), c.ms.copy()
    pu.append(pu.f64(k), slots, c.kc, c.ks, page, *((mean, ms) if means else ()))
    pu.append(pu.f64(v), slots, c.vc, c.vs, page)
    for name, a, r in (("k", c.d_kc, c.kc), ("v", c.d_vc, c.vc)):
        a = pu.codes_of(a)
        same = (a == r) | (np.isnan(pu.E4M3[a]) & np.isnan(pu.E4M3[r]))
        assert same.all(), f"{name} codes: {np.argwhere(~same)[:4].tolist()}"
    assert np.array_equal(pu.f64(c.d_ks), c.ks) and np.array_equal(pu.f64(c.d_vs), c.vs)
    assert np.array_equal(c.d_mean.cpu().numpy(), mean) and np.array_equal(c.d_ms.cpu().numpy(), ms)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
def test_append_ragged(page, D):
    lens = [0, 0, 5, page - 1, page, 3 * page + 1, 2 * page - 1, 0, 7]
    new = [1, 2 * page + 3, 1, 1, 1, page - 1, 2, page, 0]
    run_append(lens, new, 3, page, D, seed=page + D, pad=5)


def test_append_decode_and_prompt_shapes():
    run_append([i * 3 for i in range(100)], [1] * 100, 2, 64, 128, seed=1)
    run_append([0], [1500], 1, 64, 64, seed=2)
    run_append([17], [1500], 2, 16, 128, seed=3, pad=100)
    run_append([0, 9], [1, 1], 1, 128, 64, seed=4, means=False)


def test_append_skipped_tokens_inside_a_batch():
    run_append([0], [1], 1, 16, 64, seed=5)
    run_append([3, 40, 0, 11, 16, 20] * 4, [1] * 24, 2, 32, 64, seed=6, gap=True)


def test_append_special_values():
    def change(w):
        w[0] = 0.0                                  # a page of zeros has scale 1
        w[1, :, 3], w[1, :, 4] = float("inf"), float("-inf")
        w[2, :, 5] = float("nan")
        w[3] = float("nan")
        w[4] = 1.75 * 2.0 ** -12                    # exactly 448 * 2^-20
        w[5] = 1e-38                                # below what the smallest scale holds
        w[6] = 3e38
        w[7, :, 0] = 1.7578125                      # one step above 448 * 2^-8

    for page in (16, 64):
        run_append([0, 5, 0, 7, 0, 9, 0, 0], [1] * 8, 2, page, 64, seed=7, change=change)
    run_append([0, 3], [8, 8], 1, 16, 128, seed=8, change=change)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
def test_append_special_values_in_whole_pages(page, D):
    """Pages that one run fills: a zero page, infinities, NaN, the smallest and the largest numbers, and a
    page of one value; with and without means."""
    def change(w):
        w[:page] = 0.0
        w[page + 3, :, 1], w[page + 4, :, 2], w[page + 5] = float("inf"), float("-inf"), float("nan")
        w[2 * page:3 * page] = float("nan")
        w[3 * page:4 * page] = 1e-38
        w[4 * page:5 * page:2] = 3e38
        w[5 * page:6 * page] = -1.75 * 2.0 ** -12

    for means in (True, False):
        run_append([0, 0], [7 * page, page], 2, page, D, seed=page, change=change, means=means)


def test_append_beside_scales_that_are_no_powers_of_two():
    """A page whose scale the caller has set: what is added to it is divided by that scale."""
    c = pu.Cache([40, 24], 2, 16, 64, seed=9)
    c.ks *= 1.5
    c.vs *= 1.25
    c.d_ks, c.d_vs = torch.from_numpy(c.ks).float().cuda(), torch.from_numpy(c.vs).float().cuda()
    x = torch.randn((4, 2, 64), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16) * 0.5
    slots = np.array([int(c.table[0, 2]) * 16 + 5 + i for i in range(3)] + [int(c.table[1, 1]) * 16 + 3], np.int32)
    fa.fa_kv_append(x.cuda(), x.cuda(), torch.from_numpy(slots).cuda(), *c.pages)
    for codes, scale, got, got_scale in ((c.kc, c.ks, c.d_kc, c.d_ks), (c.vc, c.vs, c.d_vc, c.d_vs)):
        pu.append(pu.f64(x), slots, codes, scale, 16)
        assert np.array_equal(pu.f64(got_scale), scale)
        assert np.array_equal(pu.codes_of(got), codes)


def test_append_infinities_beside_scales_that_are_no_powers_of_two():
    """Infinities become the largest codes, whatever scale the page has."""
    for page, D in ((16, 64), (128, 128)):
        c = pu.Cache([page + 7, page + 3], 2, page, D, seed=19)
        c.ks *= 1.5
        c.vs *= 1.25
        c.d_ks, c.d_vs = torch.from_numpy(c.ks).float().cuda(), torch.from_numpy(c.vs).float().cuda()
        x = torch.randn((3, 2, D), generator=torch.Generator().manual_seed(19)).to(torch.bfloat16) * 0.5
        x[0, :, 3], x[0, :, 4], x[1, 1, 5], x[2, :, 9] = float("inf"), float("-inf"), float("nan"), float("-inf")
        slots = np.array([int(c.table[0, 1]) * page + 5 + i for i in range(2)] + [int(c.table[1, 1]) * page + 2], np.int32)
        fa.fa_kv_append(x.cuda(), x.cuda(), torch.from_numpy(slots).cuda(), *c.pages)
        for codes, scale, got, got_scale in ((c.kc, c.ks, c.d_kc, c.d_ks), (c.vc, c.vs, c.d_vc, c.d_vs)):
            pu.append(pu.f64(x), slots, codes, scale, page)
            got = pu.codes_of(got)
            assert np.array_equal(pu.f64(got_scale), scale)
            assert ((got == codes) | (np.isnan(pu.E4M3[got]) & np.isnan(pu.E4M3[codes]))).all()


def test_append_bad_slots_are_skipped_and_reported():
    c = pu.Cache([20], 2, 16, 64, seed=9)
    before = [t.clone() for t in c.pages]
    x = torch.randn((4, 2, 64), device="cuda").to(torch.bfloat16)
    slots = i32([c.num_pages * 16, 2 ** 31 - 1, -1, -2 ** 31])
    fa.fa_kv_append(x, x.clone(), slots, *c.pages)
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE
    assert all(torch.equal(a, b) for a, b in zip(before, c.pages))


# ------------------------------------------------------------------ select
def run_select(c, q, cu, d_cu, top, first, last):
    sel, count = fa.fa_page_select(q, d_cu, c.d_lens, c.d_table, c.d_mean, c.d_ms, c.page, top, first, last)
    rs, rc = pu.select(pu.f64(q), cu, c.lens, c.table, c.mean, c.ms, c.page, top, first, last)
    assert np.array_equal(count.cpu().numpy(), rc)
    assert np.array_equal(sel.cpu().numpy(), rs)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (3, 16)])
@pytest.mark.parametrize("top,first,last", [(1, 0, 0), (4, 1, 1), (8, 0, 8), (33, 2, 1)])
def test_select(D, Hkv, G, top, first, last):
    lens = [0, 1, 16, 17, 300, 0, 1600, 16 * top, 16 * top + 1]
    counts = [0, 1, 1, 2, 1, 1, 5, 1, 2]
    c = pu.Cache(lens, Hkv, 16, D, seed=D + top)
    q, cu, d_cu = pu.queries(counts, Hkv * G, D, seed=G, pad=2)
    run_select(c, q, cu, d_cu, top, first, last)


def test_select_ties_and_special_queries():
    c = pu.Cache([3000, 3000, 900, 640], 2, 16, 64, seed=3)
    q, cu, d_cu = pu.queries([1, 2, 1, 1], 4, 64, seed=4)
    c.mean[:] = c.mean[:1, :1]
    c.ms[:] = 0.25
    c.mean[::3] = -c.mean[::3]                      # two values: ties all along
    q[1] = 0.0                                      # every score 0
    q[3, 0, 5], q[3, 1, 6] = float("nan"), float("inf")
    q[4] = float("nan")
    c.d_mean, c.d_ms = torch.from_numpy(c.mean).cuda(), torch.from_numpy(c.ms).cuda()
    run_select(c, q, cu, d_cu, 20, 1, 2)


def test_select_long_sequence():
    c = pu.Cache([49000], 1, 16, 64, seed=5, num_pages=4000)
    q, cu, d_cu = pu.queries([1], 8, 64, seed=6)
    for top in (5, 64, 1000):
        run_select(c, q, cu, d_cu, top, 1, 2)


@pytest.mark.parametrize("width,G,D", [(300, 4, 64), (700, 16, 128), (2100, 3, 64)])
def test_select_wide_tables(width, G, D):
    """Tables that several blocks score: long and short sequences beside one another, some shorter than
    top_k, more query rows than are scored at a time."""
    lens = [16 * width, 1, 0, 16 * 40, 16 * 60 + 5, 16 * (width - 13) + 3, 16 * 259]
    c = pu.Cache(lens, 2, 16, D, seed=width, extra_cols=0)
    q, cu, d_cu = pu.queries([3, 1, 1, 1, 0, 2, 4], 2 * G, D, seed=G, pad=1)
    run_select(c, q, cu, d_cu, 50, 2, 3)
    c.mean[:, :, :] = c.mean[:1, :1]
    c.ms[:] = np.linspace(0.5, 2, 5).astype(np.float32)[np.arange(c.num_pages) % 5, None]   # five values: many ties
    c.d_mean, c.d_ms = torch.from_numpy(c.mean).cuda(), torch.from_numpy(c.ms).cuda()
    run_select(c, q, cu, d_cu, 64, 0, 0)


def two_threads(*calls, times=3000):
    """Makes the calls again and again, each in a thread and on a stream of its own; what they raise is raised."""
    failed = []

    def loop(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(times):
                    call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if failed:
        raise failed[0]


def test_select_in_two_threads():
    """Tables of different widths, all of which need more shared memory than a kernel has without asking."""
    calls, checks = [], []
    for width in (49152, 8300):
        c = pu.Cache([40], 1, 16, 64, seed=1)
        table, lens = torch.zeros((1, width), dtype=torch.int32, device="cuda"), i32([16 * 40])
        table[0, :40] = i32([int(p) for p in np.arange(40) % c.num_pages])
        q, cu, d_cu = pu.queries([1], 2, 64, seed=1)
        args = (q, d_cu, lens, table, c.d_mean, c.d_ms, 16, 5)
        want, _ = fa.fa_page_select(*args)
        out = dict(sel=torch.empty_like(want), sel_count=torch.empty((1, 1), dtype=torch.int32, device="cuda"))
        calls.append(lambda args=args, out=out: fa.fa_page_select(*args, **out))
        checks.append((out["sel"], want))
    two_threads(*calls)
    for got, want in checks:
        assert torch.equal(got, want)


@pytest.mark.parametrize("n", [8193, 16385, 16400, 40001, 49152])
def test_select_widest_tables(n):
    """Tables beyond what a kernel's shared memory holds without asking, and lists of more than 32 positions a
    thread; many entries of the table are the same page, so that scores tie all along."""
    rng = np.random.default_rng(n)
    c = pu.Cache([16 * 300], 1, 16, 64, seed=n)
    c.table = rng.integers(0, c.num_pages, size=(2, n)).astype(np.int32)
    c.table[1] = np.arange(n) % 3
    c.lens = [16 * n, 16 * n - 9]
    c.d_table, c.d_lens = torch.from_numpy(c.table).cuda(), i32(c.lens)
    q, cu, d_cu = pu.queries([1, 2], 3, 64, seed=n)
    for top in (7, n // 2, n - 1):
        run_select(c, q, cu, d_cu, top, 1, 2)


def test_select_pages_outside_the_cache_come_last():
    c = pu.Cache([800], 1, 16, 64, seed=5)
    q, cu, d_cu = pu.queries([1], 2, 64, seed=6)
    c.table[0, 5:40:3] = [c.num_pages, -1, 2 ** 31 - 1, -2 ** 31] * 3
    c.d_table = torch.from_numpy(c.table).cuda()
    run_select(c, q, cu, d_cu, 45, 1, 2)
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE


@pytest.mark.parametrize("outlier", [False, True])
@pytest.mark.parametrize("top,first,last", [(64, 1, 1), (1500, 2, 3), (7, 3, 4), (2999, 0, 0)])
def test_select_crowded_scores(top, first, last, outlier):
    """Scores that steps from the least to the largest do not tell apart: two values all along, or one page
    far above or below all others; and no room but for the pages that are kept anyway."""
    c = pu.Cache([16 * 3000 - 5], 1, 16, 64, seed=top, num_pages=3100)
    q, cu, d_cu = pu.queries([1], 2, 64, seed=top)
    if outlier:
        c.ms[c.table[0, 1234 + top % 2]] = 1e9
    else:
        c.mean[:] = c.mean[:1]
        c.mean[1::2] = -c.mean[1::2]
        c.ms[:] = 0.5
    c.d_mean, c.d_ms = torch.from_numpy(c.mean).cuda(), torch.from_numpy(c.ms).cuda()
    run_select(c, q, cu, d_cu, top, first, last)


def test_select_tiny_queries():
    """Queries down to bf16's smallest numbers are rounded like others: 127 / max|q| is past the largest float
    below 2^-121.  The pages' scores lie in powers of two apart, so that their 32-bit products (which are
    subnormal, with 10 bits or more) keep the order."""
    c = pu.Cache([640], 1, 16, 64, seed=7)
    rng = np.random.default_rng(8)
    c.mean[:] = rng.integers(64, 128, size=c.mean.shape[:2])[..., None] * rng.choice([-1, 1], size=64)
    c.ms[:, 0] = np.exp2(rng.permutation(c.num_pages)).astype(np.float32)
    c.d_mean, c.d_ms = torch.from_numpy(c.mean).cuda(), torch.from_numpy(c.ms).cuda()
    sign = torch.from_numpy(np.sign(c.mean[0, 0]).astype(np.float32)).cuda()
    want = None
    for e in (0, -100, -120, -121, -122, -126, -130, -133):
        q = (sign * 2.0 ** e).to(torch.bfloat16).view(1, 1, 64).expand(1, 2, 64).contiguous()
        sel, n = fa.fa_page_select(q, i32([0, 1]), c.d_lens, c.d_table, c.d_mean, c.d_ms, 16, 9)
        assert int(n) == 9
        want = sel if want is None else want
        assert torch.equal(sel, want), e
    ref = pu.select(pu.f64(sign.view(1, 1, 64).expand(1, 2, 64)), np.array([0, 1]), c.lens, c.table, c.mean, c.ms, 16, 9, 1, 1)
    assert np.array_equal(want.cpu().numpy(), ref[0])


# ------------------------------------------------------------------ attend
def run_attend(c, q, cu, d_cu, sel=None, count=None, scale=None, what="", **kw):
    T, Hq, D = q.shape
    o = torch.full((T, Hq, D), 777.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 777.0, device="cuda")
    d = {} if sel is None else dict(sel=torch.from_numpy(np.ascontiguousarray(sel, np.int32)).cuda(),
                                    sel_count=torch.from_numpy(np.ascontiguousarray(count, np.int32)).cuda())
    fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages, o=o, lse=lse, scale=scale, **d, **kw)
    torch.cuda.synchronize()
    rows = int(cu[-1])
    assert bool((o[rows:] == 777).all()) and bool((lse[rows:] == 777).all()), "padding rows were written"
    ref = pu.attend(pu.f64(q), cu, c.lens, c.table, c.kc, c.vc, c.ks, c.vs, scale or D ** -0.5, c.page, sel, count)
    pu.check_attend(o, lse, ref, what, rows)
    return o, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 3), (1, 8), (2, 16), (1, 40)])
def test_attend_decode(D, page, Hkv, G):
    lens = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 700]
    c = pu.Cache(lens, Hkv, page, D, seed=D + page + G)
    q, cu, d_cu = pu.queries([0 if L == 0 else 1 for L in lens], Hkv * G, D, seed=G, pad=3)
    run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 8, 5])
def test_attend_several_tokens(D, G):
    """Causal among a sequence's query tokens; more of them than keys, so that rows see none."""
    lens, counts = [1, 7, 40, 64, 500, 3, 0, 2, 129, 33], [1, 8, 3, 5, 8, 6, 2, 0, 2, 33]
    for page in (16, 64):
        c = pu.Cache(lens, 2, page, D, seed=D + G + page)
        q, cu, d_cu = pu.queries(counts, 2 * G, D, seed=G, pad=1)
        run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,page", [(1, 64), (16, 16)])
def test_attend_prompts(D, G, page):
    """As many query rows as a prompt has: several passes over the keys, masked tiles in most of them."""
    lens, counts = [130, 61, 300, 47], [130, 61, 90, 5]
    c = pu.Cache(lens, 1, page, D, seed=D + G)
    q, cu, d_cu = pu.queries(counts, G, D, seed=G, pad=2)
    run_attend(c, q, cu, d_cu)
    chosen = [1, 0] if page == 16 else [0]  # in any order
    sel = np.full((4, 1, 3), -1, np.int32)
    sel[:, 0, :len(chosen)] = chosen
    run_attend(c, q, cu, d_cu, sel=sel, count=np.full((4, 1), len(chosen), np.int32))


@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
def test_attend_long_and_ragged(page):
    lens = [5000, 1, 2500, 77, 9001]
    c = pu.Cache(lens, 2, page, 128, seed=page)
    q, cu, d_cu = pu.queries([1, 1, 4, 1, 2], 8, 128, seed=page)
    o1, l1 = run_attend(c, q, cu, d_cu)
    o2, l2 = run_attend(c, q, cu, d_cu)
    assert torch.equal(o1, o2) and torch.equal(l1, l2), "not deterministic"


def test_attend_many_sequences():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 150, size=700).tolist()
    c = pu.Cache(lens, 1, 16, 64, seed=1)
    q, cu, d_cu = pu.queries(rng.integers(0, 3, size=700).tolist(), 2, 64, seed=2, pad=9)
    run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("seed", range(16))
def test_attend_random_batches(seed):
    """Batches of any mixture of lengths, tokens and heads: how the work is cut must not show."""
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.choice([1, 2, 3, 17, 60, 150]))
    top = int(rng.choice([20, 120, 700, 4000 if B < 10 else 700]))
    Hkv, G, D = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 4, 7, 8, 16])), int(rng.choice([64, 128]))
    page = int(rng.choice(fa.FA_PAGE_SIZES))
    lens = [int(rng.integers(0, 1 + (top if rng.random() < 0.3 else top // 8))) for _ in range(B)]
    counts = [int(rng.choice([0, 1, 1, 1, 2, 5])) for _ in range(B)]
    c = pu.Cache(lens, Hkv, page, D, seed=seed)
    q, cu, d_cu = pu.queries(counts, Hkv * G, D, seed=seed, pad=int(rng.integers(0, 4)))
    run_attend(c, q, cu, d_cu, what=f"{B} {top} {Hkv} {G} {D} {page}")


def test_attend_heads_of_short_sequences():
    """Thousands of items of a few tiles each."""
    rng = np.random.default_rng(5)
    for hi in (33, 97, 260):
        lens = rng.integers(1, hi, size=180).tolist()
        c = pu.Cache(lens, 8, 16, 64, seed=hi)
        q, cu, d_cu = pu.queries([1] * 180, 8, 64, seed=hi)
        run_attend(c, q, cu, d_cu, what=str(hi))


def test_attend_types_streams_and_workspaces():
    """Codes as float8 tensors, an exact workspace that held other things, streams as objects and addresses."""
    c = pu.Cache([900, 40, 2000], 2, 32, 128, seed=8)
    q, cu, d_cu = pu.queries([1, 2, 1], 8, 128, seed=8)
    o, lse = run_attend(c, q, cu, d_cu)
    T, Hq, _ = q.shape
    ws = torch.full((fa.fa_fwd_paged_workspace_bytes(3, T, Hq, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    f8 = [t.view(torch.float8_e4m3fn) for t in c.pages[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream, 0):
        o2, l2 = fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *f8, *c.pages[2:], workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    before = [t.clone() for t in c.pages]
    x = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    fa.fa_kv_append(x, x, i32([-1]), *f8, *c.pages[2:], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, c.pages))


@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("D", [64, 128])
def test_attend_selected_pages(page, D):
    rng = np.random.default_rng(page)
    lens, counts = [1000, page, 3 * page - 1, 0, 777, 5 * page + 1], [1, 1, 2, 1, 3, 1]
    c = pu.Cache(lens, 2, page, D, seed=D + page)
    q, cu, d_cu = pu.queries(counts, 8, D, seed=page, pad=2)
    W = 7
    sel, count = np.full((6, 2, W), -5), np.zeros((6, 2), int)
    for b, L in enumerate(lens):
        n = -(-L // page)
        for h in range(2):
            k = int(rng.integers(0, min(n, W) + 1)) if b != 1 else 1
            sel[b, h, :k], count[b, h] = rng.permutation(n)[:k], k
    run_attend(c, q, cu, d_cu, sel, count)
    full = np.full((6, 2, 70), -1)
    for b, L in enumerate(lens):
        n = -(-L // page)
        full[b, :, :n] = np.arange(n)
    o1, l1 = run_attend(c, q, cu, d_cu, full, np.array([[-(-L // page)] * 2 for L in lens]))


def test_pages_shared_and_chosen_twice():
    """Sequences with pages in common (the same prompt), a page twice in one row of the table, and a position
    that is chosen twice, which counts twice."""
    c = pu.Cache([200, 333, 333, 64], 2, 16, 64, seed=21)
    c.table[1, :12] = c.table[0, :12]
    c.table[2, :21] = c.table[1, :21]
    c.table[2, 3] = c.table[2, 7]
    c.d_table = torch.from_numpy(c.table).cuda()
    q, cu, d_cu = pu.queries([2, 1, 1, 1], 8, 64, seed=21)
    run_attend(c, q, cu, d_cu)
    sel = np.tile(np.array([1, 0, 1, 3, 3, 2]), (4, 2, 1))
    run_attend(c, q, cu, d_cu, sel, np.array([[6, 5], [3, 6], [0, 1], [4, 2]]))
    run_select(c, q, cu, d_cu, 9, 1, 1)


def test_attend_masked_values_never_touch_a_row():
    """NaN codes behind the last key (every Cache holds them), and NaN keys and values that only a
    sequence's later query tokens see."""
    lens, counts = [40, 16, 129, 70], [3, 2, 4, 8]
    for D in (64, 128):
        c = pu.Cache(lens, 1, 16, D, seed=D)
        for b, (L, n) in enumerate(zip(lens, counts)):
            t = L - 1 - b % 2                       # the last or last but one key
            c.kc[c.table[b, t // 16], 0, t % 16, 3] = 0x7F if b < 2 else c.kc[c.table[b, t // 16], 0, t % 16, 3]
            c.vc[c.table[b, t // 16], 0, t % 16, 5:9] = 0xFF
        c.d_kc, c.d_vc = torch.from_numpy(c.kc).cuda(), torch.from_numpy(c.vc).cuda()
        q, cu, d_cu = pu.queries(counts, 4, D, seed=D)
        run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_masked_values_beside_many_rows(D):
    lens, counts = [40, 16, 129, 70], [3, 2, 4, 8]
    c = pu.Cache(lens, 1, 32, D, seed=D)
    for b, L in enumerate(lens):
        t = L - 1 - b % 2
        c.vc[c.table[b, t // 32], 0, t % 32, 5:9] = 0xFF
    c.d_vc = torch.from_numpy(c.vc).cuda()
    q, cu, d_cu = pu.queries(counts, 20, D, seed=D)
    run_attend(c, q, cu, d_cu)


def test_attend_peaky_and_uneven_scales():
    """Scores in the hundreds, and pages whose scales differ by 2^40."""
    for seed, mult in ((1, 30.0), (2, 1.0)):
        c = pu.Cache([900, 64, 333], 2, 32, 128, seed=seed)
        rng = np.random.default_rng(seed)
        c.vs *= 2.0 ** rng.integers(-20, 20, size=c.vs.shape)
        c.ks *= 2.0 ** rng.integers(-2, 3, size=c.ks.shape)
        c.ks[::3] *= 1.37                            # scales need not be powers of two
        c.ks, c.vs = c.ks.astype(np.float32).astype(np.float64), (c.vs * 1.1).astype(np.float32).astype(np.float64)
        c.d_ks, c.d_vs = torch.from_numpy(c.ks).float().cuda(), torch.from_numpy(c.vs).float().cuda()
        q, cu, d_cu = pu.queries([1, 1, 2], 4, 128, seed=seed, mult=mult)
        run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("G", [1, 8, 20])
def test_attend_small_values_beside_pages_of_zeros(page, D, G):
    """A page of zeros has scale 1.  Its keys' scores are like the others', and add nothing to O: what the
    others add keeps its accuracy however small their values are."""
    for down in (8, 13, 20, 30, 60, 90):
        lens, counts = [1024, 8 * page, 700, 5 * page + 3], [1, 1, 3, 2]
        c = pu.Cache(lens, 1, page, D, seed=D + page + down)
        c.vs *= 2.0 ** -down
        for b, zero in enumerate(([0, 5], [1, 3, 5, 7], [0, 1, 700 // page], [2])):  # first, in turn, last, inside
            for i in zero:
                c.vc[c.table[b, i]], c.vs[c.table[b, i]] = 0, 1.0
        c.d_vc, c.d_vs = torch.from_numpy(c.vc).cuda(), torch.from_numpy(c.vs).float().cuda()
        q, cu, d_cu = pu.queries(counts, G, D, seed=G, pad=1)
        run_attend(c, q, cu, d_cu, what=f"2^-{down}")
        sel = np.tile(np.array([3, 0, 5, 1, 4]), (4, 1, 1))
        run_attend(c, q, cu, d_cu, sel, np.full((4, 1), 5), what=f"2^-{down}, selected")


@pytest.mark.parametrize("D", [64, 128])
def test_attend_small_values_beside_one_large_value_that_is_hardly_seen(D):
    """A page's scale may come from a token that some queries hardly attend to, while the page's other tokens
    are rounded to 0 beside it."""
    c = pu.Cache([600, 330], 2, 16, D, seed=D)
    c.vs *= 2.0 ** -24
    q, cu, d_cu = pu.queries([1, 1], 2, D, seed=1)
    for b in range(2):
        for h in range(2):
            for i in (2, 9):
                pg = c.table[b, i]
                c.vc[pg, h], c.vs[pg, h] = 0, 1.0
                c.vc[pg, h, 7] = 0x7E                                 # 448 in every column,
                x = pu.f64(q[b, h])
                c.kc[pg, h, 7] = pu.to_e4m3(-x * (64 * D ** 0.5 / (x @ x)) / c.ks[pg, h])  # against the query, as far as codes reach
    c.d_kc, c.d_vc, c.d_vs = torch.from_numpy(c.kc).cuda(), torch.from_numpy(c.vc).cuda(), torch.from_numpy(c.vs).float().cuda()
    o, lse = (pu.f64(x) for x in fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages))
    # A weight w = 2^(x - m + 8) is rounded to fp16: by 2^-11 of itself, or, as a subnormal number, by 2^-25, or by no
    # more than itself.  m is at most the largest score plus the largest value scale so far, and value scales are
    # within 2^4 of that (others are rounded against a maximum of their own), so that 2^-25 of w is at most
    # 2^(-25 - 8 + 4) = 2^-29 of the row's largest softmax weight.  The other terms are check_attend's.
    for b, L in enumerate(c.lens):
        at = c.table[b, :-(-L // 16)]
        for r in range(2):
            h = r
            K, V = ((pu.E4M3[x[at, h]] * s[at, h][:, None, None]).reshape(-1, D)[:L] for x, s in ((c.kc, c.ks), (c.vc, c.vs)))
            s = K @ pu.f64(q[b, r]) * D ** -0.5
            p = np.exp(s - s.max())
            ro, rl, size = p @ V / p.sum(), s.max() + np.log(p.sum()), p @ np.abs(V) / p.sum()
            rounded = np.minimum(p, np.maximum(2.0 ** -11 * p, 2.0 ** -29)) @ np.abs(V) / p.sum()
            x = (1 + np.abs(s).max() * 1.4427) * 2.0 ** -20
            assert (np.abs(o[b, r] - ro) <= 2.0 ** -8 * np.abs(ro) + (rounded + 2 * x * size) * (1 + 2.0 ** -7)).all(), (b, r)
            assert abs(lse[b, r] - rl) <= x + 2.0 ** -22 * abs(rl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [8, 16, 40])
@pytest.mark.parametrize("e", [-90, -58, 0, 60, 110])
def test_attend_lse_does_not_depend_on_the_values_size(D, G, e):
    """LSE is of the scores alone: a value scale's large logarithm takes nothing from it.  All keys are alike, so
    that a row's LSE is its score and the logarithm of how many there are."""
    c = pu.Cache([333, 1], 1, 32, D, seed=G)
    c.kc[:], c.ks[:], c.vs[:] = 0x38, 1.0, 2.0 ** e       # 1.0
    c.d_kc, c.d_ks, c.d_vs = torch.from_numpy(c.kc).cuda(), torch.from_numpy(c.ks).float().cuda(), torch.from_numpy(c.vs).float().cuda()
    q, cu, d_cu = pu.queries([1, 1], G, D, seed=e)
    q[:, :, 1:] = 0.0
    run_attend(c, q, cu, d_cu)


@pytest.mark.parametrize("e", [-100, 112])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_attend_millions_of_extreme_values(D, page, e):
    """The smallest value scale that fa_kv_append gives, 2^-100, at 2^21 keys of one score (the sum of weights
    divided by it passes 2^128), and one near the largest.  O is the mean of the values, LSE is ln 2^21."""
    n = 2 ** 21 // page
    codes = (8 + torch.arange(page, device="cuda") % 100).to(torch.uint8).view(1, 1, page, 1).expand(1, 1, page, D).contiguous()
    q, table = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, n), dtype=torch.int32, device="cuda")
    o, lse = fa.fa_fwd_paged(q, i32([0, 1]), i32([2 ** 21]), table, codes, codes.clone(), torch.ones((1, 1), device="cuda"),
                             torch.full((1, 1), 2.0 ** e, device="cuda"))
    mean = pu.E4M3[8 + np.arange(page) % 100].mean() * 2.0 ** e
    # Scores of 0 give every key the same weight, a power of two, which fp16 holds: what is left are O's rounding to
    # bf16 and fp32 sums, of up to 2^21 / 152 / 8 keys by one warp (2^-24 each at worst, where all round one way)
    assert np.abs(pu.f64(o) / mean - 1).max() <= 2.0 ** -8 + 2.0 ** -24 * 2 ** 21 / 152 / 8
    assert abs(float(lse) - 21 * np.log(2)) <= 2.0 ** -24 * 2 ** 21 / 152 / 8 + 2.0 ** -22 * 15


def test_attend_tiny_and_huge_queries():
    c = pu.Cache([200, 90], 1, 64, 64, seed=11)
    q, cu, d_cu = pu.queries([1, 1], 4, 64, seed=11)
    q[0, 0] *= 2.0 ** -100
    q[0, 1] = 0.0
    q[0, 2] *= 2.0 ** 90
    run_attend(c, q[:1].contiguous(), np.array([0, 1, 1]), i32([0, 1, 1]), scale=2.0 ** -92)
    q[1, 1, 3] = float("nan")                       # one row's NaN stays in that row
    o, lse = fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages)
    assert bool(torch.isnan(o[1, 1]).all()) and bool(torch.isnan(lse[1, 1]))
    assert bool(torch.isfinite(o[1, [0, 2, 3]]).all()) and bool(torch.isfinite(lse[1, [0, 2, 3]]).all())


def test_attend_pages_and_positions_outside_the_cache():
    c = pu.Cache([100, 100, 100, 100], 2, 16, 64, seed=12)
    q, cu, d_cu = pu.queries([1, 1, 2, 1], 4, 64, seed=12)
    c.table[1, 3], c.table[2, 6], c.table[3, 0] = c.num_pages, -1, -2 ** 31
    c.d_table = torch.from_numpy(c.table).cuda()
    run_attend(c, q, cu, d_cu)
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE
    sel = np.tile(np.array([0, 2, 5, 6]), (4, 2, 1))
    sel[0, 0, 1], sel[0, 1, 2] = 7, -1              # behind the sequence, negative
    sel[2, 0, 3], sel[3, 1, 0] = 2 ** 31 - 1, 1
    run_attend(c, q, cu, d_cu, sel, np.full((4, 2), 4))
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE


def test_attend_lengths_past_the_table_are_held_to_it():
    c = pu.Cache([64, 30], 1, 16, 64, seed=13, extra_cols=0)
    q, cu, d_cu = pu.queries([1, 1], 2, 64, seed=13)
    c.lens = [64, -3]
    c.d_lens = i32([2 ** 31 - 1, -3])
    run_attend(c, q, cu, d_cu)
    d_cu = i32([0, 900, 2 ** 31 - 1])               # sums past T: the first sequence has every row
    o, lse = fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages)
    ref = pu.attend(pu.f64(q), np.array([0, 2, 2]), [64, 0], c.table, c.kc, c.vc, c.ks, c.vs, 0.125, 16)
    pu.check_attend(o, lse, ref)


@pytest.mark.parametrize("selected", [False, True])
def test_attend_refuses_tokens_that_pass_their_number_many_times(selected):
    """cu_q that does not ascend, so that every other sequence has all tokens and their work, laid end to end,
    passes what 32 bits count: nothing is written, and the status word says so."""
    B, T, Hkv, page, W = 4000, 600, 8, 128, 9000
    q = torch.zeros((T, Hkv, 64), dtype=torch.bfloat16, device="cuda")
    codes, ones = torch.zeros((1, Hkv, page, 64), dtype=torch.uint8, device="cuda"), torch.ones((1, Hkv), device="cuda")
    o, lse = torch.full_like(q, 777.0), torch.full((T, Hkv), 777.0, device="cuda")
    cu = i32([0, T] * (B // 2) + [0])
    if selected:
        table, sel = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.zeros((B, Hkv, W // 4), dtype=torch.int32, device="cuda")
        extra = dict(sel=sel, sel_count=torch.full((B, Hkv), W // 4, dtype=torch.int32, device="cuda"))
        lens = torch.full((B,), page, dtype=torch.int32, device="cuda")
    else:
        table, extra = torch.zeros((B, W // 4), dtype=torch.int32, device="cuda"), {}
        lens = torch.full((B,), W // 4 * page, dtype=torch.int32, device="cuda")
    fa.fa_fwd_paged(q, cu, lens, table, codes, codes.clone(), ones, ones.clone(), o=o, lse=lse, **extra)
    assert fa.fa_device_status() == fa.FA_ERR_BAD_SHAPE
    assert bool((o == 777).all()) and bool((lse == 777).all())


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of a cache, written and read."""
    Hkv, page, D, N = 8, 128, 128, 34000
    kc, vc = (torch.zeros((N, Hkv, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((N, Hkv), device="cuda") for _ in range(2))
    mean, ms = torch.zeros((N, Hkv, D), dtype=torch.int8, device="cuda"), torch.zeros((N, Hkv), device="cuda")
    table = i32([[N - 1, 32768, 5]])
    x = torch.randn((300, 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    slots = torch.cat([table[0, t // 128] * 128 + t % 128 for t in range(300)][:0] + [table[0].repeat_interleave(128)[:300] * 128 +
                                                                                  torch.arange(300, device="cuda", dtype=torch.int32) % 128])
    fa.fa_kv_append(x[:, :Hkv], x[:, Hkv:], slots.to(torch.int32), kc, vc, ks, vs, mean, ms)
    q, cu, d_cu = pu.queries([2], Hkv * 2, D, seed=3)
    o, lse = fa.fa_fwd_paged(q, d_cu, i32([300]), table, kc, vc, ks, vs)
    at = table[0].long()
    small = [t[at].contiguous() for t in (kc, vc, ks, vs)]
    ref = pu.attend(pu.f64(q), cu, [300], np.array([[0, 1, 2]]), small[0].cpu().numpy(), small[1].cpu().numpy(), pu.f64(small[2]),
                    pu.f64(small[3]), D ** -0.5, page)
    pu.check_attend(o, lse, ref)
    assert bool((ms[at] > 0).all()) and int(mean[at].abs().amax()) == 127
    sel, count = fa.fa_page_select(q, d_cu, i32([300]), table, mean, ms, page, 2, 0, 1)
    rs, _ = pu.select(pu.f64(q), cu, [300], np.array([[0, 1, 2]]), mean[at].cpu().numpy(), ms[at].cpu().numpy(), page, 2, 0, 1)
    assert np.array_equal(sel.cpu().numpy(), rs)


# ------------------------------------------------- streams, graphs, a whole run
class Serving:
    """A serving loop over one cache: host-side copies advance by the plain implementations."""

    def __init__(self, B, Hkv, G, page, D, num_pages, width, seed):
        self.B, self.Hkv, self.G, self.page, self.D, self.N, self.W = B, Hkv, G, page, D, num_pages, width
        self.rng = np.random.default_rng(seed)
        shape = (num_pages, Hkv, page, D)
        self.kc, self.vc = (np.full(shape, 0x7F, np.uint8) for _ in range(2))
        self.ks, self.vs = (np.ones(shape[:2]) for _ in range(2))
        self.mean, self.ms = np.zeros((num_pages, Hkv, D), np.int8), np.zeros(shape[:2], np.float32)
        self.table, self.cached = np.full((B, width), -1), [0] * B
        self.free, self.count = self.rng.permutation(num_pages).tolist(), num_pages
        t = lambda a, dt=None: torch.from_numpy(a).to(device="cuda", dtype=dt)  # noqa: E731
        self.dev = [t(self.kc), t(self.vc), t(self.ks, torch.float32), t(self.vs, torch.float32)]
        self.d_mean, self.d_ms, self.d_table = t(self.mean), t(self.ms), t(self.table, torch.int32)
        self.d_free = i32(self.free)

    def tokens(self, T, seed):
        g = torch.Generator().manual_seed(seed)
        w = torch.randn((T, (self.G + 2) * self.Hkv, self.D), generator=g).to(torch.bfloat16)
        a = self.Hkv * self.G
        return w, (slice(None), slice(0, a)), (slice(None), slice(a, a + self.Hkv)), (slice(None), slice(a + self.Hkv, None))

    def launch(self, cached, new, count, w, slots, top, out, stream=None):
        """One step on the device, into `out`'s tensors."""
        a = self.Hkv * self.G
        q, k, v = w[:, :a], w[:, a:a + self.Hkv], w[:, a + self.Hkv:]
        fa.fa_kv_plan(cached, new, self.d_free, count, self.d_table, self.N, self.page, cu_q=out["cu"], seq_lens=out["lens"], slot_map=slots,
                      free_left=out["left"], stream=stream)
        fa.fa_kv_append(k, v, slots, *self.dev, k_mean=self.d_mean, k_mean_scale=self.d_ms, stream=stream)
        fa.fa_page_select(q, out["cu"], out["lens"], self.d_table, self.d_mean, self.d_ms, self.page, top, 1, 1, sel=out["sel"],
                          sel_count=out["count"], stream=stream)
        fa.fa_fwd_paged(q, out["cu"], out["lens"], self.d_table, *self.dev, o=out["o"], lse=out["lse"], workspace=out["ws"], stream=stream)
        fa.fa_fwd_paged(q, out["cu"], out["lens"], self.d_table, *self.dev, sel=out["sel"], sel_count=out["count"], o=out["os"],
                        lse=out["ls"], workspace=out["ws"], stream=stream)

    def outputs(self, T, top):
        Hq = self.Hkv * self.G
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        return dict(cu=z(self.B + 1), lens=z(self.B), left=z(1), sel=z(self.B, self.Hkv, top), count=z(self.B, self.Hkv),
                    o=z(T, Hq, self.D, dt=torch.bfloat16), os=z(T, Hq, self.D, dt=torch.bfloat16), lse=z(T, Hq, dt=torch.float32),
                    ls=z(T, Hq, dt=torch.float32), ws=z(fa.fa_fwd_paged_workspace_bytes(self.B, T, Hq, self.Hkv, self.D), dt=torch.uint8))

    def check(self, new, w, T, top, out):
        """The same step by the plain implementations, and the comparison."""
        cu, lens, slots, left, self.table = pu.plan(self.cached, new, self.free, self.count, self.table, T, self.N, self.page)
        _, qs, kk, vv = self.tokens(1, 0)
        x = pu.f64(w)
        pu.append(x[kk], slots, self.kc, self.ks, self.page, self.mean, self.ms)
        pu.append(x[vv], slots, self.vc, self.vs, self.page)
        assert out["cu"].tolist() == cu and out["lens"].tolist() == lens and int(out["left"]) == left
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        sel, count = pu.select(x[qs], cu, lens, self.table, self.mean, self.ms, self.page, top, 1, 1)
        assert np.array_equal(out["sel"].cpu().numpy(), sel) and np.array_equal(out["count"].cpu().numpy(), count)
        args = (x[qs], cu, lens, self.table, self.kc, self.vc, self.ks, self.vs, self.D ** -0.5, self.page)
        pu.check_attend(out["o"], out["lse"], pu.attend(*args), "all pages", cu[-1])
        pu.check_attend(out["os"], out["ls"], pu.attend(*args, sel, count), "selected", cu[-1])
        self.cached = [L if L else c for L, c in zip(lens, self.cached)]
        self.count = left


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128)])
def test_serving_run(page, D):
    """Prompts, then decode steps, drafts and a late prompt; pages run out at the end."""
    s = Serving(5, 2, 4, page, D, num_pages=11 + 224 // page, width=2 + 160 // page, seed=page)
    steps = [[40, 3, 90, 0, 17], [1, 1, 1, 0, 1], [1, 0, 1, 30, 1], [3, 1, 2, 1, 4], [1, 1, 1, 1, 1], [20, 20, 20, 60, 20]]
    for i, new in enumerate(steps):
        T = sum(new) + (3 if i % 2 else 0)
        w = s.tokens(T, i)[0]
        out = s.outputs(T, 3)
        s.launch(i32(s.cached), i32(new), i32([s.count]), w.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"), 3, out)
        torch.cuda.synchronize()
        s.check(new, w, T, 3, out)


def test_captured_steps_replayed_with_other_lengths():
    """One graph of a whole step, replayed while the lengths, tokens and free pages change."""
    s = Serving(4, 1, 8, 16, 128, num_pages=60, width=12, seed=1)
    T, top = 64, 4
    w, slots = s.tokens(T, 0)[0].cuda(), torch.zeros(T, dtype=torch.int32, device="cuda")
    cached, new, count, out = i32([0] * 4), i32([0] * 4), i32([60]), s.outputs(T, top)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.launch(cached, new, count, w, slots, top, out, stream=side)   # nothing to do: loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.launch(cached, new, count, w, slots, top, out)
    for i, step in enumerate([[30, 1, 0, 20], [1, 1, 1, 1], [2, 0, 50, 1], [1, 1, 1, 1], [0, 0, 0, 0]]):
        hw = s.tokens(T, 10 + i)[0]
        w.copy_(hw)
        cached.copy_(i32(s.cached)), new.copy_(i32(step)), count.fill_(s.count)
        graph.replay()
        torch.cuda.synchronize()
        s.check(step, hw, T, top, out)


def test_captured_on_forked_streams():
    """A graph whose calls follow copies, fills, one another and other streams' calls."""
    c = pu.Cache([700, 90, 1500], 2, 32, 128, seed=31)
    q, cu, d_cu = pu.queries([1, 3, 1], 16, 128, seed=31)
    k, v = (torch.randn((6, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    free = [i for i in range(c.num_pages) if i not in c.table][:1]
    slots = i32([free[0] * 32 + i for i in range(6)])
    kc, vc, ks, vs = (x.clone() for x in c.pages)
    mean, ms = c.d_mean.clone(), c.d_ms.clone()
    want_pages = tuple(x.clone() for x in (kc, vc, ks, vs, mean, ms))
    fa.fa_kv_append(k, v, slots, *want_pages)
    want_sel = fa.fa_page_select(q, d_cu, c.d_lens, c.d_table, c.d_mean, c.d_ms, 32, 8)
    want = fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages, *want_sel)
    torch.cuda.synchronize()
    q2, sel, n = torch.zeros_like(q), torch.zeros_like(want_sel[0]), torch.zeros_like(want_sel[1])
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(fa.fa_fwd_paged_workspace_bytes(3, q.shape[0], 16, 2, 128), dtype=torch.uint8, device="cuda")
    graph, fork, done = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        q2.copy_(q)
        fork.wait_stream(main)
        with torch.cuda.stream(fork):
            ks.mul_(1.0)
            fa.fa_kv_append(k, v, slots, kc, vc, ks, vs, mean, ms, stream=fork)
            done.record(fork)
        sel.fill_(-9)
        fa.fa_page_select(q2, d_cu, c.d_lens, c.d_table, c.d_mean, c.d_ms, 32, 8, sel=sel, sel_count=n)
        o.zero_()
        main.wait_event(done)
        fa.fa_fwd_paged(q2, d_cu, c.d_lens, c.d_table, kc, vc, ks, vs, sel, n, o=o, lse=lse, workspace=ws)
    for _ in range(3):
        q2.zero_(), o.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sel, want_sel[0]) and torch.equal(n, want_sel[1])
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for got, ref in zip((kc, vc, ks, vs, mean, ms), want_pages):
            assert torch.equal(got, ref)


def test_calls_on_several_streams():
    """Independent calls at the same time, each with its own workspace, give what each gives alone."""
    made = []
    for i in range(4):
        c = pu.Cache([3000 + 100 * i, 17], 2, 64, 128, seed=i)
        q, cu, d_cu = pu.queries([1, 1], 8, 128, seed=i)
        made.append((c, q, d_cu, fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        got = []
        for st, (c, q, d_cu, _) in zip(streams, made):
            st.wait_stream(torch.cuda.current_stream())
            got.append(fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages, stream=st))
        torch.cuda.synchronize()
        for (o, lse), (_, _, _, (ro, rl)) in zip(got, made):
            assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_wrappers_check_their_tensors():
    c = pu.Cache([40], 2, 16, 64, seed=1)
    q, cu, d_cu = pu.queries([1], 4, 64, seed=1)
    ok = dict(q=q, cu_q=d_cu, seq_lens=c.d_lens, block_table=c.d_table, k_pages=c.d_kc, v_pages=c.d_vc, k_scale=c.d_ks, v_scale=c.d_vs)
    fa.fa_fwd_paged(**ok)
    for name, bad in (("q", q.float()), ("q", q[:, :, :32]), ("q", q[0]), ("cu_q", d_cu.long()), ("cu_q", d_cu[:1]), ("seq_lens", c.d_lens.cpu()),
                      ("block_table", c.d_table[0]), ("k_pages", c.d_kc[:, :1]), ("v_pages", c.d_vc.to(torch.int8)), ("k_scale", c.d_ks[:1]),
                      ("v_scale", c.d_vs.double()), ("sel", i32([[[0], [0]]])), ("workspace", torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            fa.fa_fwd_paged(**{**ok, name: bad})
    with pytest.raises(fa.FAError) as e:
        fa.fa_fwd_paged(**ok, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == fa.FA_ERR_WORKSPACE
    with pytest.raises(fa.FAError) as e:
        fa.fa_fwd_paged(**{**ok, "q": torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda")})
    assert e.value.status == fa.FA_ERR_BAD_SHAPE


def test_tensors_without_storage_are_refused():
    """A tensor that has no address raises where it is asked for it; the interpreter goes on."""
    class NoStorage(torch.Tensor):
        @staticmethod
        def __new__(cls, like):
            return torch.Tensor._make_wrapper_subclass(cls, like.shape, dtype=like.dtype, device=like.device)

        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise NotImplementedError(func)

    c = pu.Cache([40], 2, 16, 64, seed=1)
    q, cu, d_cu = pu.queries([1], 4, 64, seed=1)
    for name in ("q", "seq_lens", "k_pages", "o"):
        a = dict(q=q, cu_q=d_cu, seq_lens=c.d_lens, block_table=c.d_table, k_pages=c.d_kc, v_pages=c.d_vc, k_scale=c.d_ks,
                 v_scale=c.d_vs, o=torch.empty_like(q), lse=torch.empty(q.shape[:2], device="cuda"))
        a[name] = NoStorage(a[name])
        with pytest.raises((RuntimeError, ValueError, NotImplementedError)):
            fa.fa_fwd_paged(**a)
    with pytest.raises((RuntimeError, ValueError, NotImplementedError)):
        fa.fa_kv_append(NoStorage(q[:, :2]), q[:, :2], i32([0]), *c.pages)
    run_attend(c, q, cu, d_cu)
