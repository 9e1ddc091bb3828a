"""GPU parity of fa_fwd_paged_chunk against the 64-bit definition, at the lengths, masks and scales where it can go
wrong, and a run of the step that it belongs to (plan with positions, append with rotation, attention)."""
import math
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


def reference(c, q, cu, scale):
    """(O, LSE, the weights' mean of |v|, the largest |score|) of each row, in 64 bits; NaN rows as fa.h says."""
    T, Hq, D = q.shape
    G, page = Hq // c.Hkv, c.page
    o, lse, size, top = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b, L in enumerate(c.lens):
        q0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        if not n:
            continue
        L = min(max(L, 0), c.table.shape[1] * page)
        at = c.table[b, :-(-L // page)].astype(np.int64)
        bad = (at < 0) | (at >= c.num_pages)
        at = np.where(bad, 0, at)
        j = np.arange(L)
        limit = L - n + np.arange(n) + 1
        for h in range(c.Hkv):
            K = (pu.E4M3[c.kc[at, h]] * c.ks[at, h][:, None, None]).reshape(-1, D)[:L]
            V = (pu.E4M3[c.vc[at, h]] * c.vs[at, h][:, None, None]).reshape(-1, D)[:L]
            poison = np.repeat(bad, page)[:L]
            K, V = np.where(poison[:, None], np.nan, K), np.where(poison[:, None], 0.0, V)
            x = q[q0:q0 + n, h * G:(h + 1) * G]
            hidden = j[None, None, :] >= limit[:, None, None]
            with np.errstate(invalid="ignore"):
                s = np.where(hidden, -np.inf, scale * (x @ K.T if L else np.zeros((n, G, 0))))
            for i in range(n):
                if limit[i] <= 0:
                    continue
                y, v = s[i, :, :limit[i]], V[:limit[i]]
                mx = y.max(1, keepdims=True)
                p = np.exp(y - mx)
                l = p.sum(1, keepdims=True)
                rows = (q0 + i, slice(h * G, (h + 1) * G))
                o[rows], lse[rows] = p @ v / l, (mx + np.log(l))[:, 0]
                size[rows], top[rows] = p @ np.abs(np.nan_to_num(v)) / l, np.abs(y).max(1)
    return o, lse, size, top


def check(o, lse, ref, rows, weights=2.0 ** -11, what=""):
    """Tolerances, counted before any run: weights are rounded to fp16, half a step, 2^-11 of each (`weights`: 2^-8 where
    they are bf16), so O by that share of the weights' mean of |v|, and once to bf16, 2^-8 of itself.  Weights below 2^-14 of 2^4 times the one at the maximum in use are steps of 2^-24, off by 2^-29
    of the largest: less than 2^-15 for all of 10^4 keys, of the largest |v|.  Exponents of magnitude x carry a few
    fp32 roundings (2^-24 each), exp2 two units in the last place, log2 likewise: 2^-20 (1 + x)."""
    ro, rl, size, top = (a[:rows] for a in ref)
    o, lse = pu.f64(o)[:rows], pu.f64(lse)[:rows]
    assert np.array_equal(np.isnan(ro), np.isnan(o)), f"{what}: NaN differs"
    assert np.array_equal(np.isnan(rl), np.isnan(lse)) and np.array_equal(np.isinf(rl), np.isinf(lse)), f"{what}: LSE"
    x = (1 + top * 1.4427) * 2.0 ** -20
    biggest = np.nanmax(size, axis=-1, initial=0.0, keepdims=True) if size.size else size
    tol = 2.0 ** -8 * np.abs(ro) + (weights + 2 * x[..., None]) * size * (1 + 2.0 ** -7) + 2.0 ** -13 * biggest + 1e-30
    fine = np.isfinite(ro)
    err = np.abs(o - ro)
    assert (err[fine] <= tol[fine]).all(), f"{what}: O off by {np.max((err / tol)[fine])} of what is allowed"
    fine = np.isfinite(rl)
    with np.errstate(invalid="ignore"):
        el = np.abs(lse - rl)
    tl = x + 2.0 ** -22 * np.abs(np.where(fine, rl, 0))
    assert (el[fine] <= tl[fine]).all(), f"{what}: LSE off by {np.max((el / tl)[fine])} of what is allowed"


def run_chunk(c, q, cu, d_cu, scale=None, weights=2.0 ** -11, what="", **kw):
    T, Hq, D = q.shape
    o = torch.full((T, Hq, D), 777.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 777.0, device="cuda")
    fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages, o=o, lse=lse, scale=scale, **kw)
    torch.cuda.synchronize()
    rows = int(cu[-1])
    assert bool((o[rows:] == 777).all()) and bool((lse[rows:] == 777).all()), "padding rows were written"
    check(o, lse, reference(c, pu.f64(q), cu, scale or D ** -0.5), rows, weights, what)
    return o, lse


def put_back(c):
    """The cache's arrays, changed on the host, on the device."""
    c.d_kc, c.d_vc = torch.from_numpy(c.kc).cuda(), torch.from_numpy(c.vc).cuda()
    c.ks, c.vs = c.ks.astype(np.float32).astype(np.float64), c.vs.astype(np.float32).astype(np.float64)
    c.d_ks, c.d_vs = torch.from_numpy(c.ks).float().cuda(), torch.from_numpy(c.vs).float().cuda()
    c.d_table = torch.from_numpy(np.ascontiguousarray(c.table, np.int32)).cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
def test_one_token(D, page):
    c = pu.Cache([1], 1, page, D, seed=D + page)
    q, cu, d_cu = pu.queries([1], 1, D, seed=page)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 3), (1, 8), (1, 40)])
def test_ragged(D, page, Hkv, G):
    """Lengths around tiles, pages and halves of a tile; more tokens than keys, so that rows see none; no tokens; no keys."""
    lens = [1, 0, 15, 64, 65, 127, 128, 129, 255, 257, 400, 3, 30, 0]
    counts = [1, 0, 15, 20, 65, 1, 100, 2, 130, 257, 33, 7, 31, 2]
    c = pu.Cache(lens, Hkv, page, D, seed=D + page + G)
    q, cu, d_cu = pu.queries(counts, Hkv * G, D, seed=G, pad=3)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,page", [(1, 64), (4, 16), (5, 128)])
def test_prompts(D, G, page):
    """Many items of one head, nothing cached before them, and a chunk behind a cached part."""
    lens, counts = [1000, 700, 513], [1000, 699, 200]
    c = pu.Cache(lens, 2, page, D, seed=D + G)
    q, cu, d_cu = pu.queries(counts, 2 * G, D, seed=G, pad=2)
    o1, l1 = run_chunk(c, q, cu, d_cu)
    o2, l2 = run_chunk(c, q, cu, d_cu)
    assert torch.equal(o1, o2) and torch.equal(l1, l2), "not deterministic"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (37, 4), (64, 1), (130, 2)])
def test_few_rows_of_long_sequences(D, n, G):
    """Items cut over many blocks and joined."""
    c = pu.Cache([20011, 9000], 1, 64, D, seed=n + G)
    q, cu, d_cu = pu.queries([n, n], G, D, seed=n, pad=1)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("page", [16, 128])
def test_many_sequences(page):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 150, size=1500).tolist()
    c = pu.Cache(lens, 1, page, 64, seed=1)
    q, cu, d_cu = pu.queries(rng.integers(0, 4, size=1500).tolist(), 2, 64, seed=2, pad=9)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Batches of any mixture of lengths, tokens and heads: how the work is cut must not show."""
    rng = np.random.default_rng(2000 + seed)
    B = int(rng.choice([1, 2, 3, 17, 60]))
    top = int(rng.choice([20, 300, 2000, 6000 if B < 10 else 1000]))
    Hkv, G, D = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 4, 7, 8, 16])), int(rng.choice([64, 128]))
    page = int(rng.choice(fa.FA_PAGE_SIZES))
    lens = [int(rng.integers(0, 1 + (top if rng.random() < 0.3 else top // 8))) for _ in range(B)]
    most = max(2, 4000 // (B * G))
    counts = [int(rng.integers(0, min(most, L + 3))) if rng.random() < 0.6 else int(rng.choice([0, 1])) for L in lens]
    c = pu.Cache(lens, Hkv, page, D, seed=seed)
    q, cu, d_cu = pu.queries(counts, Hkv * G, D, seed=seed, pad=int(rng.integers(0, 4)))
    run_chunk(c, q, cu, d_cu, what=f"{B} {top} {Hkv} {G} {D} {page}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mult", [4.0, 30.0])
def test_growing_scores(D, mult):
    """Scores of hundreds, and keys that grow towards the sequence's beginning, which is read last: the maximum is taken
    again in many tiles, in their first and in their second half."""
    c = pu.Cache([1500, 777], 2, 32, D, seed=D)
    for b, L in enumerate(c.lens):
        n = -(-L // 32)
        for i, pg in enumerate(c.table[b, :n]):
            c.ks[pg] = 2.0 ** (-9 + (n - i) // 8)
    put_back(c)
    q, cu, d_cu = pu.queries([300, 90], 4, D, seed=D, mult=mult)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
def test_value_scales_near_one_another(D):
    """Pages whose value scales differ by less than fp16's range beside the codes allows."""
    c = pu.Cache([900, 64, 333], 2, 16, D, seed=3)
    c.vs *= 2.0 ** np.random.default_rng(4).integers(-2, 1, size=c.vs.shape)
    put_back(c)
    q, cu, d_cu = pu.queries([150, 64, 5], 4, D, seed=5)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [8, 20, 45])
def test_value_scales_far_apart(D, spread):
    """Weights times value scales as bf16 (2^-8 of each)."""
    c = pu.Cache([900, 64, 333, 2000], 1, 32, D, seed=spread)
    c.vs *= 2.0 ** np.random.default_rng(spread).integers(-spread, spread, size=c.vs.shape)
    put_back(c)
    q, cu, d_cu = pu.queries([150, 64, 5, 40], 2, D, seed=5)
    run_chunk(c, q, cu, d_cu, weights=2.0 ** -8)


@pytest.mark.parametrize("exponent", [-100, 100])
def test_value_scales_at_the_ends(exponent):
    """The smallest and very large scales, and a page of zeros, whose scale is 1, beside small values."""
    c = pu.Cache([700, 90], 1, 32, 128, seed=7)
    c.vs[:] = 2.0 ** exponent
    if exponent < 0:
        c.vs[:] = 2.0 ** -60
        z = c.table[0, 3]
        c.vc[z], c.vs[z] = 0, 1.0
        z = c.table[0, 21]  # the last page: the pass begins with it
        c.vc[z, :, :], c.vs[z] = 0, 1.0
    put_back(c)
    q, cu, d_cu = pu.queries([100, 90], 2, 128, seed=8)
    run_chunk(c, q, cu, d_cu, weights=2.0 ** -8)


def test_scales_that_are_no_powers_of_two():
    """Scores take the rest of the key scale in fp32; weights times the value scale are rounded to bf16, 2^-8 of each."""
    c = pu.Cache([900, 64, 333], 2, 32, 128, seed=9)
    c.ks[::3] *= 1.37
    c.vs[1::3] *= 1.1
    put_back(c)
    q, cu, d_cu = pu.queries([140, 60, 7], 4, 128, seed=9)
    run_chunk(c, q, cu, d_cu, weights=2.0 ** -8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 20])
def test_masked_nan_never_touches_a_row(D, G):
    """NaN codes behind the last key (every Cache holds them), NaN values that only later tokens see, in tiles that the mask
    cuts, NaN values that every row sees, and NaN keys that later tokens see."""
    lens, counts = [400, 170, 129, 700], [300, 160, 40, 200]
    c = pu.Cache(lens, 1, 16, D, seed=D)
    rng = np.random.default_rng(G)
    for b, (L, n) in enumerate(zip(lens, counts)):
        for t in rng.integers(L - n, L, size=4).tolist() + ([5] if b == 3 else []):
            c.vc[c.table[b, t // 16], 0, t % 16, int(rng.integers(0, D))] = 0xFF if t % 2 else 0x7F
        if b == 1:
            t = L - 30
            c.kc[c.table[b, t // 16], 0, t % 16, 3] = 0x7F
    put_back(c)
    q, cu, d_cu = pu.queries(counts, G, D, seed=D)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_scales_that_are_not_finite(what, scale):
    """Only the rows that see a key of such a page are other than finite; the page is in a tile that the mask cuts."""
    c = pu.Cache([300, 200], 2, 16, 128, seed=14)
    page = c.table[0, 15]  # keys 240 .. 255
    (c.ks if what == "k" else c.vs)[page, 1] = scale
    put_back(c)
    q, cu, d_cu = pu.queries([120, 100], 8, 128, seed=14)
    o, lse = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages)
    (c.ks if what == "k" else c.vs)[page, 1] = math.nan  # (where an infinity ends up as NaN, where not, is not looked at)
    with np.errstate(invalid="ignore"):
        ro, rl, size, top = reference(c, pu.f64(q), cu, 128 ** -0.5)
    keep = np.ones((220, 8), bool)
    keep[60:120, 4:] = False
    assert np.array_equal(np.isnan(ro).all(2), ~keep) and not bool(torch.isfinite(o[60:120, 4:]).any())
    got = np.where(keep[..., None], pu.f64(o), 0), np.where(keep, pu.f64(lse), 0)
    want = np.where(keep[..., None], ro, 0), np.where(keep, rl, 0), np.where(keep[..., None], size, 0), np.where(keep, top, 0)
    # weights are bf16 in the tile with the page
    check(*(torch.from_numpy(a) for a in got), want, 220, 2.0 ** -8)


def test_nan_values_in_items_that_are_cut():
    c = pu.Cache([20000], 1, 64, 128, seed=3)
    for t, d in ((19990, 7), (19800, 64), (12345, 100)):
        c.vc[c.table[0, t // 64], 0, t % 64, d] = 0x7F
    put_back(c)
    q, cu, d_cu = pu.queries([250], 1, 128, seed=3)
    run_chunk(c, q, cu, d_cu)


def test_pages_outside_the_cache():
    """Rows that would have read such a page are NaN, others not, and the status word says so."""
    for bad in (-1, 10 ** 9, None):
        c = pu.Cache([300, 200], 2, 16, 64, seed=4)
        c.table[0, 15] = c.num_pages if bad is None else bad  # keys 240 .. 255: only rows from there on see them
        put_back(c)
        q, cu, d_cu = pu.queries([120, 100], 4, 64, seed=4)
        o, lse = run_chunk(c, q, cu, d_cu)
        assert bool(torch.isnan(o[100]).all()) and not bool(torch.isnan(o[50]).any())
        assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE


def test_pages_in_common():
    c = pu.Cache([200, 333, 333], 2, 16, 64, seed=21)
    c.table[1, :12] = c.table[0, :12]
    c.table[2, :21] = c.table[1, :21]
    c.table[2, 3] = c.table[2, 7]
    put_back(c)
    q, cu, d_cu = pu.queries([20, 100, 300], 8, 64, seed=21)
    run_chunk(c, q, cu, d_cu)


def test_lengths_beyond_the_table():
    """Lengths past what a row of the table holds are clamped; negative ones see nothing."""
    c = pu.Cache([64, 96, 32], 1, 32, 64, seed=6, extra_cols=0)
    c.lens = [64, 96, -5]
    c.d_lens = i32([64, 1000, -5])
    q, cu, d_cu = pu.queries([10, 20, 3], 2, 64, seed=6)
    run_chunk(c, q, cu, d_cu)


def test_special_queries():
    """Infinities and NaN in one row's query do not reach another row."""
    c = pu.Cache([300], 1, 32, 128, seed=8)
    q, cu, d_cu = pu.queries([200], 2, 128, seed=8)
    q[17, 0, 5], q[18, 1, 6], q[19, 0, 7] = float("nan"), float("inf"), float("-inf")
    o, lse = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages)
    ref = reference(c, np.nan_to_num(pu.f64(q), nan=0.0, posinf=0.0, neginf=0.0), cu, 128 ** -0.5)
    assert all(bool(torch.isnan(o[t, h]).all()) for t, h in ((17, 0), (18, 1), (19, 0)))
    keep = np.ones((200, 2), bool)
    keep[17, 0] = keep[18, 1] = keep[19, 0] = False
    o[17, 0] = o[18, 1] = o[19, 0] = 0
    assert not bool(torch.isnan(o).any())
    for a in (ref[0], ref[2]):
        a[~keep] = 0
    ok = lse.cpu().numpy()
    assert np.abs(ok - ref[1])[keep].max() < 1e-4
    assert (np.abs(pu.f64(o) - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -9 * ref[2] + 2.0 ** -12)[keep].all()


def test_types_streams_and_workspaces():
    """Codes as float8 tensors, an exact workspace that held other things, streams as objects and addresses."""
    c = pu.Cache([900, 40, 2000], 2, 32, 128, seed=8)
    q, cu, d_cu = pu.queries([100, 20, 1], 8, 128, seed=8)
    o, lse = run_chunk(c, q, cu, d_cu)
    T, Hq, _ = q.shape
    ws = torch.full((fa.fa_fwd_paged_chunk_workspace_bytes(3, T, Hq, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    f8 = [t.view(torch.float8_e4m3fn) for t in c.pages[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream, 0):
        o2, l2 = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *f8, *c.pages[2:], workspace=ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_two_threads():
    c = pu.Cache([900, 3000], 2, 32, 128, seed=8)
    q, cu, d_cu = pu.queries([100, 70], 8, 128, seed=8)
    want = run_chunk(c, q, cu, d_cu)
    torch.cuda.synchronize()
    got, errors = [], []

    def work():
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                r = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages, stream=stream)
            stream.synchronize()
            got.append(r)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(torch.equal(a, b) for r in got for a, b in zip(r, want))


def test_captured_and_replayed_with_other_lengths():
    c = pu.Cache([400, 260, 33], 2, 32, 64, seed=5)
    q, cu, d_cu = pu.queries([100, 50, 33], 4, 64, seed=5, pad=10)
    o = torch.full(q.shape, 777.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 777.0, device="cuda")
    ws = torch.empty(fa.fa_fwd_paged_chunk_workspace_bytes(3, q.shape[0], 4, 2, 64), dtype=torch.uint8, device="cuda")
    call = lambda: fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages, o=o, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for counts, lens in (([100, 50, 33], [400, 260, 33]), ([3, 120, 0], [380, 200, 20]), ([0, 0, 1], [400, 0, 1])):
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        d_cu.copy_(torch.from_numpy(cu))
        c.d_lens.copy_(i32(lens))
        c.lens = lens
        o.fill_(777), lse.fill_(777)
        graph.replay()
        torch.cuda.synchronize()
        rows = int(cu[-1])
        assert bool((o[rows:] == 777).all()) and bool((lse[rows:] == 777).all())
        check(o, lse, reference(c, pu.f64(q), cu, 0.125), rows, what=str(counts))


def test_agrees_with_the_kernel_for_few_tokens():
    """Where both calls apply: their roundings of weights (2^-11) and of O (2^-8) lie between them, each once or twice."""
    c = pu.Cache([500, 3000, 77], 4, 64, 128, seed=11)
    q, cu, d_cu = pu.queries([3, 5, 1], 16, 128, seed=11)
    a, la = fa.fa_fwd_paged(q, d_cu, c.d_lens, c.d_table, *c.pages)
    b, lb = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages)
    _, _, size, _ = reference(c, pu.f64(q), cu, 128 ** -0.5)
    assert (np.abs(pu.f64(a) - pu.f64(b)) <= 2.0 ** -7 * np.abs(pu.f64(a)) + 2.0 ** -9 * size).all()
    assert float((la - lb).abs().max()) < 1e-4


def test_most_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 9, size=8192).tolist()
    c = pu.Cache(lens, 1, 16, 64, seed=2)
    q, cu, d_cu = pu.queries([min(L, 1) for L in lens], 1, 64, seed=2)
    run_chunk(c, q, cu, d_cu)


def test_more_heads_in_a_group_than_an_item_has_rows():
    c = pu.Cache([700, 130], 1, 32, 64, seed=2)
    q, cu, d_cu = pu.queries([3, 2], 300, 64, seed=2)
    run_chunk(c, q, cu, d_cu)


def test_caches_past_32_bits():
    """Pages behind 4 GB of codes."""
    c = pu.Cache([500, 300], 1, 128, 128, seed=12)
    much = 2 ** 32 // (128 * 128) + 50
    first = much - c.num_pages
    big = [torch.zeros((much, 1, 128, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((much, 1), device="cuda") for _ in range(2)]
    for b, s in zip(big + scales, c.pages):
        b[first:] = s
    q, cu, d_cu = pu.queries([100, 50], 4, 128, seed=12)
    want = run_chunk(c, q, cu, d_cu)
    got = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, torch.where(c.d_table >= 0, c.d_table + first, c.d_table), *big, *scales)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_waits_that_give_up():
    """The kernel winds down where its waits run out at once, says so, and the next call is as good as any."""
    c = pu.Cache([3000, 900], 2, 32, 128, seed=8)
    q, cu, d_cu = pu.queries([100, 70], 8, 128, seed=8)
    o, lse = run_chunk(c, q, cu, d_cu)
    ws = torch.empty(fa.fa_fwd_paged_chunk_workspace_bytes(2, 170, 8, 2, 128), dtype=torch.uint8, device="cuda")
    args = (q, d_cu, c.d_lens, c.d_table, *c.pages, torch.empty_like(o), torch.empty_like(lse), ws, 128 ** -0.5)
    assert fa.fa_selftest_paged_chunk_timeout(*args, 0) == fa.FA_OK
    assert fa.fa_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_selftest_paged_chunk_timeout(*args, 2_000_000_001) == fa.FA_ERR_BAD_SHAPE
    o2, lse2 = run_chunk(c, q, cu, d_cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ------------------------------------------------------------- the step
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_step_with_positions_rotation_and_chunks(interleaved):
    """Two prompts come in two chunks each, beside a chat with single tokens: plan, append and attention, against a dense
    softmax over what the cache holds, and rotations applied to the keys that went in."""
    B, page, Hkv, G, D, width, num_pages = 3, 32, 2, 4, 128, 24, 60
    gen = torch.Generator().manual_seed(7)
    phases, amplitude = fa.fa_rope_phases(64, base=500.0, scaling="linear", factor=2.0)
    inv = 500.0 ** (-np.arange(32) / 32) / 2.0
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = i32(list(range(num_pages))), i32([num_pages])
    k_pages, v_pages = (torch.zeros((num_pages, Hkv, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    k_scale, v_scale = (torch.zeros((num_pages, Hkv), device="cuda") for _ in range(2))
    cached = [0, 0, 0]
    past = [[] for _ in range(B)]
    for new in ([300, 120, 1], [170, 200, 1], [1, 1, 1]):
        T = sum(new) + 5
        fused = torch.randn((T, (G + 2) * Hkv, D), generator=gen).to(torch.bfloat16).cuda()
        q, k, v = fused[:, :G * Hkv], fused[:, G * Hkv:-Hkv], fused[:, -Hkv:]
        positions = torch.full((T,), 99, dtype=torch.int32, device="cuda")
        cu, lens, slots, left = fa.fa_kv_plan(i32(cached), i32(new), free, count, table, num_pages, page, num_tokens=T, positions=positions)
        want = [c + i for c, n in zip(cached, new) for i in range(n)] + [-1] * 5
        assert positions.tolist() == want
        turned = fa.fa_kv_append_rope(k, v, positions, phases, slots, k_pages, v_pages, k_scale, v_scale, q=q, interleaved=interleaved, amplitude=amplitude)
        attend = fa.fa_fwd_paged if max(new) == 1 else fa.fa_fwd_paged_chunk
        o, lse = attend(turned, cu, lens, table, k_pages, v_pages, k_scale, v_scale)
        torch.cuda.synchronize()

        def rotate(x, pos):
            a = np.array(pos)[:, None, None] * inv
            y = x.copy()
            i, j = (np.arange(0, 64, 2), np.arange(1, 64, 2)) if interleaved else (np.arange(32), np.arange(32, 64))
            y[..., i], y[..., j] = x[..., i] * np.cos(a) - x[..., j] * np.sin(a), x[..., i] * np.sin(a) + x[..., j] * np.cos(a)
            return y

        kr = rotate(pu.f64(k)[:-5], want[:-5])
        qr = rotate(pu.f64(q)[:-5], want[:-5])
        err = np.abs(pu.f64(turned)[:-5] - qr)
        assert (err <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -20 * np.abs(pu.f64(q)).max()).all()
        at = 0
        for b, n in enumerate(new):
            past[b].append(kr[at:at + n])
            keys = np.concatenate(past[b])
            L = cached[b] + n
            pages = table[b, :-(-L // page)].cpu().numpy()
            K, V = (np.concatenate([(pu.E4M3[pu.codes_of(c)[p]] * pu.f64(s)[p][:, None, None]).transpose(1, 0, 2) for p in pages])[:L]
                    for c, s in ((k_pages, k_scale), (v_pages, v_scale)))
            # a code is off by half a step, 2^-4 of its value (a step of the smallest, 2^-10, times the scale), twice where its page's scale grew
            step = np.concatenate([np.broadcast_to(pu.f64(k_scale)[p][None, :, None], (page, Hkv, 1)) for p in pages])[:L]
            assert (np.abs(K - keys) <= 2.0 ** -3 * 1.07 * np.abs(keys) + 2.0 ** -9 * step).all()
            x = pu.f64(turned)[at:at + n]
            for h in range(Hkv):
                s = np.einsum("ngd,ld->ngl", x[:, h * G:(h + 1) * G], K[:, h]) * D ** -0.5
                s = np.where(np.arange(L)[None, None] > cached[b] + np.arange(n)[:, None, None], -np.inf, s)
                p = np.exp(s - s.max(2, keepdims=True))
                ro, size = (np.einsum("ngl,ld->ngd", p, y) / p.sum(2)[..., None] for y in (V[:, h], np.abs(V[:, h])))
                got = pu.f64(o)[at:at + n, h * G:(h + 1) * G]
                assert (np.abs(got - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * size + 1e-6).all()
                rl = s.max(2) + np.log(p.sum(2))
                assert np.abs(pu.f64(lse)[at:at + n, h * G:(h + 1) * G] - rl).max() < 2e-5 * (1 + math.log(L))
            at += n
        cached = [c + n for c, n in zip(cached, new)]
        count.copy_(left)
