"""fa_fwd_paged_chunk at the edges of what fa.h defines: far more tokens than keys, last tiles without a page that can be
read, scores that vanish, scales far apart, and waits that give up."""
import math

import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import paged_util as pu
from test_gpu_paged_chunk import check, put_back, reference, run_chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert fa.fa_device_status() == fa.FA_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L,Hkv", [(3841, 462, 1), (6397, 1125, 1), (4117, 475, 2), (6128, 871, 1)])
def test_thousands_of_tokens_more_than_keys(n, L, Hkv, D):
    """Most rows see no key, and the blocks' shares are by far longer than the few tiles of the rows that do: cuts that fall on
    the same tile (on 152 SMs; a replay of the cuts found the sizes).  The workspace holds what an earlier call may have left."""
    c = pu.Cache([L], Hkv, 64, D, seed=n)
    q, cu, d_cu = pu.queries([n], Hkv, D, seed=L)
    ws = torch.full((fa.fa_fwd_paged_chunk_workspace_bytes(1, n, Hkv, Hkv, D) // 4,), 3.0, device="cuda").view(torch.uint8)
    run_chunk(c, q, cu, d_cu, workspace=ws)


def reached(c, q, cu, d_cu, hidden_from, heads, weights):
    """Rows of sequence 0 from token hidden_from on and of `heads` are other than finite; all others are as the definition has them."""
    o, lse = fa.fa_fwd_paged_chunk(q, d_cu, c.d_lens, c.d_table, *c.pages)
    T, Hq, _ = q.shape
    with np.errstate(invalid="ignore"):
        ref = reference(c, pu.f64(q), cu, q.shape[2] ** -0.5)
    keep = np.ones((T, Hq), bool)
    keep[hidden_from:int(cu[1]), heads] = False
    assert np.array_equal(np.isnan(ref[0]).all(2), ~keep), "the test's own definition"
    assert not np.isfinite(pu.f64(o))[~keep].any(), "rows that see the page"
    got = np.where(keep[..., None], pu.f64(o), 0), np.where(keep, pu.f64(lse), 0)
    want = [np.where(keep[..., None] if a.ndim == 3 else keep, a, 0) for a in ref]
    check(*(torch.from_numpy(a) for a in got), want, T, weights)


# The last tile's only page: pages of a whole tile, and sequences whose last tile has one page.
ONLY_PAGES = [(128, 300), (64, 300), (16, 260), (32, 385), (16, 513)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,L", ONLY_PAGES)
@pytest.mark.parametrize("bad", [-1, 10 ** 9])
def test_a_last_tile_without_a_page(page, L, D, bad):
    """Rows that would read the page are NaN; earlier ones of the same 256 rows do not see it and are as ever."""
    for G, n in ((1, 250), (4, 60)):
        c = pu.Cache([L, 200], 2, page, D, seed=L + G)
        last = (L - 1) // page
        c.table[0, last] = bad
        put_back(c)
        q, cu, d_cu = pu.queries([n, 100], 2 * G, D, seed=L)
        reached(c, q, cu, d_cu, last * page - (L - n), slice(None), 2.0 ** -11)
        assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,L", ONLY_PAGES)
@pytest.mark.parametrize("what,scale", [("k", math.nan), ("v", math.nan), ("v", math.inf)])
def test_a_last_tile_whose_scale_is_not_finite(page, L, what, scale, D):
    last_scale(page, L, what, scale, D)


def last_scale(page, L, what, scale, D):
    for G, n in ((1, 250), (4, 60)):
        c = pu.Cache([L, 200], 2, page, D, seed=L + G)
        last = (L - 1) // page
        scales = c.ks if what == "k" else c.vs
        scales[c.table[0, last], 1] = scale
        put_back(c)
        q, cu, d_cu = pu.queries([n, 100], 2 * G, D, seed=L)
        scales = c.ks if what == "k" else c.vs
        scales[c.table[0, last], 1] = math.nan  # (where an infinity ends up as NaN, where not, is not looked at)
        reached(c, q, cu, d_cu, last * page - (L - n), slice(G, 2 * G), 2.0 ** -11)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,L", ONLY_PAGES)
def test_keys_whose_scale_is_infinite(page, L, D):
    """A row that sees such keys is other than finite whatever the sign of its products with their codes."""
    last_scale(page, L, "k", math.inf, D)


def test_no_page_at_all():
    """Every page of a sequence lies outside the cache: its rows are NaN, its neighbour's are not."""
    c = pu.Cache([700, 300], 1, 128, 128, seed=3)
    c.table[0, :] = -1
    put_back(c)
    q, cu, d_cu = pu.queries([200, 200], 2, 128, seed=3)
    o, _ = run_chunk(c, q, cu, d_cu)
    assert bool(torch.isnan(o[:200]).all()) and not bool(torch.isnan(o[200:]).any())
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_exponent,k_exponent", [(-60, -100), (-120, -20), (-126, -126), (0, -126)])
def test_scores_that_vanish(q_exponent, k_exponent, D):
    """Queries times key scales below fp32: all scores are 0, and a row is the mean of the values that it sees."""
    c = pu.Cache([400, 90], 2, 32, D, seed=D)
    c.ks[:] = 2.0 ** k_exponent
    put_back(c)
    q, cu, d_cu = pu.queries([300, 90], 4, D, seed=D, mult=2.0 ** q_exponent)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("first", ["small", "large"])
def test_value_scales_apart_by_all_that_is_allowed(first):
    """Pages whose value scales differ by 2^100, the pass beginning at either end, behind 60,000 equally weighted keys: in fp32 the
    largest's sum in units of the smallest is infinite.  160 items, so that most are a block's from end to end."""
    L, page, Hkv, G, D, B, n = 60000, 128, 32, 32, 64, 5, 8
    pages = -(-L // page)
    near, far = (2.0 ** -60, 2.0 ** 40) if first == "small" else (2.0 ** 40, 2.0 ** -60)
    codes = torch.full((pages, Hkv, page, D), 0x7E, dtype=torch.uint8, device="cuda")  # 448
    codes[:, :, :, 1::2] = 0xFE  # -448
    k_pages = torch.zeros_like(codes)
    scale = torch.full((pages, Hkv), far, device="cuda")
    scale[-1] = near  # the pass begins with it
    if first == "large":
        codes[-1] = 0  # (else nothing of the others would be seen)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1).contiguous()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    q = torch.zeros((B * n, Hkv * G, D), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_fwd_paged_chunk(q, cu, lens, table, k_pages, codes, torch.ones_like(scale), scale)
    # all weights alike: the mean over the keys that a row sees, of which those in the last page count for nothing
    keys = L - n + 1 + torch.arange(n, device="cuda", dtype=torch.float64)
    want = (448.0 * far * (pages - 1) * page / keys).repeat(B)[:, None, None] * torch.tensor([1.0, -1.0], device="cuda").double().repeat(D // 2)
    assert bool(torch.isfinite(o).all())
    # weights are powers of two and sums of 448 times fewer than 2^16 keys are exact, so O has its one rounding, 2^-8, and a division's
    # and a product's in fp32
    assert float(((o.double() - want).abs() / want.abs()).max()) <= 2.0 ** -8 + 2.0 ** -20
    assert float((lse.double() - torch.log(keys).repeat(B)[:, None]).abs().max()) <= 2.0 ** -20 * 12


@pytest.mark.parametrize("D", [64, 128])
def test_weights_keep_their_bits_where_scales_are_no_powers_of_two(D):
    """A quantiser that divides by its largest / 448: weights are rounded to fp16 as ever."""
    c = pu.Cache([900, 64, 333, 5000], 2, 32, D, seed=9)
    rng = np.random.default_rng(D)
    c.ks *= rng.uniform(1, 2, size=c.ks.shape)
    c.vs *= rng.uniform(1, 2, size=c.vs.shape)
    put_back(c)
    q, cu, d_cu = pu.queries([140, 60, 7, 20], 4, D, seed=9)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [16, 30, 60])
def test_keys_keep_their_bits_beside_larger_ones(spread, D):
    """Pages of keys 2^spread below others of the same tile, and queries that make their scores count: what a row's later keys
    are must not show in its scores."""
    c = pu.Cache([400, 300], 1, 16, D, seed=spread)
    c.ks[:] = 2.0 ** (-7 - spread)
    big = c.table[0, 22]  # keys 352 .. 367: of zeros, so that rows that see them have a score of 0 there
    c.ks[big], c.kc[big] = 2.0 ** -7, 0
    put_back(c)
    q, cu, d_cu = pu.queries([120, 100], 2, D, seed=D, mult=2.0 ** spread)
    run_chunk(c, q, cu, d_cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,counts", [([3000, 900], [100, 70]), ([1], [1]), ([20000], [1])])
def test_no_time_at_all(lens, counts, D):
    """With a limit of 0 no wait is tried, so that the kernel winds down whatever the hardware's waits do, every time."""
    c = pu.Cache(lens, 2, 32, D, seed=8)
    q, cu, d_cu = pu.queries(counts, 8, D, seed=8)
    o, lse = run_chunk(c, q, cu, d_cu)
    ws = torch.empty(fa.fa_fwd_paged_chunk_workspace_bytes(len(lens), sum(counts), 8, 2, D), dtype=torch.uint8, device="cuda")
    args = (q, d_cu, c.d_lens, c.d_table, *c.pages, torch.empty_like(o), torch.empty_like(lse), ws, D ** -0.5)
    for _ in range(20):
        assert fa.fa_selftest_paged_chunk_timeout(*args, 0) == fa.FA_OK
        assert fa.fa_device_status() == fa.FA_ERR_TIMEOUT
    o2, lse2 = run_chunk(c, q, cu, d_cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
