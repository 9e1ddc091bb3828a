"""GPU parity of rotary positions (fa_rope, fa_rope_bwd), of appending with rotation (fa_kv_append_rope) and of the plan's
positions, against plain 64-bit implementations, and a gradient through rotation and attention against differences."""
import numpy as np
import pytest
import torch

import exact_attention_82_gb300 as fa
import paged_util as pu
import rope_util as ru

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert fa.fa_device_status() == fa.FA_OK


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# A result is rounded once to bf16, half a step, 2^-8 of it.  Before that, in fp32: the angle is off by at most 2^-25 half turns
# (2^-23.3 radians) and 2^-32 turns, sine and cosine by two units in the last place (2^-23), the amplitude and two products and
# their sum by half a unit each (2^-24): together less than 2^-21 of the pair's length.
def check_turned(got, want, size, what=""):
    got = pu.f64(got)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size * (1 + 2.0 ** -8) + 1e-38
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{what}: off by {np.max(err / tol)} of what is allowed"


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def phases_of(rot, kw):
    phases, amplitude = fa.fa_rope_phases(rot, **kw)
    f, a = ru.frequencies(rot, **kw)
    return phases, amplitude, f, a


SCALED = [dict(), dict(scaling="yarn", factor=16.0, span=4096), dict(scaling="ntk", factor=4.0, base=500.0)]


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 112), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_packed(D, rot, interleaved, inverse):
    """Columns of a fused projection at positions near, far, repeated and negative; odd counts of tokens and heads."""
    T, Hq, Hk = 77, 7, 3
    phases, amplitude, f, a = phases_of(rot, SCALED[rot % 3])
    fused = normal((T, Hq + 2 * Hk, D), rot)
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hk]
    pos = np.random.default_rng(D).integers(0, 1 << 20, size=T)
    pos[:6] = 0, 1, 2 ** 31 - 1, -1, -70000, pos[7]
    call = fa.fa_rope_bwd if inverse else fa.fa_rope
    before = fused.clone()
    qo, ko = call(q, k, phases, positions=i32(pos.tolist()), interleaved=interleaved, amplitude=amplitude)
    assert torch.equal(fused, before)
    for x, y in ((q, qo), (k, ko)):
        x = pu.f64(x)
        check_turned(y, ru.rotate(x, pos[:, None], f, a, interleaved, inverse), ru.size(x, f, a, interleaved))
        assert np.array_equal(pu.f64(y)[..., rot:], x[..., rot:])


@pytest.mark.parametrize("B,S,Hq,Hk", [(1, 1, 1, 0), (3, 1, 4, 4), (1, 65, 40, 8), (2, 33, 5, 1), (5, 200, 16, 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts(B, S, Hq, Hk, D):
    """[B, H, S, D]: views of a fused [B, S, H, D] into contiguous tensors and back, positions of all kinds, in place."""
    phases, amplitude, f, a = phases_of(D // 2, SCALED[1])
    fused = normal((B, S, Hq + Hk + 1, D), S)
    q = fused[:, :, :Hq].transpose(1, 2)
    k = fused[:, :, Hq:Hq + Hk].transpose(1, 2) if Hk else None
    rng = np.random.default_rng(S)
    for kind in range(3):
        pos = [np.arange(S), rng.integers(0, 9999, size=S), rng.integers(0, 9999, size=(B, S))][kind]
        d_pos = None if kind == 0 else i32(pos.tolist())
        at = np.broadcast_to(pos, (B, S))[:, None, :]
        qo, ko = fa.fa_rope(q, k, phases, positions=d_pos, amplitude=amplitude)
        assert qo.is_contiguous() and (ko is None) == (k is None)
        wq = ru.rotate(pu.f64(q), at, f, a)
        check_turned(qo, wq, ru.size(pu.f64(q), f, a))
        if k is not None:
            check_turned(ko, ru.rotate(pu.f64(k), at, f, a), ru.size(pu.f64(k), f, a))
        # back into a fused tensor, whose last columns stay
        grads = torch.full_like(fused, 3.0)
        out = [grads[:, :, :Hq].transpose(1, 2), grads[:, :, Hq:Hq + Hk].transpose(1, 2) if Hk else None]
        fa.fa_rope_bwd(qo, ko, phases, positions=d_pos, amplitude=amplitude, q_out=out[0], k_out=out[1])
        check_turned(out[0], ru.rotate(pu.f64(qo), at, f, a, inverse=True), ru.size(pu.f64(qo), f, a))
        assert bool((grads[:, :, Hq + Hk:] == 3.0).all())
        # in place, inside the fused tensor
        same = fused.clone()
        q2 = same[:, :, :Hq].transpose(1, 2)
        k2 = same[:, :, Hq:Hq + Hk].transpose(1, 2) if Hk else None
        fa.fa_rope(q2, k2, phases, positions=d_pos, amplitude=amplitude, q_out=q2, k_out=k2)
        assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko)) and torch.equal(same[:, :, Hq + Hk:], fused[:, :, Hq + Hk:])


def test_broadcast_input():
    """An input may have strides of 0: one head's rows for all."""
    phases, amplitude, f, a = phases_of(64, {})
    q = normal((2, 1, 20, 64), 5).expand(2, 6, 20, 64)
    qo, _ = fa.fa_rope(q, None, phases)
    check_turned(qo, ru.rotate(pu.f64(q), np.arange(20), f), ru.size(pu.f64(q), f))


def test_special_values_stay_in_their_pair():
    phases, _, f, _ = phases_of(128, {})
    q = normal((9, 2, 128), 1)
    q[4, 1, 3], q[5, 0, 70] = float("nan"), float("inf")
    out, _ = fa.fa_rope(q, None, phases)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[4, 1, 3], [4, 1, 67], [5, 0, 6], [5, 0, 70]]


def test_streams_and_capture():
    phases, amplitude, f, a = phases_of(128, {})
    q, k = normal((50, 8, 128), 2), normal((50, 2, 128), 3)
    pos = i32(list(range(50)))
    want = [t.clone() for t in fa.fa_rope(q, k, phases, positions=pos)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        got = fa.fa_rope(q, k, phases, positions=pos, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = [torch.zeros_like(q), torch.zeros_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, k, phases, positions=pos, q_out=out[0], k_out=out[1])
        fa.fa_rope_bwd(out[0], out[1], phases, positions=pos, q_out=out[0], k_out=out[1])
    pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((q, k), out):  # there and back: two roundings
        x = pu.f64(x)
        assert (np.abs(pu.f64(y) - x) <= 2.0 ** -8 * np.abs(x) + 2.0 ** -7 * ru.size(x, f)).all()


def test_wrapper_refusals():
    phases, _ = fa.fa_rope_phases(64)
    q, k = normal((10, 4, 64), 1), normal((10, 2, 64), 2)
    for bad in (dict(positions=i32([1] * 9)), dict(positions=torch.zeros(10, dtype=torch.int64, device="cuda")), dict(q_out=torch.empty_like(q).float()),
                dict(q_out=torch.empty((10, 3, 64), dtype=torch.bfloat16, device="cuda")), dict(k_out=torch.empty((9, 2, 64), dtype=torch.bfloat16, device="cuda")),
                dict(amplitude="x")):
        with pytest.raises(ValueError):
            fa.fa_rope(q, k, phases, **bad)
    with pytest.raises(ValueError):
        fa.fa_rope(q, k, phases.cpu())
    with pytest.raises(ValueError):
        fa.fa_rope(q, k, torch.zeros(65, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        fa.fa_rope(q.transpose(1, 2), None, phases)
    with pytest.raises(ValueError):
        fa.fa_rope(q, k[:, :, :32], phases)
    with pytest.raises(fa.FAError):
        fa.fa_rope(q, k, phases[:5].contiguous())
    with pytest.raises(fa.FAError):
        fa.fa_rope(q, k, phases, q_out=q[:, :, :], k_out=q[:, :2])


def test_gradient_through_attention():
    """dq and dk of sum(dO . attention(rope(q), rope(k), v)) by fa_bwd and fa_rope_bwd: the rotation's share against the formula, and the whole
    against differences of a 64-bit forward in random directions."""
    B, H, S, D = 1, 2, 150, 64
    phases, amplitude, f, a = phases_of(32, {})
    q, k, v, do = (normal((B, H, S, D), s) for s in range(4))
    qr, kr = fa.fa_rope(q, k, phases, interleaved=True)
    o, lse = fa.fa_fwd(qr, kr, v, causal=True)
    dqr, dkr, _ = fa.fa_bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk = fa.fa_rope_bwd(dqr, dkr, phases, interleaved=True)
    at = np.arange(S)
    for g, gr in ((dq, dqr), (dk, dkr)):
        x = pu.f64(gr)
        check_turned(g, ru.rotate(x, at, f, 1.0, True, inverse=True), ru.size(x, f, 1.0, True))
    mask = np.triu(np.ones((S, S), bool), 1)
    vn, don = pu.f64(v), pu.f64(do)

    def loss(qn, kn):
        s = ru.rotate(qn, at, f, 1.0, True) @ ru.rotate(kn, at, f, 1.0, True).swapaxes(2, 3) * D ** -0.5
        s = np.where(mask, -np.inf, s)
        p = np.exp(s - s.max(3, keepdims=True))
        return ((p / p.sum(3, keepdims=True)) @ vn * don).sum()

    qn, kn = pu.f64(q), pu.f64(k)
    rng = np.random.default_rng(1)
    for i in range(4):
        uq, uk = rng.standard_normal(qn.shape), rng.standard_normal(kn.shape)
        h = 1e-4
        diff = (loss(qn + h * uq, kn + h * uk) - loss(qn - h * uq, kn - h * uk)) / (2 * h)
        got = (uq * pu.f64(dq)).sum() + (uk * pu.f64(dk)).sum()
        # fa_bwd's own tolerance is 2% of the largest gradient an element, in random directions: its root mean square
        # over all elements, which add up with random signs, within four deviations
        size = np.sqrt((pu.f64(dq) ** 2).sum() + (pu.f64(dk) ** 2).sum())
        assert abs(diff - got) <= 4 * 0.02 * size, (diff, got, size)


# -------------------------------------------------------------- plan's positions
def test_plan_positions():
    cached, new = [5, -4, 9, 30, 3, 0, 0], [20, 9, 12, 40, 2, 0, 30]
    table = [[3, -1, -1], [-1] * 3, [40, -1, -1], [2, 6, -1], [-9, -1, -1], [-1] * 3, [-1] * 3]
    for T in (118, 60, 1):
        t1, t2 = i32(table), i32(table)
        args = (i32(cached), i32(new), i32([10, 11, 9, 8, 12, 13]), i32([6]))
        pos = torch.full((T,), 55, dtype=torch.int32, device="cuda")
        a = fa.fa_kv_plan(*args, t1, 30, 16, num_tokens=T)
        b = fa.fa_kv_plan(*args, t2, 30, 16, num_tokens=T, positions=pos)
        assert all(torch.equal(x, y) for x, y in zip((*a, t1), (*b, t2)))
        want = [max(c, 0) + i for c, n in zip(cached, new) for i in range(max(n, 0))] + [-1] * T
        assert pos.tolist() == want[:T]
    with pytest.raises(ValueError):
        fa.fa_kv_plan(*args, t1, 30, 16, num_tokens=9, positions=pos[:1].expand(8))


# ------------------------------------------------------------ append with rotation
def values(codes, scale):
    return pu.E4M3[codes] * scale[..., None, None]


def run_append(lens, new, Hkv, page, D, rot, seed, interleaved=False, pad=0, means=False, G=2, gap=False, change=None, kw=SCALED[1]):
    """Appends `new` tokens behind `lens` cached ones.  V and everything that a code does not decide is compared exactly; a key's code may be the
    neighbour's where the rotated value lies within the rotation's error of the border between them, and a scale the next where the largest does."""
    c = pu.Cache([x + y for x, y in zip(lens, new)], Hkv, page, D, seed)
    rng = np.random.default_rng(seed)
    T = sum(new) + pad
    phases, amplitude, f, a = phases_of(rot, kw)
    slots = np.array([int(c.table[b, t // page]) * page + t % page for b, (x, n) in enumerate(zip(lens, new)) for t in range(x, x + n)] + [-1] * pad, np.int32)
    pos = np.array([t for x, n in zip(lens, new) for t in range(x, x + n)] + [0] * pad) + 100_000
    if gap:
        slots[rng.integers(0, T, size=max(1, T // 9))] = -1
    gen = torch.Generator().manual_seed(seed)
    H = (G + 2) * Hkv
    fused = (torch.randn((T, H, D), generator=gen) * torch.exp(torch.randn((T, H, 1), generator=gen))).to(torch.bfloat16)
    if change:
        change(fused[:, G * Hkv:])
    dev = fused.cuda()
    q, k, v = dev[:, :G * Hkv], dev[:, G * Hkv:-Hkv], dev[:, -Hkv:]
    old = dict(kc=c.kc.copy(), ks=c.ks.copy())
    out = fa.fa_kv_append_rope(k, v, i32(pos.tolist()), phases, torch.from_numpy(slots).cuda(), *c.pages, k_mean=c.d_mean if means else None,
                               k_mean_scale=c.d_ms if means else None, q=q if G else None, interleaved=interleaved, amplitude=amplitude)
    torch.cuda.synchronize()
    if G:
        qn = pu.f64(q)
        check_turned(out, ru.rotate(qn, pos[:, None], f, a, interleaved), ru.size(qn, f, a, interleaved), "q")
    else:
        assert out is None
    pu.append(pu.f64(v), slots, c.vc, c.vs, page)
    got = pu.codes_of(c.d_vc)
    assert ((got == c.vc) | (np.isnan(pu.E4M3[got]) & np.isnan(pu.E4M3[c.vc]))).all() and np.array_equal(pu.f64(c.d_vs), c.vs)
    kn = pu.f64(k)
    with np.errstate(invalid="ignore"):
        turned, size = ru.rotate(kn, pos[:, None], f, a, interleaved), ru.size(kn, f, a, interleaved)
    kc, ks = pu.codes_of(c.d_kc), pu.f64(c.d_ks)
    rc, rs = old["kc"].copy(), old["ks"].copy()
    pu.append(turned, slots, rc, rs, page)
    # where a scale differs, the largest rotated key is within its error of what the smaller one holds
    for pg, h in np.argwhere(ks != rs):
        rows = [t for t in range(T) if slots[t] // page == pg and slots[t] >= 0]
        top = np.abs(turned[rows, h]).max()
        border = 448.0 * min(ks[pg, h], rs[pg, h])
        assert abs(top - border) <= 2.0 ** -20 * np.abs(size[rows, h]).max() and max(ks[pg, h], rs[pg, h]) == 2 * min(ks[pg, h], rs[pg, h])
    same = ks == rs
    assert same.mean() > 0.99
    x, y = values(kc, ks), values(rc, rs)
    differ = (kc != rc) & ~(np.isnan(x) & np.isnan(y)) & same[..., None, None] & ~((x == 0) & (y == 0))
    where = {int(s): t for t, s in enumerate(slots) if s >= 0}
    for pg, h, r, d in np.argwhere(differ):
        t = where[int(pg) * page + int(r)]  # a row that was written: the others are compared exactly
        mid = (x[pg, h, r, d] + y[pg, h, r, d]) / 2
        assert abs(int(kc[pg, h, r, d] & 0x7F) - int(rc[pg, h, r, d] & 0x7F)) <= 1
        assert abs(turned[t, h, d] - mid) <= 2.0 ** -20 * size[t, h, d], (turned[t, h, d], mid)
    if means:  # of the codes that are there, exactly
        f32 = np.float32
        t = 0
        mean, ms = c.d_mean.cpu().numpy(), c.d_ms.cpu().numpy()
        for t in range(T):
            s = int(slots[t])
            if s < 0 or (t + 1 < T and slots[t + 1] == s + 1 and (s + 1) % page):
                continue
            pg, rows = s // page, s % page + 1
            for h in range(Hkv):
                w = pu.E4M3[kc[pg, h, :rows]]
                S = (np.where(np.isnan(w), 0.0, w) * 512).sum(0)
                A = np.abs(S).max()
                inv = f32(127) / f32(A) if A > 0 else f32(0)
                assert np.array_equal(mean[pg, h], np.rint(S.astype(f32) * inv).astype(np.int8))
                assert ms[pg, h] == (f32(A) * (f32(ks[pg, h]) * f32(1 / 512))) / f32(127 * rows)
    return c


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 48), (128, 128)])
@pytest.mark.parametrize("page", fa.FA_PAGE_SIZES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_ragged(page, D, rot, interleaved):
    lens = [0, 0, 5, page - 1, page, 3 * page + 1, 2 * page - 1, 0, 7]
    new = [1, 2 * page + 3, 1, 1, 1, page - 1, 2, page, 0]
    run_append(lens, new, 3, page, D, rot, seed=page + D, interleaved=interleaved, pad=5, means=True)


def test_append_shapes():
    run_append([i * 3 for i in range(100)], [1] * 100, 2, 64, 128, 128, seed=1)
    run_append([0], [1500], 1, 64, 64, 64, seed=2, G=0)
    run_append([17], [1500], 2, 16, 128, 64, seed=3, pad=100, G=4, interleaved=True)
    run_append([0, 9], [1, 1], 1, 128, 64, 32, seed=4, means=True, G=1)
    run_append([3, 40, 0, 11, 16, 20] * 4, [1] * 24, 2, 32, 64, 64, seed=6, gap=True, means=True)


def test_append_a_window_for_each_sm():
    """As many tokens as make a block look after all runs of its tokens: prompts, and a few tokens each of many requests."""
    run_append([50, 0], [6000, 4100], 1, 128, 128, 128, seed=11, G=2)
    run_append([0, 7], [6000, 4100], 5, 64, 64, 32, seed=13, G=1, interleaved=True)
    run_append([33], [10000], 1, 32, 128, 64, seed=14, G=0)
    run_append([i * 7 % 40 for i in range(2600)], [4] * 2600, 1, 16, 64, 64, seed=12, G=1, pad=9, means=True)


def test_append_agrees_with_append_where_nothing_turns():
    """At position 0 a rotation is the identity: the very same codes, scales and means."""
    c1, c2 = pu.Cache([40, 200, 3], 2, 32, 128, seed=9), pu.Cache([40, 200, 3], 2, 32, 128, seed=9)
    T = 243
    x = normal((T, 4, 128), 10)
    slots = i32([int(c1.table[b, t // 32]) * 32 + t % 32 for b, L in enumerate(c1.lens) for t in range(L)])
    phases, _ = fa.fa_rope_phases(128)
    fa.fa_kv_append(x[:, :2], x[:, 2:], slots, *c1.pages, k_mean=c1.d_mean, k_mean_scale=c1.d_ms)
    fa.fa_kv_append_rope(x[:, :2], x[:, 2:], torch.zeros_like(slots), phases, slots, *c2.pages, k_mean=c2.d_mean, k_mean_scale=c2.d_ms)
    for a, b in zip((*c1.pages, c1.d_mean, c1.d_ms), (*c2.pages, c2.d_mean, c2.d_ms)):
        assert torch.equal(a, b)


def test_append_special_values():
    """Zeros, infinities and NaN among keys: their pair is infinite or NaN too, scales come from what is finite."""
    def change(w):
        w[0] = 0.0
        w[1, :, 3] = float("inf")
        w[2, :, 5] = float("nan")
        w[3] = 2.0 ** -120
    c = run_append([0, 16, 0], [1, 3, 30], 2, 16, 64, 0 or 32, seed=12, means=False, change=change)
    kc = pu.codes_of(c.d_kc)
    pg = c.table[1, 1]
    nan = np.isnan(pu.E4M3[kc[pg, 0, 1]])
    assert nan.nonzero()[0].tolist() == [5, 21]


def test_append_slots_outside_the_cache():
    c = pu.Cache([40], 1, 16, 64, seed=5)
    before = [t.clone() for t in c.pages]
    x = normal((3, 1, 64), 1)
    phases, _ = fa.fa_rope_phases(64)
    fa.fa_kv_append_rope(x, x, i32([1, 2, 3]), phases, i32([c.num_pages * 16, 2 ** 31 - 1, -5]), *c.pages)
    assert fa.fa_device_status() == fa.FA_ERR_BAD_PAGE
    assert all(torch.equal(a, b) for a, b in zip(before, c.pages))


def test_append_in_place_queries_and_streams():
    c = pu.Cache([90], 2, 16, 128, seed=5)
    phases, _, f, _ = phases_of(128, {})
    fused = normal((90, 8, 128), 3)
    slots = i32([int(c.table[0, t // 16]) * 16 + t % 16 for t in range(90)])
    pos = i32(list(range(90)))
    want = pu.f64(fused[:, :4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = fused[:, :4]
    out = fa.fa_kv_append_rope(fused[:, 4:6], fused[:, 6:], pos, phases, slots, *c.pages, q=q, q_out=q, stream=side)
    torch.cuda.synchronize()
    assert out.data_ptr() == q.data_ptr()
    check_turned(q, ru.rotate(want, np.arange(90)[:, None], f), ru.size(want, f))
