"""Plain 64-bit implementations of the paged 8-bit cache's operators, in numpy and
with loops, and the inputs their tests share.  They follow the definitions in
include/fa.h and use nothing of the library."""
import math

import numpy as np
import torch


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if s else x
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]  # 0 .. 448, ascending


def to_e4m3(x):
    """float64 -> e4m3 codes: nearest, ties to the even code, held to +-448; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.searchsorted(_POS, a)
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = np.where(np.signbit(x), c | 0x80, c)
    return np.where(np.isnan(x), 0x7F, c).astype(np.uint8)


def pow2_scale(amax: float) -> float:
    if not amax > 0:
        return 1.0
    m, e = math.frexp(amax / 448.0)
    return 2.0 ** max(-100, min(120, e - 1 if m == 0.5 else e))


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def codes_of(t: torch.Tensor) -> np.ndarray:
    return t.detach().view(torch.uint8).cpu().numpy()


# -------------------------------------------------------------------- plan
def plan(cached, new, free, count, table, T, num_pages, page):
    """(cu_q, seq_lens, slot_map, left, table) as fa.h defines them."""
    table = np.array(table)
    B, width = table.shape
    cu, lens, slots, taken, asked = [0], [], [-1] * T, 0, 0
    count = max(0, min(count, len(free)))
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        valid = c >= 0 and n >= 0 and c + n <= width * page
        held = -(-max(c, 0) // page)
        need = -(-(c + n) // page) - held if valid else 0
        asked += need
        served = valid and (need == 0 or asked <= count)
        if served:
            for i in range(need):
                table[b, held + i] = free[count - 1 - (asked - need + i)]
            taken = max(taken, asked if need else 0)
            for i in range(n):
                t, pos = cu[-1] + i, c + i
                pg = table[b, pos // page]
                if t < T and 0 <= pg < num_pages:
                    slots[t] = pg * page + pos % page
        lens.append(c + n if served else 0)
        cu.append(cu[-1] + max(n, 0))
    return [min(x, T) for x in cu], lens, slots, count - taken, table


# ------------------------------------------------------------------ append
def append(x, slots, codes, scale, page, mean=None, mean_scale=None):
    """Writes the tokens x [T, Hkv, D] (float64) into codes / scale (and the means), in place."""
    T, Hkv, D = x.shape
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= codes.shape[0] * page:
            t += 1
            continue
        pg, off, n = s // page, s % page, 1
        while t + n < T and slots[t + n] == s + n and off + n < page:
            n += 1
        for h in range(Hkv):
            y = x[t:t + n, h]
            fine = np.abs(y[np.isfinite(y)])
            sc = pow2_scale(fine.max() if fine.size else 0.0)
            was = float(scale[pg, h])
            if off:
                sc = max(sc, was)
                if sc != was:
                    codes[pg, h, :off] = to_e4m3(E4M3[codes[pg, h, :off]] * (was / sc))
            scale[pg, h] = sc
            codes[pg, h, off:off + n] = to_e4m3(y / sc)
            if mean is not None:
                v = E4M3[codes[pg, h, :off + n]]
                S = (np.where(np.isnan(v), 0.0, v) * 512).sum(0)  # whole numbers
                A = np.abs(S).max()
                f = np.float32
                inv = f(127) / f(A) if A > 0 else f(0)
                mean[pg, h] = np.rint(S.astype(f) * inv).astype(np.int8)
                mean_scale[pg, h] = (f(A) * (f(sc) * f(1 / 512))) / f(127 * (off + n))
        t += n


# ------------------------------------------------------------------ select
def select(q, cu, lens, table, mean, mean_scale, page, top_k, first, last):
    """(sel, count) with scores as fa.h defines them (products in 32 bits, sums in whole numbers)."""
    f = np.float32
    num_pages, Hkv, D = mean.shape
    B, G = len(lens), q.shape[1] // Hkv
    sel, count = np.full((B, Hkv, top_k), -1), np.zeros((B, Hkv), int)
    for b in range(B):
        n = -(-min(max(int(lens[b]), 0), table.shape[1] * page) // page)
        for h in range(Hkv):
            rows = q[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, D).astype(f)
            if not len(rows):
                continue
            rows = np.where(np.isfinite(rows), rows, f(0))
            amax = np.abs(rows).max(1)
            inv = np.array([f(127) / a if a > 0 else f(0) for a in amax], f)
            q8 = np.rint(rows * inv[:, None]).astype(np.int64)
            score = []
            for i in range(n):
                pg = table[b, i]
                if i < first or i >= n - last:
                    score.append(math.inf)
                elif not 0 <= pg < num_pages:
                    score.append(-math.inf)
                else:
                    dot = q8 @ mean[pg, h].astype(np.int64)
                    score.append(float(((dot.astype(f) * (amax / f(127))) * f(mean_scale[pg, h])).max()))
            k = min(n, top_k)
            best = sorted(range(n), key=lambda i: (-score[i], i))[:k]
            sel[b, h, :k] = sorted(best)
            count[b, h] = k
    return sel, count


# ------------------------------------------------------------------ attend
def attend(q, cu, lens, table, kc, vc, ks, vs, scale, page, sel=None, count=None):
    """O, LSE, the weights' mean of |v| and the largest |score| of each row, in 64 bits; rows that
    read a page outside the cache are NaN."""
    T, Hq, D = q.shape
    num_pages, Hkv = kc.shape[:2]
    G, B = Hq // Hkv, len(lens)
    o, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    size, top = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(B):
        q0, q1 = (min(max(int(c), 0), T) for c in (cu[b], cu[b + 1]))
        L = min(max(int(lens[b]), 0), table.shape[1] * page)
        n_pages = -(-L // page)
        for h in range(Hkv):
            pos = list(range(n_pages)) if sel is None else [int(i) for i in sel[b, h, :count[b, h]]]
            for t in range(q0, q1):
                limit = L - (q1 - q0) + (t - q0) + 1
                keys, vals, bad = [], [], False
                for i in pos:
                    inside = 0 <= i < n_pages
                    if inside and i * page >= limit:
                        continue
                    pg = table[b, i] if inside else -1
                    if not 0 <= pg < num_pages:
                        bad = True
                        continue
                    m = min(page, limit - i * page)
                    keys.append(E4M3[kc[pg, h, :m]] * float(ks[pg, h]))
                    vals.append(E4M3[vc[pg, h, :m]] * float(vs[pg, h]))
                for g in range(G):
                    r = h * G + g
                    if bad:
                        o[t, r], lse[t, r] = math.nan, math.nan
                        continue
                    if not keys:
                        o[t, r], lse[t, r] = 0.0, -math.inf
                        continue
                    K, V = np.concatenate(keys), np.concatenate(vals)
                    s = scale * (K @ q[t, r])
                    mx = s.max()
                    p = np.exp(s - mx)
                    o[t, r], lse[t, r] = p @ V / p.sum(), mx + math.log(p.sum())
                    size[t, r], top[t, r] = p @ np.abs(V) / p.sum(), np.abs(s).max()
    return o, lse, size, top


def check_attend(o, lse, ref, what="", rows=None):
    """O and LSE against `ref` (attend's answer).

    Tolerances, counted before any run: the weights are rounded to fp16 (half a step: 2^-11 of
    each, so 2^-11 of the weights' mean of |v|) and O once to bf16 (2^-8 of itself); an exponent of
    magnitude x carries a few fp32 roundings (2^-24 each) and exp2 two units in the last place, so
    weights are off by at most 2^-20 (1 + x) and so are l, O's share of it and LSE."""
    ro, rl, size, top = ref
    o, lse = f64(o), f64(lse)
    if rows is not None:
        o, lse, ro, rl, size, top = (a[:rows] for a in (o, lse, ro, rl, size, top))
    assert np.array_equal(np.isnan(ro), np.isnan(o)), f"{what}: NaN rows differ"
    assert np.array_equal(np.isnan(rl), np.isnan(lse)) and np.array_equal(np.isinf(rl), np.isinf(lse)), f"{what}: LSE"
    x = (1 + top * 1.4427) * 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * x[..., None]) * size * (1 + 2.0 ** -7) + 1e-30
    err = np.abs(o - ro)
    fine = np.isfinite(ro)
    assert (err[fine] <= tol[fine]).all(), f"{what}: O off by {np.max((err / tol)[fine])} of what is allowed"
    fine = np.isfinite(rl)
    el = np.abs(lse - rl, where=fine, out=np.zeros_like(rl))
    tl = x + 2.0 ** -22 * np.abs(np.where(fine, rl, 0))
    assert (el[fine] <= tl[fine]).all(), f"{what}: LSE off by {np.max((el / tl)[fine])} of what is allowed"


# ------------------------------------------------------------------ inputs
class Cache:
    """A random paged cache on a device, with B sequences' pages in a shuffled block table.  Rows
    behind a sequence's last token hold `stale` codes (NaN by default)."""

    def __init__(self, lens, Hkv, page, D, seed, extra_cols=1, num_pages=None, stale=0x7F, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.Hkv, self.D = list(lens), page, Hkv, D
        n = [-(-max(L, 0) // page) for L in lens]
        self.num_pages = max(num_pages or 0, sum(n) + 2)
        ids = rng.permutation(self.num_pages)[:sum(n)]
        self.table = np.full((len(lens), max(n + [1]) + extra_cols), -7, np.int32)
        at = 0
        shape = (self.num_pages, Hkv, page, D)
        kx, vx = (torch.randn(shape, generator=g, dtype=torch.float64).numpy() for _ in range(2))
        self.ks, self.vs = (2.0 ** rng.integers(-9, -5, size=shape[:2]) for _ in range(2))
        self.kc, self.vc = to_e4m3(kx / self.ks[..., None, None]), to_e4m3(vx / self.vs[..., None, None])
        for b, m in enumerate(n):
            self.table[b, :m] = ids[at:at + m]
            at += m
            if m and lens[b] % page:
                for c in (self.kc, self.vc):
                    c[self.table[b, m - 1], :, lens[b] % page:] = stale
        self.mean = rng.integers(-127, 128, size=(self.num_pages, Hkv, D)).astype(np.int8)
        self.ms = np.exp(0.3 * rng.standard_normal(shape[:2])).astype(np.float32) / 64
        t = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=dt)  # noqa: E731
        self.d_table, self.d_lens = t(self.table), t(np.array(lens, np.int32))
        self.d_kc, self.d_vc = t(self.kc), t(self.vc)
        self.d_ks, self.d_vs = t(self.ks, torch.float32), t(self.vs, torch.float32)
        self.d_mean, self.d_ms = t(self.mean), t(self.ms)

    @property
    def pages(self):
        return self.d_kc, self.d_vc, self.d_ks, self.d_vs


def queries(counts, Hq, D, seed, pad=0, mult=1.0, device="cuda"):
    """Packed query tokens as a strided slice of a wider tensor, and cu_q."""
    g = torch.Generator().manual_seed(seed)
    T = max(1, sum(counts) + pad)
    wide = (torch.randn((T, Hq + 2, D), generator=g) * mult).to(torch.bfloat16).to(device)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return wide[:, :Hq], cu, torch.from_numpy(cu).to(device)
